"""The tile kernel of the INT8 products at the ends of its ranges: the longest K with sums next to +-2^31, rows
as far apart as 32-bit offsets inside a tile allow, experts and up rows past 4 GiB of weights."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import close, dev
from _int8 import matmul_inputs, matmul_reference, quantised_close

pytestmark = pytest.mark.gpu

BF16, FP32, I8 = torch.bfloat16, torch.float32, torch.int8


def _call(tile_rows, what, *args, **kw):
    call = F.GroupedMatmulInt8Call(*args, **kw)
    plan = F.moe_grouped_matmul_int8_plan(call.desc)
    print(what, plan, flush=True)
    assert plan["lds_tiles"] and plan["tile_rows"] == tile_rows
    out = call.run()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("rows,n,tile_rows,epilogue,dtype", [(600, 4096, 64, "none", FP32), (1100, 4096, 128, "none", FP32),
                                                             (1100, 8192, 256, "none", FP32), (300, 8192, 64, "swiglu", FP32),
                                                             (600, 8192, 128, "swiglu", BF16), (1100, 8192, 256, "swiglu", I8)])
def test_the_longest_k_of_the_largest_codes(rows, n, tile_rows, epilogue, dtype):
    # -128 * -128 * 131056 is 2^31 - 262144; two kinds of rows, two of columns
    k, odd = 131056, rows // 2
    x, w = torch.full((rows, k), -128, dtype=I8, device="cuda"), torch.full((1, n, k), -128, dtype=I8, device="cuda")
    x[odd, ::3] = 127
    w[0, 1::2] = 127
    xs, ws = torch.full((rows,), 2.0 ** -30, device="cuda"), torch.ones((1, n), device="cuda")
    swiglu = epilogue == "swiglu"
    out = _call(tile_rows, f"largest sums {rows} x {n} {epilogue} {dtype}", x, xs, w, ws, out_dtype=dtype,
                epilogue=F.FFNWB_EPI_SWIGLU if swiglu else F.FFNWB_EPI_NONE)
    # the same rows and columns once each (SwiGLU: gate and up columns of either kind; n / 2 is even)
    c = dict(x=x[[0, odd]].cpu().numpy(), xs=np.full(2, 2.0 ** -30, np.float32), w=w[:, [0, 1, 0, 1] if swiglu else [0, 1]].cpu().numpy(),
             ws=np.ones((1, 4 if swiglu else 2), np.float32))
    want, off, _ = matmul_reference(c, None, epilogue, dtype)
    cols = n // 2 if swiglu else n
    row, col = (np.arange(rows) == odd).astype(int), np.arange(cols) % 2
    want, off = want[row][:, col], off[row][:, col]
    if dtype == I8:
        quantised_close(out["y"], out["y_scale"], want, off)
    else:
        close(out["y"], want, off, dtype)


@pytest.mark.parametrize("rows,k,n,tile_rows", [(615, 112, 1695, 32), (449, 80, 4376, 64), (656, 448, 6240, 128), (654, 80, 11910, 256)])
def test_rows_at_the_largest_stride_of_a_tile(rows, k, n, tile_rows):
    # rows 4 MiB apart: a tile of 256 spans 1 GiB
    c = matmul_inputs(rows + n, rows, k, n)
    x = torch.empty((rows, 1 << 22), dtype=I8, device="cuda")[:, 1 << 21:][:, :k]
    x.copy_(dev(c["x"]))
    y = _call(tile_rows, f"rows 4 MiB apart {rows} x {k} x {n}", x, dev(c["xs"]), dev(c["w"]), dev(c["ws"]), out_dtype=FP32)["y"]
    want, off, _ = matmul_reference(c)
    close(y, want, off, FP32)


@pytest.mark.parametrize("group_num,tile_rows", [(3, 64), (257, 32)])   # more than 256 are listed by a launch of their own
def test_experts_past_4_gib(group_num, tile_rows):
    # 9 experts of 512 MiB: the last one starts past 2^32 bytes
    n, k, rows = 4096, 131040, 600
    w = torch.zeros((9, n, k), dtype=I8, device="cuda")
    c = matmul_inputs(17, rows, k, 16)
    w[8, :8], w[8, n - 8:] = dev(c["w"][0, :8]), dev(c["w"][0, 8:])
    ws = torch.ones((9, n), device="cuda")
    ws[8, :8], ws[8, n - 8:] = dev(c["ws"][0, :8]), dev(c["ws"][0, 8:])
    groups = torch.zeros((group_num, 2), dtype=torch.int64)
    groups[0] = torch.tensor([8, rows])
    y = _call(tile_rows, f"experts past 4 GiB, {group_num} groups", dev(c["x"]), dev(c["xs"]), w, ws, group_list=groups.cuda(), out_dtype=FP32)["y"]
    want, off, _ = matmul_reference(c)
    close(torch.cat([y[:, :8], y[:, n - 8:]], 1), want, off, FP32)
    assert bool((y[:, 8:n - 8] == 0).all())


@pytest.mark.parametrize("f,rows,tile_rows,dtype", [(16400, 300, 128, FP32), (32640, 600, 256, BF16)])
def test_up_rows_past_2_gib(f, rows, tile_rows, dtype):
    # an up row lies F K bytes behind its gate row: 2^31 and some, and the last F below 2^32
    k = 131040
    c = matmul_inputs(19, rows, k, 32)
    w, ws = torch.zeros((1, 2 * f, k), dtype=I8, device="cuda"), torch.ones((1, 2 * f), device="cuda")
    at = [*range(8), *range(f - 8, f)]
    at += [f + i for i in at]
    w[0, at], ws[0, at] = dev(c["w"][0]), dev(c["ws"][0])
    y = _call(tile_rows, f"up rows past 2 GiB, F = {f}", dev(c["x"]), dev(c["xs"]), w, ws, epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=dtype)["y"]
    want, off, _ = matmul_reference(c, None, "swiglu", dtype)
    close(torch.cat([y[:, :8], y[:, f - 8:]], 1), want, off, dtype)
    assert bool((y[:, 8:f - 8] == 0).all())

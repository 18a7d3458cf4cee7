"""SwiGLU of the INT8 products where the sigmoid is among the smallest FP32 numbers: gates from -80 to -88.7,
beside values of u that bring the results back to ordinary size.

Gates and u are exact in FP32 (sums of one product, one scale of 1), so how far results may be off is
counted for SwiGLU alone.  Its 10 half-units of 2^-24, or in 16-bit results 8 and 2.02 |g| for the exponent's
own rounding, as in tests/_int8.py; and the rounding of the sigmoid, which is subnormal from -87.3 on: half a
step of 2^-149 beside values of 2^-128 or more, 2^-22."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import close, dev
from _int8 import SWIGLU, quantised_close

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


def _product(rows, gates, up, dtype):
    """Every row: gates[f] and u = up through the product, whole numbers of 1 and -1 times their channels' scales."""
    f, k = len(gates), 16
    x = np.zeros((rows, k), np.int8)
    x[:, :2] = 1
    w = np.zeros((1, 2 * f, k), np.int8)
    w[0, :f, 0], w[0, f:, 1] = np.where(gates < 0, -1, 1), 1
    ws = np.concatenate([np.abs(gates), np.full(f, up, np.float32)])[None].astype(np.float32)
    call = F.GroupedMatmulInt8Call(dev(x), torch.ones(rows, device="cuda"), dev(w), dev(ws), epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=dtype)
    plan = F.moe_grouped_matmul_int8_plan(call.desc)
    print(f"tail of the sigmoid {rows} x {f} {dtype} {plan}", flush=True)
    out = call.run()
    torch.cuda.synchronize()
    return out, plan


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16, I8])
@pytest.mark.parametrize("rows,tiles", [(4, 0), (1100, 1)])
def test_gates_whose_sigmoid_is_subnormal(rows, tiles, dtype):
    # INT8: only the subnormal ones, whose results a row's scale would otherwise hide
    gates = np.linspace(-87.4 if dtype == I8 else -80, -88.7, 2048).astype(np.float32)
    g, up = gates.astype(np.float64), 2.0 ** 120
    want = np.broadcast_to(g / (1 + np.exp(-g)) * up, (rows, len(g)))
    relative = SWIGLU + 2.0 ** -22 + (0 if dtype in (FP32, I8) else 2.02 * np.abs(g) * 2.0 ** -24)
    out, plan = _product(rows, gates, up, dtype)
    assert plan["lds_tiles"] == tiles
    if dtype == I8:
        quantised_close(out["y"], out["y_scale"], want, relative * np.abs(want))
    else:
        close(out["y"], want, relative * np.abs(want), dtype)


@pytest.mark.parametrize("rows,tiles", [(4, 0), (1100, 1)])
def test_gates_past_the_exponential(rows, tiles):
    # exp(-g) is infinite: the limit, and the largest gates as they are
    gates = np.resize(np.array([-88.75, -89, -200, -1e30, -3.4e38, 3.4e38, 1e30, 200], np.float32), 2048)
    out, plan = _product(rows, gates, 0.5, FP32)
    assert plan["lds_tiles"] == tiles
    want = torch.from_numpy(np.where(gates < 0, -0.0, gates * np.float32(0.5)).astype(np.float32)).cuda()
    assert torch.equal(out["y"], want.expand(rows, -1)) and torch.equal(out["y"].signbit(), want.signbit().expand(rows, -1))

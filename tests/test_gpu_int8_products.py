"""GPU parity of moe_grouped_matmul_int8 with its definition in 64 bits: every element of every
row, at the sizes, groups and layouts where it can go wrong.  Sums are exact, so the tolerance is
three roundings of the result, however much cancels."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import canary, dev, untouched
from _int8 import close, matmul_inputs, matmul_reference, quantised_close

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
NAMES = {BF16: "bf16", FP16: "fp16", FP32: "fp32", I8: "int8"}


def check(c, groups=None, epilogue="none", out_dtype=BF16, pad=0, what=""):
    """Runs the product into canaries, twice, and compares everything it wrote and left."""
    rows, n = c["x"].shape[0], c["w"].shape[1]
    f = n // 2 if epilogue == "swiglu" else n
    whole = canary((rows, f + pad), out_dtype)
    out = {"y": whole[:, :f]}
    if out_dtype == I8:
        out["y_scale"] = canary((rows, 3), FP32)[:, 1]
    # the gaps between the rows of x hold other codes
    x = torch.full((rows, c["x"].shape[1] + 48), 77, dtype=I8, device="cuda")
    x[:, :c["x"].shape[1]] = dev(c["x"])
    call = F.GroupedMatmulInt8Call(x[:, :c["x"].shape[1]], dev(c["xs"]), dev(c["w"]), dev(c["ws"]), out_dtype=out_dtype, out=out,
                                   group_list=None if groups is None else dev(np.array(groups, np.int64).reshape(-1, 2)),
                                   epilogue=F.FFNWB_EPI_SWIGLU if epilogue == "swiglu" else F.FFNWB_EPI_NONE)
    plan = F.moe_grouped_matmul_int8_plan(call.desc)
    print(f"int8 product {c['x'].shape} x {c['w'].shape} {NAMES[out_dtype]} {epilogue} {what} {plan}", flush=True)
    call.run()
    torch.cuda.synchronize()
    want, off, written = matmul_reference(c, groups, epilogue, out_dtype)
    w = dev(written)
    if out_dtype == I8:
        quantised_close(out["y"][w], out["y_scale"][w], want[written], off[written])
        side = out["y_scale"]._base.view(FP32).reshape(rows, 3)
        assert untouched(side[~w]) and untouched(side[:, :1]) and untouched(side[:, 2:])
    else:
        close(out["y"][w], want[written], off[written], out_dtype)
    assert untouched(whole[~w]) and (pad == 0 or untouched(whole[:, f:]))
    first = whole.clone()
    call.run()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.uint8), whole.view(torch.uint8))
    return plan


DENSE = [(1, 16, 1), (1, 16, 32), (1, 128, 16), (3, 48, 96), (16, 64, 64), (17, 80, 96), (33, 144, 160), (65, 272, 288), (100, 1040, 1000),
         (1, 7168, 512), (5, 4112, 272), (128, 128, 256), (129, 192, 544), (257, 400, 1056), (600, 336, 2080)]


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("size", DENSE, ids=str)
def test_dense(size, out_dtype):
    check(matmul_inputs(sum(size), *size), out_dtype=out_dtype, pad=5)


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32, I8])
@pytest.mark.parametrize("size", [s for s in DENSE if s[2] % 32 == 0], ids=str)
def test_dense_swiglu(size, out_dtype):
    check(matmul_inputs(sum(size) + 1, *size), epilogue="swiglu", out_dtype=out_dtype, pad=5)


GROUPS = {
    "uneven": [(0, 5), (2, 1), (3, 40), (5, 17)],
    "empty and bad": [(1, 0), (9, 3), (0, 16), (-1, 2), (4, -5), (5, 33), (0, 0)],
    "past the rows": [(3, 30), (1, 1 << 40), (2, 9)],
    "repeated key": [(4, 7), (4, 9), (1, 20), (4, 1)],
    "rows behind": [(2, 11), (3, 0), (0, 0)],
    "none": [(0, 0), (0, 0)],
    "large": [(0, 63), (1, 300), (5, 129)],
}


@pytest.mark.parametrize("epilogue,out_dtype", [("none", BF16), ("none", FP32), ("swiglu", FP16), ("swiglu", I8)])
@pytest.mark.parametrize("name", list(GROUPS))
def test_grouped(name, epilogue, out_dtype):
    check(matmul_inputs(len(name), 500 if name == "large" else 70, 272, 160, 6), GROUPS[name], epilogue, out_dtype, what=name)


@pytest.mark.parametrize("epilogue,out_dtype", [("none", BF16), ("swiglu", I8)])
def test_many_groups(epilogue, out_dtype):
    rng = np.random.default_rng(8)
    keys = np.sort(rng.permutation(3000)[:1500])
    groups = [(int(k) % 8, int(n)) for k, n in zip(keys, rng.integers(0, 3, 1500))] + [(0, 0)] * 500
    check(matmul_inputs(9, 1600, 128, 64, 8), groups, epilogue, out_dtype, what="2000 groups")


@pytest.mark.parametrize("epilogue,out_dtype", [("none", FP32), ("swiglu", I8)])
def test_the_most_groups_and_experts(epilogue, out_dtype):
    rng = np.random.default_rng(8192)
    m = rng.integers(0, 3, 8192)
    m[rng.integers(0, 8192, 4)] = 300
    keys = rng.permutation(8192)
    keys[::7] = 9000  # no expert
    check(matmul_inputs(3, int(m.sum()) + 5, 32, 64, 8192), list(zip(keys.tolist(), m.tolist())), epilogue, out_dtype)


@pytest.mark.parametrize("rows,n,epilogue,dtype", [(1, 64, "none", FP32), (40, 64, "swiglu", FP32), (300, 512, "none", FP32), (300, 512, "swiglu", I8)])
def test_the_longest_k_of_the_largest_codes(rows, n, epilogue, dtype):
    # -128 * -128 * 131056 is 2^31 - 262144: sums that reach the end of 32 bits on either side
    k = 131056
    c = dict(x=np.full((rows, k), -128, np.int8), xs=np.full(rows, 2.0 ** -30, np.float32), w=np.full((1, n, k), -128, np.int8),
             ws=np.full((1, n), 1.0, np.float32))
    c["w"][0, 1::2] = 127
    c["x"][rows // 2, ::3] = 127
    check(c, None, epilogue, dtype, what="largest sums")


# many rows: the largest tiles, K that ends inside a block, odd widths, more than 4096 tiles (whose
# list a launch of its own makes)
LARGE = [
    (1100, 272, 4104, BF16, "none", 1), (2304, 400, 1001, BF16, "none", 3), (2304, 400, 1001, FP32, "none", 3),
    (5000, 144, 2080, FP16, "swiglu", 7), (5000, 144, 2080, FP32, "swiglu", 7), (5000, 144, 2080, I8, "swiglu", 7),
    (3000, 528, 7168, BF16, "none", 1), (5000, 272, 4096, FP32, "none", 1), (6100, 272, 4128, I8, "swiglu", 5),
    (2500, 1040, 3008, BF16, "swiglu", 0), (2500, 1040, 3008, FP32, "none", 0),
    (20000, 272, 1024, FP16, "none", 8), (600, 80, 9248, I8, "swiglu", 3),
]


@pytest.mark.parametrize("rows,k,n,dtype,epilogue,experts", LARGE)
def test_large(rows, k, n, dtype, epilogue, experts):
    rng = np.random.default_rng(rows + n)
    groups = None
    if experts:
        cut = np.sort(rng.integers(0, rows, experts - 1))
        groups = [(int(e), int(m)) for e, m in enumerate(np.diff([0, *cut, rows]))]
    check(matmul_inputs(rows + k, rows, k, n, max(experts, 1)), groups, epilogue, dtype, pad=7 if dtype != I8 else 0)


# few tiles and a long K, which the waves of a workgroup split: blocks that they do not divide, odd widths, rows behind
SPLIT = [(300, 6160, 1333, FP16, "none", 0), (256, 7184, 2048, BF16, "none", 0), (520, 4112, 1504, FP32, "swiglu", 0),
         (260, 8192, 2080, BF16, "swiglu", 0), (330, 8000, 1600, I8, "swiglu", 0), (1000, 8192, 1056, I8, "swiglu", 3),
         (400, 12304, 1201, FP32, "none", 2), (200, 12304, 600, FP32, "none", 2)]


@pytest.mark.parametrize("rows,k,n,dtype,epilogue,experts", SPLIT)
def test_split_over_k(rows, k, n, dtype, epilogue, experts):
    groups = None if experts == 0 else [(e, (rows - 9) // experts) for e in range(experts)] + [(experts, 4)]
    plan = check(matmul_inputs(rows + k + n, rows, k, n, max(experts, 1)), groups, epilogue, dtype, pad=5)
    assert plan["waves"] > 1, "this size is not split"


def test_strided_scales_and_packed_rows():
    # the batching's INT8 rows as its data area packs them: the scale behind each row's codes
    rows, k, n = 50, 272, 96
    c = matmul_inputs(31, rows, k, n)
    packed = torch.zeros((rows, k + 16), dtype=I8, device="cuda")
    packed[:, :k] = dev(c["x"])
    scale = packed.view(FP32)[:, k // 4]
    scale.copy_(dev(c["xs"]))
    y = F.moe_grouped_matmul_int8(packed[:, :k], scale, dev(c["w"][0]), dev(c["ws"][0]), out_dtype=FP32)["y"]
    torch.cuda.synchronize()
    want, off, _ = matmul_reference(c)
    close(y, want, off, FP32)


@pytest.mark.parametrize("rows,dtype", [(5, FP32), (40, BF16), (700, FP32)])
def test_scales_that_are_not_finite_stay_in_their_rows_and_columns(rows, dtype):
    c = matmul_inputs(12, rows, 272, 96)
    c["x"][0], c["x"][1], c["w"][0, 7] = 5, 7, 3          # no zero sums beside infinities
    c["xs"][0], c["xs"][1], c["ws"][0, 7] = np.nan, np.inf, np.nan
    y = F.moe_grouped_matmul_int8(dev(c["x"]), dev(c["xs"]), dev(c["w"]), dev(c["ws"]), out_dtype=dtype)["y"]
    torch.cuda.synchronize()
    keep_r, keep_c = np.arange(rows) > 1, np.arange(96) != 7
    assert bool(y[0].isnan().all()) and not bool(y[1].isfinite().any()) and bool(y[:, 7].isnan().all())
    want, off, _ = matmul_reference(dict(c, xs=np.where(keep_r, c["xs"], 0), ws=np.where(keep_c, c["ws"], 0)))
    close(y[dev(keep_r)][:, dev(keep_c)], want[keep_r][:, keep_c], off[keep_r][:, keep_c], dtype)


def test_quantised_rows_that_are_not_finite_or_zero():
    c = matmul_inputs(13, 40, 128, 64)
    c["xs"][3], c["xs"][4] = np.nan, np.inf
    c["x"][5] = 0
    out = F.moe_grouped_matmul_int8(dev(c["x"]), dev(c["xs"]), dev(c["w"]), dev(c["ws"]), out_dtype=I8, epilogue=F.FFNWB_EPI_SWIGLU)
    torch.cuda.synchronize()
    q, s = out["y"].cpu().numpy(), out["y_scale"].cpu().numpy()
    assert np.isnan(s[3]) and not np.isfinite(s[4]) and s[5] == 2.0 ** -126
    assert (q[3:6] == 0).all()
    keep = np.delete(np.arange(40), [3, 4])
    want, off, _ = matmul_reference(dict(c, xs=np.nan_to_num(c["xs"], posinf=0)), None, "swiglu", I8)
    quantised_close(out["y"][dev(keep)], out["y_scale"][dev(keep)], want[keep], off[keep])


def test_no_rows():
    c = matmul_inputs(14, 4, 128, 32)
    out = F.moe_grouped_matmul_int8(dev(c["x"])[:0], dev(c["xs"])[:0], dev(c["w"]), dev(c["ws"]))
    assert out["y"].shape == (0, 32)


def test_rows_past_4_gib():
    # rows 64 MiB apart: the last ones start beyond 2^32 bytes, and 256 rows pass 32-bit offsets
    rows, k, n = 70, 256, 96
    c = matmul_inputs(16, rows, k, n)
    wide = torch.empty((rows, 1 << 26), dtype=I8, device="cuda")
    x = wide[:, 64:64 + k]
    x.copy_(dev(c["x"]))
    y = torch.empty((rows, 1 << 25), dtype=BF16, device="cuda")[:, :n]
    print("int8 product of rows 64 MiB apart", flush=True)
    F.moe_grouped_matmul_int8(x, dev(c["xs"]), dev(c["w"]), dev(c["ws"]), out={"y": y})
    torch.cuda.synchronize()
    want, off, _ = matmul_reference(c)
    close(y, want, off, BF16)


def test_weights_past_4_gib():
    n, k = 4096, 131040
    w = torch.zeros((9, n, k), dtype=I8, device="cuda")      # 4.8 GB; the last expert starts past 2^32 bytes
    c = matmul_inputs(17, 40, k, 16)
    w[8, :8], w[8, n - 8:] = dev(c["w"][0, :8]), dev(c["w"][0, 8:])
    ws = torch.ones((9, n), device="cuda")
    ws[8, :8], ws[8, n - 8:] = dev(c["ws"][0, :8]), dev(c["ws"][0, 8:])
    print("int8 product with weights past 4 GiB", flush=True)
    y = F.moe_grouped_matmul_int8(dev(c["x"]), dev(c["xs"]), w, ws, group_list=torch.tensor([[8, 40]], device="cuda"), out_dtype=FP32)["y"]
    torch.cuda.synchronize()
    want, off, _ = matmul_reference(c)
    close(torch.cat([y[:, :8], y[:, n - 8:]], 1), want, off, FP32)
    assert bool((y[:, 8:n - 8] == 0).all())


@pytest.mark.parametrize("dtype", [FP32, BF16, I8])
@pytest.mark.parametrize("rows", [4, 300])
def test_swiglu_over_its_whole_range(rows, dtype):
    # one product a column: gates from -110 to 110 and far beyond, infinities among the scales
    n, k = 512, 16
    c = dict(x=np.zeros((rows, k), np.int8), xs=np.ones(rows, np.float32), w=np.zeros((1, n, k), np.int8), ws=np.ones((1, n), np.float32))
    c["x"][:, 0], c["x"][:, 1] = 1, 3
    c["w"][0, :256, 0], c["w"][0, 256:, 1] = np.arange(256) - 128, 1
    c["ws"][0, :256] = 0.8671875
    c["xs"][1] = 7.0
    check(c, None, "swiglu", dtype, what="range of gates")
    c["xs"][2] = np.inf                                        # gates of +-inf, NaN where the sum is 0
    out = F.moe_grouped_matmul_int8(dev(c["x"]), dev(c["xs"]), dev(c["w"]), dev(c["ws"]), out_dtype=FP32, epilogue=F.FFNWB_EPI_SWIGLU)["y"]
    torch.cuda.synchronize()
    assert bool(out[2, :129].isnan().all()) and bool((out[2, 129:] == float("inf")).all())

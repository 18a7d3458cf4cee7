"""Every kernel of the experts' products, whole: each size asserts the kernel that it takes, so that
the tests keep reaching all of them when the rule that chooses changes.

Every element is compared with an FP32 product of the dequantised operands, as far as that may be
off; rows at the ends of groups and tiles, and others, with the definition in 64 bits.  K ends
inside a block of 128 and widths inside a tile; the gaps between the rows of x, one of its rows, one
weight row and a whole expert that has no rows hold NaN, which has to stay where the definition puts it."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import FP8, SWIGLU, canary, close, dev, dropped_bits, fp8, host, matmul_inputs, product_error, quantised_close, untouched
from oracle import expert_ffn as O

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = {BF16: "bf16", FP16: "fp16", FP32: "fp32", FP8: "fp8"}

# (rows, K, N, experts), type of the results, epilogue, kernel and tile rows, and how: "split" over K; row
# tiles "listed" by a launch of their own; of 128 and 256 rows, whether the last round of tiles is "halved"
FORMS = [
    ((21, 272, 131, 0), BF16, "none", "direct16", ""), ((24, 272, 131, 3), FP16, "none", "direct16", ""),
    ((21, 272, 131, 3), FP32, "none", "direct16", ""), ((369, 400, 341, 0), BF16, "none", "direct32", ""),
    ((594, 400, 197, 3), FP16, "none", "direct32", ""), ((655, 400, 177, 3), FP32, "none", "direct32", ""),
    ((641, 400, 699, 0), BF16, "none", "direct64", ""), ((1162, 400, 371, 3), FP16, "none", "direct64", ""),
    ((1117, 400, 385, 3), FP32, "none", "direct64", ""), ((20, 272, 288, 0), BF16, "swiglu", "direct16", ""),
    ((20, 272, 288, 3), FP16, "swiglu", "direct16", ""), ((20, 272, 288, 3), FP32, "swiglu", "direct16", ""),
    ((20, 400, 288, 0), FP8, "swiglu", "direct16", ""), ((875, 400, 288, 3), BF16, "swiglu", "direct32", ""),
    ((880, 400, 288, 3), FP16, "swiglu", "direct32", ""), ((456, 400, 576, 0), FP32, "swiglu", "direct32", ""),
    ((875, 400, 288, 3), FP8, "swiglu", "direct32", ""), ((1291, 400, 448, 3), BF16, "swiglu", "direct64", ""),
    ((642, 400, 896, 0), FP16, "swiglu", "direct64", ""), ((1276, 400, 448, 3), FP32, "swiglu", "direct64", ""),
    ((768, 912, 320, 3), FP8, "swiglu", "direct64", ""), ((729, 1040, 611, 0), BF16, "none", "tiles32", ""),
    ((1212, 1040, 355, 3), FP16, "none", "tiles32", ""), ((1338, 1040, 321, 3), FP32, "none", "tiles32", ""),
    ((1352, 1056, 1293, 0), BF16, "none", "tiles64", ""), ((2662, 1040, 519, 3), FP16, "none", "tiles64", ""),
    ((2659, 1040, 525, 3), FP32, "none", "tiles64", ""), ((4705, 2832, 3335, 0), BF16, "none", "tiles128", "halved"),
    ((3156, 1040, 1029, 3), BF16, "none", "tiles128", "whole"), ((3955, 1072, 819, 3), FP16, "none", "tiles128", "halved"),
    ((2377, 1056, 1557, 0), FP16, "none", "tiles128", "whole"), ((3964, 1040, 807, 3), FP32, "none", "tiles128", "halved"),
    ((3165, 1040, 1063, 3), FP32, "none", "tiles128", "whole"), ((4618, 1040, 3447, 0), BF16, "none", "tiles256", "halved"),
    ((5188, 1056, 1287, 3), BF16, "none", "tiles256", "whole"), ((7928, 1056, 897, 3), FP16, "none", "tiles256", "halved"),
    ((2965, 1072, 2561, 0), FP16, "none", "tiles256", "whole"), ((1543, 1040, 416, 3), BF16, "swiglu", "tiles32", ""),
    ((1352, 1040, 480, 3), FP16, "swiglu", "tiles32", ""), ((757, 1040, 864, 0), FP32, "swiglu", "tiles32", ""),
    ((1022, 1040, 448, 3), FP8, "swiglu", "tiles32", ""), ((2671, 1040, 544, 3), BF16, "swiglu", "tiles64", ""),
    ((1158, 1040, 1568, 0), FP16, "swiglu", "tiles64", ""), ((2675, 1072, 544, 3), FP32, "swiglu", "tiles64", ""),
    ((2682, 1040, 544, 3), FP8, "swiglu", "tiles64", ""), ((6833, 2832, 2336, 0), BF16, "swiglu", "tiles128", "halved"),
    ((4008, 1040, 800, 3), BF16, "swiglu", "tiles128", "whole"),
    ((3949, 1088, 800, 3), FP16, "swiglu", "tiles128", "halved"),
    ((2062, 1056, 1888, 0), FP16, "swiglu", "tiles128", "whole"),
    ((3949, 1072, 832, 3), FP32, "swiglu", "tiles128", "halved"),
    ((3985, 1040, 832, 3), FP32, "swiglu", "tiles128", "whole"),
    ((2986, 1040, 2592, 0), FP8, "swiglu", "tiles128", "halved"),
    ((3982, 1040, 800, 3), FP8, "swiglu", "tiles128", "whole"),
    ((7905, 1040, 960, 3), BF16, "swiglu", "tiles256", "halved"),
    ((3347, 1040, 2368, 0), BF16, "swiglu", "tiles256", "whole"),
    ((7906, 1136, 832, 3), FP16, "swiglu", "tiles256", "halved"),
    ((5219, 1040, 1312, 3), FP16, "swiglu", "tiles256", "whole"), ((485, 2080, 521, 0), BF16, "none", "tiles32", "split"),
    ((1098, 2112, 209, 3), FP16, "none", "tiles32", "split"), ((639, 2080, 357, 3), FP32, "none", "tiles32", "split"),
    ((843, 2112, 295, 0), BF16, "none", "tiles64", "split"), ((752, 2080, 309, 3), FP16, "none", "tiles64", "split"),
    ((1453, 1808, 419, 3), FP32, "none", "tiles64", "split"),
    ((1024, 3552, 329, 3), BF16, "none", "tiles128", "split halved"),
    ((895, 3616, 263, 3), BF16, "none", "tiles128", "split whole"),
    ((957, 2928, 637, 3), FP16, "none", "tiles128", "split halved"),
    ((1346, 4512, 271, 0), FP16, "none", "tiles128", "split whole"),
    ((128, 3488, 1357, 3), FP32, "none", "tiles128", "split halved"),
    ((764, 4112, 313, 3), FP32, "none", "tiles128", "split whole"),
    ((802, 1872, 672, 0), BF16, "swiglu", "tiles32", "split"), ((1198, 1840, 448, 3), FP16, "swiglu", "tiles32", "split"),
    ((1198, 2096, 448, 3), FP32, "swiglu", "tiles32", "split"), ((21, 6208, 288, 0), FP8, "swiglu", "tiles32", "split"),
    ((1318, 2160, 384, 3), BF16, "swiglu", "tiles64", "split"), ((1449, 2160, 352, 3), FP16, "swiglu", "tiles64", "split"),
    ((743, 2192, 800, 0), FP32, "swiglu", "tiles64", "split"), ((950, 1808, 480, 3), FP8, "swiglu", "tiles64", "split"),
    ((948, 2464, 544, 3), BF16, "swiglu", "tiles128", "split halved"),
    ((1798, 3104, 544, 0), BF16, "swiglu", "tiles128", "split whole"),
    ((946, 2384, 544, 3), FP16, "swiglu", "tiles128", "split halved"),
    ((956, 2640, 576, 3), FP16, "swiglu", "tiles128", "split whole"),
    ((1668, 2624, 320, 0), FP32, "swiglu", "tiles128", "split whole"),
    ((1500, 2576, 320, 3), FP8, "swiglu", "tiles128", "split whole"),
    ((21, 272, 131, 300), BF16, "none", "direct16", "listed"), ((182, 272, 131, 300), FP16, "none", "direct32", "listed"),
    ((178, 272, 133, 300), FP32, "none", "direct32", "listed"), ((291, 272, 305, 300), FP16, "none", "tiles32", "listed"),
    ((292, 272, 307, 300), FP32, "none", "tiles32", "listed"), ((215, 288, 411, 300), FP16, "none", "tiles128", "listed"),
    ((217, 272, 409, 300), FP32, "none", "tiles128", "listed"), ((210, 528, 320, 300), BF16, "swiglu", "tiles64", "listed"),
    ((3131, 368, 480, 300), FP32, "swiglu", "tiles64", "listed"),
]

# the same for 16-bit results that keep every bit of their products (`exact`); their direct kernels are those above
EXACT_FORMS = [
    ((1068, 1040, 403, 3), BF16, "none", "tiles32", ""), ((619, 1056, 721, 0), FP16, "none", "tiles32", ""),
    ((1683, 1040, 1055, 0), BF16, "none", "tiles64", ""), ((2720, 1040, 517, 3), FP16, "none", "tiles64", ""),
    ((3968, 1168, 845, 3), BF16, "none", "tiles128", "halved"), ((1812, 1040, 2141, 0), FP16, "none", "tiles128", "whole"),
    ((884, 1040, 736, 0), BF16, "swiglu", "tiles32", ""), ((1352, 1040, 480, 3), FP16, "swiglu", "tiles32", ""),
    ((2677, 1040, 544, 3), BF16, "swiglu", "tiles64", ""), ((1709, 1040, 1056, 0), FP16, "swiglu", "tiles64", ""),
    ((1853, 1040, 2080, 0), BF16, "swiglu", "tiles128", "whole"), ((3949, 1088, 800, 3), FP16, "swiglu", "tiles128", "halved"),
    ((474, 2112, 473, 3), FP16, "none", "tiles32", "split"), ((957, 2160, 451, 3), BF16, "none", "tiles64", "split"),
    ((1201, 2112, 448, 3), FP16, "swiglu", "tiles32", "split"), ((1500, 2608, 352, 3), BF16, "swiglu", "tiles128", "split whole"),
]


def _groups(rows, experts):
    """{key, rows} pairs: ragged groups and a tiny one, rows of no expert; or many groups; the last expert has none."""
    if experts == 0:
        return None
    if experts == 3:
        return [(2, rows * 9 // 20), (0, 5), (1, rows - rows * 9 // 20 - 9), (9, 4)]
    return [(i % 3, rows // experts + (i < rows % experts)) for i in range(experts)]


def _last_round_halved(plan, groups, rows, f, n, swiglu):
    """Whether the last tiles of each of the 8 XCDs, 32 at a time, are at most half a round."""
    bm, parts = plan["tile_rows"], plan["k_parts"]
    mt = sum(-(-m // bm) for _, m in groups) if groups else -(-rows // bm)
    nt = -(-n // 256) * parts if parts > 1 else -(-f // (128 if swiglu else 256))
    return 2 * (-(-mt * nt // 8) % 32) <= 32


def check_form(plan, size, dtype, epilogue, kernel, how, exact=False):
    rows, _, n, experts = size
    swiglu, groups = epilogue == "swiglu", _groups(rows, experts)
    assert ("tiles" if plan["lds_tiles"] else "direct") + str(plan["tile_rows"]) == kernel
    assert (plan["k_parts"] > 1) == ("split" in how) and bool(plan["listed"]) == ("listed" in how)
    if plan["tile_rows"] >= 128 and "listed" not in how:
        groups = [g for g in groups or [] if g[0] < 4]
        assert _last_round_halved(plan, groups, rows, n // 2 if swiglu else n, n, swiglu) == ("halved" in how)
    assert plan["e4m3_products"] == int(bool(plan["lds_tiles"]) and dtype in (BF16, FP16) and not exact)


def _reference(c, epilogue, e4m3):
    """(values, how far they may be off) of rows of one expert, in 64 bits from their codes."""
    n, k = c["w"].shape[1:]
    p, spread, _ = O.grouped_matmul(O.e4m3_values(c["x"]), c["xs"], O.e4m3_values(c["w"]), c["ws"])
    off = product_error(k) * spread
    if e4m3:
        off += dropped_bits(c["x"], c["xs"], c["w"][0], c["ws"][0])
    if epilogue == "none":
        return p, off
    g, u, dg, du = p[:, :n // 2], p[:, n // 2:], off[:, :n // 2], off[:, n // 2:]
    y = O.swiglu(g, u)
    return y, 1.1 * dg * (np.abs(u) + du) + np.abs(O.silu(g)) * du + SWIGLU * np.abs(y)


def _whole(c, x, w, groups, swiglu, e4m3):
    """(values, how far they may be off) of all rows, from FP32 products on the device."""
    k, n = c["x"].shape[1], c["w"].shape[1]
    cols = torch.arange(k, device="cuda") // 128
    xf = x.float() * dev(c["xs"])[:, cols]
    p, spread = torch.zeros((2, x.shape[0], n), device="cuda")
    at = 0
    for e, m in groups:
        if e < 4 and m:
            wf = w[e].float() * dev(c["ws"][e])[torch.arange(n, device="cuda") // 128][:, cols]
            p[at:at + m], spread[at:at + m] = xf[at:at + m] @ wf.t(), xf[at:at + m].abs() @ wf.abs().t()
        at += m
    # the FP32 products' own error, and all that e4m3 instructions may drop: 7 * 2^-13 of a group's largest
    # product, which is at most the sum of the group's sizes
    off = spread.double() * (2 * product_error(k) + (7 * 2.0 ** -13 if e4m3 else 0.0))
    p = p.double()
    if not swiglu:
        return p, off
    g, u, dg, du = p[:, :n // 2], p[:, n // 2:], off[:, :n // 2], off[:, n // 2:]
    silu = g * torch.sigmoid(g)
    y = silu * u
    return y, 1.1 * dg * (u.abs() + du) + silu.abs() * du + SWIGLU * y.abs()


def _all_close(out, want, off, rows, dtype):
    y = out["y"]
    nan = want.isnan()
    if dtype != FP8:
        got = y.double()[rows]
        assert torch.equal(got.isnan(), nan[rows])
        half, floor = {FP32: (2.0 ** -24, 2.0 ** -149), BF16: (2.0 ** -8, 2.0 ** -134), FP16: (2.0 ** -11, 2.0 ** -25)}[dtype]
        room = off * (1 + 2 * half) + half * want.abs() + floor
        assert bool((((got - want[rows]).abs() <= room[rows]) | nan[rows]).all())
        return
    f = want.shape[1]
    pad = -(-f // 128) * 128 - f
    blocks = [torch.nn.functional.pad(t, (0, pad)).view(t.shape[0], -1, 128) for t in (want, off)]
    amax, far = blocks[0].abs().amax(2), blocks[1].amax(2)
    s = out["y_scale"].double()
    assert torch.equal(s.isnan()[rows], amax.isnan()[rows])
    near = (s - (amax / 448).clamp_min(2.0 ** -126)).abs() <= far / 448 + amax / 448 * 2.0 ** -23
    assert bool((near | amax.isnan())[rows].all())
    sc = s[:, torch.arange(f, device="cuda") // 128]
    value = y.float().double() * sc
    room = torch.maximum(want.abs() * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -20) + off * (1 + 2.0 ** -4)
    assert bool((((value - want).abs() <= room) | sc.isnan())[rows].all())


def _picks(groups, rows, bm, rng):
    at, picks = 0, set(rng.integers(0, rows, 6).tolist())
    for e, m in groups[:12]:
        if m:
            full = m // bm * bm
            picks |= {at + i for i in (0, 16, bm // 2 - 1, bm // 2, bm - 1, bm, full - 1, full, m - 1) if 0 <= i < m}
        at += m
    return sorted(picks)


def _run(size, dtype, epilogue, exact=False):
    rows, k, n, experts = size
    swiglu, f = epilogue == "swiglu", n // 2 if epilogue == "swiglu" else n
    rng = np.random.default_rng(sum(size))
    c = matmul_inputs(sum(size), rows, k, n, 4 if experts else 1)
    groups = _groups(rows, experts)
    bad_row, bad_w = rows * 3 // 10, 131 % f
    c["x"][bad_row] = 0xFF
    if dtype != FP8:
        c["w"][0, bad_w] = 0x7F           # a column (SwiGLU: a gate column) of expert 0
    if experts:
        c["w"][3] = 0x7F                  # no rows
    gaps = np.full((rows, k + 48), 0x7F, np.uint8)
    gaps[:, 16:16 + k] = c["x"]
    x, w = fp8(gaps)[:, 16:16 + k], fp8(c["w"])
    wide = canary((rows, f + 16), dtype)
    out = {"y": wide[:, 3:3 + f]}
    if dtype == FP8:
        scales = canary((rows, -(-f // 128) + 2), FP32)
        out["y_scale"] = scales[:, 1:-1]
    call = F.GroupedMatmulFp8Call(x, dev(c["xs"]), w, dev(c["ws"]), out_dtype=dtype, out=out, exact=exact,
                                  group_list=None if groups is None else dev(np.array(groups, np.int64)),
                                  epilogue=F.FFNWB_EPI_SWIGLU if swiglu else F.FFNWB_EPI_NONE)
    plan = F.moe_grouped_matmul_fp8_plan(call.desc)
    print(f"product {size} {NAMES[dtype]} {epilogue}: {plan}", flush=True)
    call.run()
    torch.cuda.synchronize()
    groups = groups or [(0, rows)]
    e4m3 = bool(plan["e4m3_products"])
    written = np.repeat([e < 4 for e, _ in groups], [m for _, m in groups])
    written = np.concatenate([written, np.zeros(rows - len(written), bool)])
    want, off = _whole(c, x, w, groups, swiglu, e4m3)
    assert bool(want[bad_row].isnan().all())
    _all_close(out, want, off, dev(written), dtype)
    assert untouched(wide[:, :3]) and untouched(wide[:, 3 + f:]) and untouched(wide[dev(~written)])
    if dtype == FP8:
        assert untouched(scales[:, :1]) and untouched(scales[:, -1:]) and untouched(scales[dev(~written)])
    # the picked rows in 64 bits, those of an expert at a time
    picks = [r for r in _picks(groups, rows, plan["tile_rows"], rng) if written[r] and r != bad_row]
    owner = np.repeat([e for e, _ in groups], [m for _, m in groups])
    for e in range(3 if experts else 1):
        at = np.array([r for r in picks if owner[r] == e], int)
        if len(at) == 0:
            continue
        one = dict(x=c["x"][at], xs=c["xs"][at], w=c["w"][e:e + 1].copy(), ws=c["ws"][e:e + 1])
        one["w"][(one["w"] & 0x7F) == 0x7F] = 0
        v, o = _reference(one, epilogue, e4m3)
        rows_at = torch.from_numpy(at).cuda()
        if dtype == FP8:
            quantised_close(out["y"].view(torch.uint8)[rows_at].view(FP8), out["y_scale"][rows_at], v, o)
        else:
            cols = np.arange(f) != (bad_w if e == 0 else -1)
            close(out["y"][rows_at][:, dev(cols)], v[:, cols], o[:, cols], dtype)
    first = wide.clone()
    call.run()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.uint8), wide.view(torch.uint8))
    return plan


def _ids(v):
    return "x".join(map(str, v)) if isinstance(v, tuple) else NAMES.get(v, v) if not isinstance(v, str) else v.replace(" ", "-")


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", FORMS, ids=_ids)
def test_product_kernel(size, dtype, epilogue, kernel, how):
    check_form(_run(size, dtype, epilogue), size, dtype, epilogue, kernel, how)


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", EXACT_FORMS, ids=_ids)
def test_exact_product_kernel(size, dtype, epilogue, kernel, how):
    check_form(_run(size, dtype, epilogue, exact=True), size, dtype, epilogue, kernel, how, exact=True)


def _cancelling(rows, k, n):
    """Two products of 448 * 448 that cancel, and beside the first, in its group of 8 columns, seven of 10 to 15."""
    rng = np.random.default_rng(rows + n)
    x, w = np.zeros((rows, k), np.float64), np.zeros((1, n, k), np.float64)
    x[:, [0, 136]], w[0, :, 0], w[0, :, 136] = 448, 448, -448
    x[:, 1:8], w[0, :, 1:8] = rng.choice([3.0, 3.25, 3.5, 3.75], (rows, 7)), rng.choice([3.5, 3.75, 4.0], (n, 7))
    return dict(x=O.e4m3_bits(x), w=O.e4m3_bits(w), xs=np.ones((rows, -(-k // 128)), np.float32),
                ws=np.ones((1, -(-n // 128), -(-k // 128)), np.float32))


@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,k,n,tiles", [(3, 1040, 100, 0), (729, 1040, 611, 1), (494, 2080, 515, 1), (717, 1856, 893, 1)], ids=str)
def test_large_products_that_cancel(rows, k, n, tiles, dtype, exact):
    # the results, 70 to 105, are what is left of 2 * 448^2: FP32 sums are off by 8 at most (product_error of the sizes), and
    # e4m3 instructions by 7 * 2^-13 * 448^2 = 172 for each of the two groups, unless the caller refuses it
    c = _cancelling(rows, k, n)
    call = F.GroupedMatmulFp8Call(fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), out_dtype=dtype, exact=exact)
    plan = F.moe_grouped_matmul_fp8_plan(call.desc)
    if dtype != FP32 and not exact:
        assert plan["lds_tiles"] == plan["e4m3_products"] == tiles
    else:
        assert not plan["e4m3_products"]
    call.run()
    torch.cuda.synchronize()
    want, off = _reference(c, "none", bool(plan["e4m3_products"]))
    assert want.min() > 70 and off.max() < (360 if plan["e4m3_products"] else 8)
    print(f"cancelling {rows} x {k} x {n} {NAMES[dtype]}: {plan}, off by {np.abs(host(call.out['y']) - want).max():.3g}", flush=True)
    close(call.out["y"], want, off, dtype)


def test_exact_results_of_tiles_are_the_rounded_fp32_ones():
    # the tile kernels add the same blocks in the same order whatever the height
    for rows, k, n in ((3165, 1040, 1063), (1068, 1040, 803)):
        c = matmul_inputs(rows, rows, k, n)
        args = (fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]))
        calls = {t: F.GroupedMatmulFp8Call(*args, out_dtype=t, exact=True) for t in (BF16, FP16, FP32)}
        for call in calls.values():
            plan = F.moe_grouped_matmul_fp8_plan(call.desc)
            assert plan["lds_tiles"] and plan["k_parts"] == 1
            call.run()
        torch.cuda.synchronize()
        full = calls[FP32].out["y"]
        for t in (BF16, FP16):
            assert torch.equal(calls[t].out["y"], full.to(t))


def test_exact_leaves_fp32_and_e4m3_results_as_they_are():
    c = matmul_inputs(77, 700, 1040, 608)
    args = (fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]))
    for epilogue, dtype in ((F.FFNWB_EPI_NONE, FP32), (F.FFNWB_EPI_SWIGLU, FP32), (F.FFNWB_EPI_SWIGLU, FP8)):
        a, b, flag = (F.moe_grouped_matmul_fp8(*args, epilogue=e, out_dtype=dtype, exact=x)
                      for e, x in ((epilogue, False), (epilogue, True), (epilogue | F.FFNWB_EPI_EXACT, False)))
        torch.cuda.synchronize()
        for key in a:
            assert torch.equal(a[key].view(torch.uint8), b[key].view(torch.uint8))
            assert torch.equal(a[key].view(torch.uint8), flag[key].view(torch.uint8))

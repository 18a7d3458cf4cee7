"""GPU parity of the expert operators (moe_quant_fp8, moe_grouped_matmul_fp8, moe_layer)
against their definitions in 64 bits, at the sizes, layouts and masks where they can go
wrong."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import (FP8, canary, close, dev, fp8, host, layer_inputs, layer_reference, matmul_inputs, matmul_reference,
                     quantised_close, untouched)
from oracle import expert_ffn as O
from unpermute_ffnwb_batching_amd.hip_events import HipEvent

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


# ----------------------------------------------------------------------------- quantising

def _check_quant(x, call, rows=None):
    call.run()
    torch.cuda.synchronize()
    rows = x.shape[0] if rows is None else rows
    codes, scales = O.quantise_rows(x[:rows].float().cpu().numpy())
    q = call.out["q"]
    got = q[:rows].view(torch.uint8).cpu().numpy()
    nan = (codes & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)       # the sign of a NaN is free
    assert np.array_equal(got[~nan], codes[~nan])
    np.testing.assert_array_equal(call.out["scale"][:rows].cpu().numpy(), scales)


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 8), (3, 128), (5, 129), (7, 136), (2, 1000), (33, 7168), (130, 24)])
def test_quant(shape, dtype):
    g = torch.Generator().manual_seed(shape[0] * 10007 + shape[1])
    x = (torch.randn(shape, generator=g) * torch.exp(2 * torch.randn((shape[0], 1), generator=g))).to(dtype).cuda()
    print(f"quant {shape} {dtype}", flush=True)
    _check_quant(x, F.QuantFp8Call(x))


def test_quant_extreme_blocks():
    x = torch.zeros(12, 256)
    x[1, 0] = 1e-45                       # the smallest subnormal
    x[2, :5] = torch.tensor([1e-38, -3e-39, 1e-40, 0.0, 2e-38])
    x[3, 7], x[3, 8] = 3.4e38, -1e30      # near the largest float
    x[4, 3], x[4, 200] = float("inf"), 2.0
    x[5, 3], x[5, 4] = float("-inf"), float("nan")
    x[6] = float("nan")
    x[7] = torch.linspace(-448, 448, 256)
    x[8, :128] = 448 * 2.0 ** -85          # around the border of the two divisions
    x[9, :128] = 448 * 2.0 ** -80
    x[9, 5] = 1.7 * 2.0 ** -89
    x[10, 128:] = 448 * 2.0 ** 100
    x[11] = torch.arange(256) * 1.0009765625e-3
    print("quant: zeros, subnormals, largest values, infinities, NaN", flush=True)
    _check_quant(x.cuda(), F.QuantFp8Call(x.cuda()))


def test_quant_midpoints():
    # quotients at and one step beside every midpoint of e4m3, at scales that are no powers of two
    rng = np.random.default_rng(5)
    v = np.abs(O.e4m3_values(np.arange(0x7F, dtype=np.uint8)))
    mid = (v[1:] + v[:-1])[:124] / 2
    rows = []
    for _ in range(64):
        s = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-12, 12))
        m = (mid * s).astype(np.float32)
        for step in (-1, 0, 1):
            r = (m.view(np.int32) + step).view(np.float32)
            rows.append(np.concatenate([[448 * s], r, np.zeros(3)]).astype(np.float32))
    x = torch.from_numpy(np.stack(rows)).cuda()
    print("quant: midpoints", flush=True)
    _check_quant(x, F.QuantFp8Call(x))


def test_quant_strides_alignment_and_actual_rows():
    for hidden, pad, off, dtype in ((256, 64, 8, BF16), (250, 6, 3, FP16), (128, 4, 4, FP32), (130, 1, 1, FP32)):
        rows = 40
        base = torch.randn(rows, hidden + pad + off, device="cuda").to(dtype)
        x = base[:, off:off + hidden]
        for actual in (0, 1, 17, 40, 99, -3):
            q, s = canary((rows, hidden + 16), FP8), canary((rows, -(-hidden // 128) + 2), FP32)
            call = F.QuantFp8Call(x, actual_rows=torch.tensor([actual], device="cuda"),
                                  out={"q": q[:, 8:8 + hidden], "scale": s[:, 1:-1]})
            print(f"quant strided {hidden} {dtype} actual {actual}", flush=True)
            n = min(max(actual, 0), rows)
            _check_quant(x, call, n)
            assert untouched(q[n:]) and untouched(s[n:])
            assert untouched(q[:, :8]) and untouched(q[:, 8 + hidden:]) and untouched(s[:, :1]) and untouched(s[:, -1:])


# ----------------------------------------------------------------------------- products

def _matmul_call(c, groups=None, epilogue="none", out_dtype=BF16, out=None):
    gl = None if groups is None else torch.tensor(groups, dtype=torch.int64, device="cuda").reshape(-1, 2)
    return F.GroupedMatmulFp8Call(fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), group_list=gl,
                                  epilogue=F.FFNWB_EPI_SWIGLU if epilogue == "swiglu" else F.FFNWB_EPI_NONE,
                                  out_dtype=out_dtype, out=out)


def _check_matmul(c, groups=None, epilogue="none", out_dtype=BF16):
    rows, n = c["x"].shape[0], c["w"].shape[1]
    cols = n // 2 if epilogue == "swiglu" else n
    out = {"y": canary((rows, cols), out_dtype)}
    if out_dtype == FP8:
        out["y_scale"] = canary((rows, -(-cols // 128)), FP32)
    call = _matmul_call(c, groups, epilogue, out_dtype, out)
    call.run()
    torch.cuda.synchronize()
    want, off, written = matmul_reference(c, groups, epilogue, out_dtype in (BF16, FP16))
    y = call.out["y"]
    idx = torch.from_numpy(written).cuda()
    if out_dtype == FP8:
        quantised_close(y[idx], call.out["y_scale"][idx], want[written], off[written])
        assert untouched(call.out["y_scale"][~idx])
    else:
        close(y[idx], want[written], off[written], out_dtype)
    assert untouched(y[~idx])
    return call


DENSE = [(1, 16, 1), (1, 128, 32), (1, 1040, 100), (3, 144, 33), (16, 256, 130), (17, 128, 64), (33, 384, 256),
         (64, 1040, 200), (65, 112, 17), (129, 256, 257), (300, 640, 520), (520, 144, 300)]


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("size", DENSE, ids=str)
def test_dense_product(size, out_dtype):
    print(f"dense {size} {out_dtype}", flush=True)
    _check_matmul(matmul_inputs(sum(size), *size), out_dtype=out_dtype)


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32, FP8])
@pytest.mark.parametrize("size", [(1, 128, 32), (1, 1040, 512), (5, 144, 96), (17, 128, 288), (33, 512, 256), (70, 256, 800),
                                  (140, 384, 512), (300, 272, 544)], ids=str)
def test_dense_swiglu(size, out_dtype):
    print(f"dense swiglu {size} {out_dtype}", flush=True)
    _check_matmul(matmul_inputs(sum(size) + 1, *size), epilogue="swiglu", out_dtype=out_dtype)


GROUPS = {
    "uneven": [(0, 5), (2, 1), (3, 40), (5, 17)],
    "empty and bad": [(1, 0), (9, 3), (0, 16), (-1, 2), (4, -5), (5, 33), (0, 0)],
    "past the rows": [(3, 30), (1, 1 << 40), (2, 9)],
    "repeated key": [(4, 7), (4, 9), (1, 20), (4, 1)],
    "rows behind": [(2, 11), (3, 0), (0, 0)],
    "none": [(0, 0), (0, 0)],
    "large": [(0, 63), (1, 300), (5, 129)],
}


@pytest.mark.parametrize("epilogue,out_dtype", [("none", BF16), ("none", FP32), ("swiglu", FP16), ("swiglu", FP8)])
@pytest.mark.parametrize("name", list(GROUPS))
def test_grouped_product(name, epilogue, out_dtype):
    groups = GROUPS[name]
    rows = 500 if name == "large" else 70
    print(f"grouped {name} {epilogue} {out_dtype}", flush=True)
    _check_matmul(matmul_inputs(len(name), rows, 272, 160, 6), groups, epilogue, out_dtype)


def test_many_groups():
    rng = np.random.default_rng(8)
    keys = np.sort(rng.permutation(3000)[:1500])
    groups = [(int(k) % 8, int(n)) for k, n in zip(keys, rng.integers(0, 3, 1500))] + [(0, 0)] * 500
    print("grouped: 2000 groups", flush=True)
    _check_matmul(matmul_inputs(9, 1600, 128, 48, 8), groups)


def test_product_views_of_wider_buffers():
    c = matmul_inputs(11, 40, 272, 96)
    x = canary((40, 320), FP8)
    x[:, 16:288] = fp8(c["x"])
    xs = torch.full((40, 5), float("nan"), device="cuda")
    xs[:, 1:4] = dev(c["xs"])
    for epilogue, out_dtype in (("none", BF16), ("swiglu", FP8), ("none", FP32), ("swiglu", FP16)):
        cols = 48 if epilogue == "swiglu" else 96
        y = canary((40, cols + 7), out_dtype)
        out = {"y": y[:, 3:3 + cols]}
        if out_dtype == FP8:
            out["y_scale"] = canary((40, 3), FP32)[:, 1:2]
        call = F.GroupedMatmulFp8Call(x[:, 16:288], xs[:, 1:4], fp8(c["w"][0]), dev(c["ws"][0]), out_dtype=out_dtype, out=out,
                                      epilogue=F.FFNWB_EPI_SWIGLU if epilogue == "swiglu" else F.FFNWB_EPI_NONE)
        print(f"product of strided views {epilogue} {out_dtype}", flush=True)
        call.run()
        torch.cuda.synchronize()
        want, off, _ = matmul_reference(c, None, epilogue, out_dtype in (BF16, FP16))
        if out_dtype == FP8:
            quantised_close(out["y"], out["y_scale"], want, off)
        else:
            close(out["y"], want, off, out_dtype)
        assert untouched(y[:, :3]) and untouched(y[:, 3 + cols:])


def test_nan_and_infinite_scales_stay_in_their_rows():
    c = matmul_inputs(12, 70, 256, 96)
    c["x"][3, 5] = 0x7F
    c["xs"][40, 1] = np.inf
    c["xs"][41, 0] = np.nan
    y = _matmul_call(c, out_dtype=FP32)
    y.run()
    torch.cuda.synchronize()
    got = host(y.out["y"])
    bad = ~np.isfinite(got)
    assert bad[3].all() and bad[40].all() and bad[41].all()
    assert not bad[[i for i in range(70) if i not in (3, 40, 41)]].any()
    # unread: the rows of no group, and the weights of absent experts
    c = matmul_inputs(13, 64, 144, 64, 3)
    c["x"][30:] = 0x7F
    c["w"][1] = 0x7F
    print("product beside NaN rows and NaN experts", flush=True)
    _check_matmul(c, [(0, 20), (2, 10)], out_dtype=FP32)


def test_no_rows():
    c = matmul_inputs(14, 4, 128, 32)
    x, xs = fp8(c["x"])[:0], dev(c["xs"])[:0]
    out = F.moe_grouped_matmul_fp8(x, xs, fp8(c["w"]), dev(c["ws"]))
    assert out["y"].shape == (0, 32)
    assert F.moe_quant_fp8(torch.zeros(0, 64, device="cuda"))["q"].shape == (0, 64)
    assert F.moe_layer(torch.zeros(0, 64, device="cuda", dtype=BF16), torch.zeros(0, 2, device="cuda", dtype=torch.int32),
                       torch.zeros(2, 32, 64, device="cuda", dtype=BF16), torch.zeros(2, 64, 16, device="cuda", dtype=BF16)
                       )["y"].shape == (0, 64)
    torch.cuda.synchronize()


def _sampled(c, groups, picks, epilogue, narrow):
    # the picked rows' values, each with its own expert's weights
    ends = np.cumsum([0] + [n for _, n in groups])
    want, off = [], []
    for r in picks:
        e = groups[int(np.searchsorted(ends, r, side="right")) - 1][0]
        one = dict(x=c["x"][r:r + 1], xs=c["xs"][r:r + 1], w=c["w"][e:e + 1], ws=c["ws"][e:e + 1])
        v, o, _ = matmul_reference(one, None, epilogue, narrow)
        want.append(v)
        off.append(o)
    return np.concatenate(want), np.concatenate(off)


# many rows: the largest tiles, K that ends inside a block, odd widths, more than 4096 tiles (whose
# list a launch of its own makes)
LARGE = [
    (1100, 272, 8208, BF16, "none", 1), (2304, 400, 1001, BF16, "none", 3), (2304, 400, 1001, FP32, "none", 3),
    (5000, 144, 4128, FP16, "swiglu", 7), (5000, 144, 4128, FP32, "swiglu", 7), (5000, 144, 4128, FP8, "swiglu", 7),
    # a last round of tiles that is at most half full, whose tiles are halved
    (3000, 2048, 7168, BF16, "none", 1), (5000, 1040, 4096, FP32, "none", 1), (6100, 528, 4128, FP8, "swiglu", 5),
    (20000, 272, 1024, FP16, "none", 8),
    (40000, 128, 4096, BF16, "none", 32), (40000, 128, 8192, FP8, "swiglu", 32), (30000, 16, 8191, FP32, "none", 40),
]


@pytest.mark.parametrize("rows,k,n,dtype,epilogue,experts", LARGE)
def test_large_products(rows, k, n, dtype, epilogue, experts):
    rng = np.random.default_rng(rows + n)
    c = matmul_inputs(rows + k, rows, k, n, experts)
    cut = np.sort(rng.integers(0, rows, experts - 1))
    groups = [(int(e), int(m)) for e, m in enumerate(np.diff([0, *cut, rows]))]
    swiglu, f = epilogue == "swiglu", n // 2 if epilogue == "swiglu" else n
    out = {"y": canary((rows, f + 7 if dtype != FP8 else f), dtype)[:, :f]}
    if dtype == FP8:
        out["y_scale"] = canary((rows, -(-f // 128)), FP32)
    print(f"product {rows} x {k} x {n} {dtype} {epilogue}, {experts} experts", flush=True)
    got = F.moe_grouped_matmul_fp8(fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), out_dtype=dtype, out=out,
                                   group_list=dev(np.array(groups, np.int64)), epilogue=F.FFNWB_EPI_SWIGLU if swiglu else F.FFNWB_EPI_NONE)
    torch.cuda.synchronize()
    picks = np.unique(np.concatenate([[0, rows - 1], cut[:4], rng.integers(0, rows, 20), np.arange(rows - 390, rows, 13)]))
    want, off = _sampled(c, groups, picks, epilogue, dtype in (BF16, FP16))
    at = torch.from_numpy(picks).cuda()
    if dtype == FP8:
        quantised_close(got["y"].view(torch.uint8)[at].view(FP8), got["y_scale"][at], want, off)
    else:
        close(got["y"][at], want, off, dtype)
        whole = out["y"]._base.view(dtype).reshape(rows, f + 7)
        assert untouched(whole[:, f:])


# few tiles and a long K, which is split: parts that do not divide it, odd widths, rows behind
SPLIT = [(128, 7168, 1000, BF16, "none", 0), (128, 7184, 1001, FP32, "none", 0), (300, 6160, 333, FP16, "none", 0),
         (520, 4112, 1504, FP32, "swiglu", 0), (260, 8192, 1056, BF16, "swiglu", 0), (330, 8000, 800, FP8, "swiglu", 0),
         (1000, 8192, 1056, FP8, "swiglu", 3), (260, 8000, 1000, BF16, "none", 2), (200, 12304, 600, FP32, "none", 2)]


@pytest.mark.parametrize("rows,k,n,dtype,epilogue,experts", SPLIT)
def test_products_split_over_k(rows, k, n, dtype, epilogue, experts):
    c = matmul_inputs(rows + k + n, rows, k, n, max(experts, 1))
    swiglu, f = epilogue == "swiglu", n // 2 if epilogue == "swiglu" else n
    groups = None if experts == 0 else [(e, (rows - 9) // experts) for e in range(experts)] + [(experts, 4)]
    out = {"y": canary((rows, f + 5), dtype)[:, :f]}
    if dtype == FP8:
        out["y_scale"] = canary((rows, -(-f // 128) + 1), FP32)[:, :-1]
    call = F.GroupedMatmulFp8Call(fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), out_dtype=dtype, out=out,
                                  group_list=None if groups is None else dev(np.array(groups, np.int64)),
                                  epilogue=F.FFNWB_EPI_SWIGLU if swiglu else F.FFNWB_EPI_NONE)
    assert call.ws_bytes >= 2 * rows * n * 4, "this size is not split"
    print(f"split product {rows} x {k} x {n} {dtype} {epilogue}, {experts} experts", flush=True)
    call.run()
    torch.cuda.synchronize()
    want, off, written = matmul_reference(c, groups, epilogue, dtype in (BF16, FP16))
    w = dev(written)
    if dtype == FP8:
        quantised_close(out["y"].view(torch.uint8)[w].view(FP8), out["y_scale"][w], want[written], off[written])
        assert untouched(out["y_scale"].contiguous().view(torch.uint8)[~w])
    else:
        close(out["y"][w], want[written], off[written], dtype)
    assert untouched(out["y"].contiguous().view(torch.uint8)[~w])
    whole = out["y"]._base.view(torch.uint8).reshape(rows, -1)
    assert untouched(whole[:, f * out["y"].element_size():])
    first = {key: t.clone() for key, t in out.items()}
    for _ in range(10):
        call.run()
    torch.cuda.synchronize()
    for key, t in out.items():
        assert torch.equal(first[key].view(torch.uint8), t.contiguous().view(torch.uint8))


@pytest.mark.parametrize("rows", [5, 40, 300, 1500])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_nan_stays_in_its_rows_and_columns(rows, dtype):
    # K ends 16 into a block: what a tile reads past it are the next row's first columns, or the gap
    # between rows; both hold NaN here
    k, n, bad_row, bad_col = 272, 272, rows // 2, 130
    c = matmul_inputs(61, rows, k, n, 2)
    gaps = np.full((rows, 400), 0x7F, np.uint8)
    gaps[:, :k] = c["x"]
    gaps[bad_row, :k] = 0xFF
    c["w"][1, bad_col] = 0x7F
    c["w"][0] = 0x7F                            # an expert without rows
    x = fp8(gaps)[:, :k]
    print(f"NaN: {rows} rows {dtype}", flush=True)
    y = F.moe_grouped_matmul_fp8(x, dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), group_list=torch.tensor([[0, 0], [1, rows]], device="cuda"),
                                 out_dtype=dtype)["y"]
    torch.cuda.synchronize()
    nan = np.zeros((rows, n), bool)
    nan[bad_row], nan[:, bad_col] = True, True
    got = torch.isnan(y).cpu().numpy()
    assert (got == nan).all()
    clean = dict(c, w=np.where(c["w"][1:] == 0x7F, 0, c["w"][1:]), ws=c["ws"][1:])
    want, off, _ = matmul_reference(clean, None, "none", dtype == BF16)
    keep_rows, keep_cols = np.arange(rows) != bad_row, np.arange(n) != bad_col
    close(y[dev(keep_rows)][:, dev(keep_cols)], want[keep_rows][:, keep_cols], off[keep_rows][:, keep_cols], dtype)


@pytest.mark.parametrize("tokens", [3, 20])
def test_layer_nan_stays_with_its_token_and_expert(tokens):
    c = layer_inputs(62, tokens, 2, 6, 272, 144)
    c["ids"] = np.stack([[1, 3 if t % 2 else 4] for t in range(tokens)]).astype(np.int32)
    c["w13"][0], c["w2"][0], c["w13"][2], c["w2"][2], c["w13"][5], c["w2"][5] = (0x7F,) * 6   # nobody's experts
    xt = dev(c["x"], BF16)
    wide = torch.full((tokens, 400), float("nan"), dtype=BF16, device="cuda")
    wide[:, :272] = xt
    wide[1] = float("nan")
    args = dict(w13_scale=dev(c["w13s"]), w2_scale=dev(c["w2s"]), expert_scales=dev(c["scales"]))
    print(f"layer: NaN in one of {tokens} tokens", flush=True)
    y = F.moe_layer(wide[:, :272], dev(c["ids"]), fp8(c["w13"]), fp8(c["w2"]), **args)["y"]
    c4 = dict(c, w2=c["w2"].copy())
    c4["w2"][4, 17] = 0x7F                     # one column of one expert, of the even tokens
    y4 = F.moe_layer(xt, dev(c["ids"]), fp8(c4["w13"]), fp8(c4["w2"]), **args)["y"]
    torch.cuda.synchronize()
    for e in (0, 2, 5):
        c["w13"][e], c["w2"][e] = 0, 0
    want, off = layer_reference(c, xt)
    keep = np.arange(tokens) != 1
    assert bool(torch.isnan(y[1]).all())
    close(y[dev(keep)], want[keep], off[keep], BF16)
    nan = np.zeros((tokens, 272), bool)
    nan[::2, 17] = True
    assert (torch.isnan(y4).cpu().numpy() == nan).all()
    close(y4[1::2], want[1::2], off[1::2], BF16)


def test_quant_of_the_most_rows():
    # 2^28 - 16 rows of one element: the largest grid
    rows = (1 << 28) - 16
    x = torch.arange(rows, device="cuda", dtype=torch.int32).remainder_(2001).sub_(1000).to(FP16)[:, None]
    print("quant: 2^28 - 16 rows", flush=True)
    out = F.moe_quant_fp8(x)
    torch.cuda.synchronize()
    want, scales = O.quantise_rows(x[:2001].float().cpu().numpy())
    whole = rows // 2001 * 2001
    q = out["q"].view(torch.uint8)
    for t, w in ((q, dev(want)), (out["scale"], dev(scales))):
        assert bool((t[:whole].view(-1, 2001) == w.view(1, 2001)).all())
        assert torch.equal(t[whole:], w[:rows - whole])


def test_empty_calls_record_their_events():
    e = [(HipEvent(), HipEvent()) for _ in range(3)]
    F.moe_quant_fp8(torch.zeros(0, 64, device="cuda"), ev_quant=e[0])
    F.moe_grouped_matmul_fp8(torch.zeros(0, 64, device="cuda", dtype=torch.uint8).view(FP8), torch.zeros(0, 1, device="cuda"),
                             torch.zeros(32, 64, device="cuda", dtype=torch.uint8).view(FP8), torch.zeros(1, 1, device="cuda"),
                             ev_matmul=e[1])
    F.moe_layer(torch.zeros(0, 64, device="cuda", dtype=BF16), torch.zeros(0, 2, device="cuda", dtype=torch.int32),
                torch.zeros(2, 32, 64, device="cuda", dtype=BF16), torch.zeros(2, 64, 16, device="cuda", dtype=BF16), ev_layer=e[2])
    torch.cuda.synchronize()
    for b, end in e:
        assert 0.0 <= b.elapsed_ms(end) < 1000.0


def test_rows_past_4_gib():
    # rows 64 MiB apart: the last ones start beyond 2^32 bytes, and 256 rows pass 32-bit offsets
    rows, k, n = 70, 256, 96
    c = matmul_inputs(16, rows, k, n)
    stride = 1 << 26
    wide = torch.empty(rows * stride, dtype=torch.uint8, device="cuda").view(rows, stride)
    x = wide[:, 64:64 + k].view(FP8)
    x.view(torch.uint8).copy_(dev(c["x"]))
    y = torch.empty((rows, 1 << 25), dtype=BF16, device="cuda")[:, :n]
    q = wide[:, 4096:4096 + 130].view(FP8)
    print("product and quantising of rows 64 MiB apart", flush=True)
    F.moe_grouped_matmul_fp8(x, dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), out={"y": y})
    src = torch.randn(rows, 130, device="cuda")
    F.moe_quant_fp8(src, out={"q": q})
    torch.cuda.synchronize()
    want, off, _ = matmul_reference(c, None, "none", True)
    close(y, want, off, BF16)
    codes, _ = O.quantise_rows(src.cpu().numpy())
    np.testing.assert_array_equal(q.contiguous().view(torch.uint8).cpu().numpy(), codes)


def test_weights_past_4_gib():
    # the last expert's weights start beyond 2^32 bytes
    experts, n, k = 40, 8192, 16384
    c = matmul_inputs(15, 5, k, 64)
    w = torch.zeros((experts, n, k), dtype=torch.uint8, device="cuda").view(FP8)
    w[experts - 1, -64:] = fp8(c["w"][0])
    ws = torch.zeros((experts, n // 128, k // 128), device="cuda")
    ws[experts - 1, -1] = dev(c["ws"][0, 0])
    gl = torch.tensor([[experts - 1, 5]], device="cuda")
    print("product with 5 GiB of weights", flush=True)
    y = F.moe_grouped_matmul_fp8(fp8(c["x"]), dev(c["xs"]), w, ws, group_list=gl, out_dtype=FP32)["y"]
    want, off, _ = matmul_reference(c)
    close(y[:, -64:], want, off, FP32)
    assert (y[:, :-64] == 0).all()


# ----------------------------------------------------------------------------- layer

def _layer_call(c, dtype, mask=None, scales="own", ids=None, **kw):
    fp = c["w13s"] is not None
    w13, w2 = (fp8(c["w13"]), fp8(c["w2"])) if fp else (c["w13"].cuda(), c["w2"].cuda())
    return F.LayerCall(dev(c["x"], dtype), dev(c["ids"]) if ids is None else ids, w13, w2,
                       w13_scale=dev(c["w13s"]) if fp else None, w2_scale=dev(c["w2s"]) if fp else None,
                       expert_scales=dev(c["scales"]) if isinstance(scales, str) else scales,
                       active_mask=None if mask is None else dev(mask), **kw)


def _check_layer(c, dtype, mask=None):
    call = _layer_call(c, dtype, mask)
    call.run()
    torch.cuda.synchronize()
    want, off = layer_reference(c, dev(c["x"], dtype), mask)
    close(call.out["y"], want, off, dtype)
    return call


def test_layer_every_slot_an_expert_of_its_own():
    # 64 tokens x 64 slots over 8192 experts: the largest table (4096 experts of one token each)
    T, K, E, H, inter = 64, 64, 8192, 16, 16
    rng = np.random.default_rng(51)
    c = layer_inputs(52, T, K, 4, H, inter)
    pick = rng.permutation(E)[:T * K].reshape(T, K).astype(np.int32)
    kind = pick % 4                              # expert e has the weights of kind e % 4
    w13, w13s, w2, w2s = (np.tile(c[k], (E // 4,) + (1,) * (c[k].ndim - 1)) for k in ("w13", "w13s", "w2", "w2s"))
    call = F.LayerCall(dev(c["x"], BF16), dev(pick), fp8(w13), fp8(w2), w13_scale=dev(w13s), w2_scale=dev(w2s),
                       expert_scales=dev(c["scales"]))
    print("layer: 4096 experts", flush=True)
    call.run()
    torch.cuda.synchronize()
    c["ids"] = kind.astype(np.int32)
    want, off = layer_reference(c, dev(c["x"], BF16))
    close(call.out["y"], want, off, BF16)


def test_layer_every_token_on_the_same_experts():
    # 64 tokens on each of 5 experts: the widest operands, and groups of 16
    c = layer_inputs(53, 64, 5, 5, 272, 144)
    for dtype, weights in ((BF16, "fp8"), (FP16, "fp8"), (BF16, "bf16")):
        print(f"layer: 64 tokens to an expert {dtype} {weights}", flush=True)
        _check_layer(layer_inputs(53, 64, 5, 5, 272, 144, weights), dtype)


LAYERS = [(1, 1, 1, 16, 16), (1, 2, 4, 128, 32), (1, 9, 16, 272, 144), (2, 3, 16, 128, 256), (5, 4, 6, 144, 112),
          (16, 3, 8, 256, 128), (17, 2, 4, 400, 48), (33, 2, 3, 128, 144), (64, 8, 64, 64, 32), (64, 1, 2, 1040, 272),
          (64, 64, 64, 32, 16)]


@pytest.mark.parametrize("kind", [(BF16, "fp8"), (FP16, "fp8"), (BF16, "bf16")], ids=["bf16-fp8", "fp16-fp8", "bf16-bf16"])
@pytest.mark.parametrize("size", LAYERS, ids=str)
def test_layer(size, kind):
    dtype, weights = kind
    print(f"layer {size} {dtype} {weights}", flush=True)
    _check_layer(layer_inputs(sum(size), *size, weights), dtype)


def test_layer_masks_bad_ids_and_repeated_experts():
    c = layer_inputs(21, 12, 4, 10, 144, 48)
    c["ids"][0] = -1                       # no expert at all
    c["ids"][1] = [3, 3, 3, 3]             # one expert four times
    c["ids"][2] = [-7, 10, 1 << 30, 2]     # one of four in range
    c["ids"][3] = [5, 2, 5, 2]
    mask = np.random.default_rng(22).random((12, 4)) < 0.7
    mask[1], mask[2, 3], mask[4] = [True, False, True, True], True, False
    c["x"][0] = np.nan                     # tokens without an expert are not read
    c["x"][4] = np.inf
    for dtype in (BF16, FP16):
        print(f"layer: masks, bad and repeated ids {dtype}", flush=True)
        call = _layer_call(c, dtype, mask)
        call.run()
        torch.cuda.synchronize()
        x = dev(c["x"], dtype)
        x[0], x[4] = 0, 0
        want, off = layer_reference(c, x, mask)
        close(call.out["y"], want, off, dtype)
        zero = host(call.out["y"])[[0, 4]]
        assert (zero == 0).all() and not np.signbit(zero).any()


def test_layer_nothing_active():
    c = layer_inputs(23, 6, 3, 4, 64, 32)
    call = _layer_call(c, BF16, np.zeros((6, 3), bool), out={"y": canary((6, 64), BF16)})
    print("layer: every slot masked", flush=True)
    call.run()
    torch.cuda.synchronize()
    assert (call.out["y"] == 0).all()


@pytest.mark.parametrize("scale_dtype", [FP16, BF16, FP32, None])
def test_layer_id_and_scale_types_and_strided_views(scale_dtype):
    c = layer_inputs(24, 9, 4, 6, 144, 64)
    T, K, H = 9, 4, 144
    x = canary((T, H + 24), BF16)
    x[:, 8:8 + H] = dev(c["x"], BF16)
    ids = torch.full((T, K + 3), 1, dtype=torch.int64, device="cuda")
    ids[:, 2:2 + K] = dev(c["ids"])
    mask = np.random.default_rng(25).random((T, K)) < 0.8
    mw = torch.ones((T, K + 1), dtype=torch.bool, device="cuda")
    mw[:, 1:] = dev(mask)
    scales = None
    if scale_dtype is not None:
        sw = torch.full((T, K + 2), float("nan"), dtype=scale_dtype, device="cuda")
        sw[:, 1:1 + K] = dev(c["scales"], scale_dtype)
        scales = sw[:, 1:1 + K]
    y = canary((T, H + 5), BF16)
    call = F.LayerCall(x[:, 8:8 + H], ids[:, 2:2 + K], fp8(c["w13"]), fp8(c["w2"]), w13_scale=dev(c["w13s"]),
                       w2_scale=dev(c["w2s"]), expert_scales=scales, active_mask=mw[:, 1:], out={"y": y[:, 2:2 + H]})
    print(f"layer of strided views, scales {scale_dtype}", flush=True)
    call.run()
    torch.cuda.synchronize()
    want, off = layer_reference(c, x[:, 8:8 + H], mask, None if scales is None else host(scales))
    close(y[:, 2:2 + H], want, off, BF16)
    assert untouched(y[:, :2]) and untouched(y[:, 2 + H:])


def test_layer_many_experts():
    # 8192 experts, a few of them used, at both ends of the range
    c = layer_inputs(26, 3, 3, 6, 64, 32)
    place = np.array([0, 31, 32, 4095, 8190, 8191])
    big = dict(c, ids=place[c["ids"]].astype(np.int32))
    for name in ("w13", "w2"):
        b = np.zeros((8192,) + c[name].shape[1:], np.uint8)
        b[place] = c[name]
        s = np.zeros((8192,) + c[name + "s"].shape[1:], np.float32)
        s[place] = c[name + "s"]
        big[name], big[name + "s"] = b, s
    print("layer: 8192 experts", flush=True)
    call = _layer_call(big, BF16)
    call.run()
    torch.cuda.synchronize()
    want, off = layer_reference(c, dev(c["x"], BF16))
    close(call.out["y"], want, off, BF16)


def test_layer_large_activations_keep_their_range():
    # h far above the largest FP16: it is held in the range of FP32
    c = layer_inputs(27, 4, 2, 4, 128, 64)
    c["w13s"] *= 3000.0
    c["w2s"] *= 1e-6
    print("layer: |h| above 65504", flush=True)
    _check_layer(c, FP16)


# ----------------------------------------------------------------------------- together

def test_repeats_are_bit_identical():
    c = matmul_inputs(31, 200, 1040, 288, 5)
    lc = layer_inputs(32, 20, 4, 12, 272, 144)
    calls = [_matmul_call(c, [(0, 50), (2, 100), (4, 50)], "swiglu", FP8), _matmul_call(c, None if c["w"].shape[0] == 1 else
             [(1, 200)]), _layer_call(lc, BF16)]
    for call in calls:
        call.run()
        torch.cuda.synchronize()
        first = {k: v.clone() for k, v in call.out.items()}
        call.run()
        torch.cuda.synchronize()
        for k, v in first.items():
            assert torch.equal(v.view(torch.uint8), call.out[k].view(torch.uint8)), k

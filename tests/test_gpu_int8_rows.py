"""GPU parity of moe_quant_int8 and moe_rmsnorm_quant with their definitions, at the sizes,
layouts and values where they can go wrong."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import FP8, canary, host, quantised_close as fp8_close, untouched
from _int8 import close, norm_error, quantised_close
from oracle import int8_rows as O
from unpermute_ffnwb_batching_amd.hip_events import HipEvent

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8

# rows held by one wave (one and two runs), by a workgroup (one to four runs to a thread), and read twice; each
# at, below and past its border, whole runs of 8 and not
HIDDEN = [1, 7, 8, 127, 128, 129, 512, 513, 1000, 1024, 1025, 1032, 2047, 4095, 4096, 7168, 8192, 8193, 20000, 32768, 32769, 40000]


def _rows(seed, rows, hidden, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, hidden), generator=g) * torch.exp(2 * torch.randn((rows, 1), generator=g))).to(dtype)


# ----------------------------------------------------------------------------- quantising

def _check_quant(x, call, rows=None):
    call.run()
    torch.cuda.synchronize()
    rows = x.shape[0] if rows is None else rows
    codes, scales = O.quantise_rows(x[:rows].float().cpu().numpy())
    np.testing.assert_array_equal(call.out["scale"][:rows].cpu().numpy(), scales)
    np.testing.assert_array_equal(call.out["q"][:rows].cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32])
@pytest.mark.parametrize("hidden", HIDDEN)
def test_quant(hidden, dtype):
    for rows in (1, 6):
        print(f"quant int8 {rows} x {hidden} {dtype}", flush=True)
        x = _rows(hidden * 10 + rows, rows, hidden, dtype).cuda()
        _check_quant(x, F.QuantInt8Call(x))


@pytest.mark.parametrize("hidden", [256, 2000, 33000])
def test_quant_extreme_rows(hidden):
    x = torch.zeros(13, hidden)
    x[1, 0] = 1e-45                       # the smallest subnormal
    x[2, :5] = torch.tensor([1e-38, -3e-39, 1e-40, 0.0, 2e-38])
    x[3, 7], x[3, 8] = 3.4e38, -1e30      # near the largest float
    x[4, 3], x[4, 200] = float("inf"), 2.0
    x[5, 3], x[5, 255] = float("-inf"), float("nan")
    x[6] = float("nan")
    x[7] = torch.linspace(-127, 127, hidden)
    x[8, 1], x[8, 9] = 127 * 2.0 ** -80, 1.7 * 2.0 ** -81    # around the border of the two divisions
    x[9, 1], x[9, 9] = 127 * 2.0 ** -85, 63.5 * 2.0 ** -85
    x[10, 5] = 127 * 2.0 ** 101
    x[11] = torch.arange(hidden) * 1.0009765625e-3
    x[12] = torch.where(torch.arange(hidden) % 2 == 0, -0.0, 0.0)
    print("quant int8: zeros, subnormals, largest values, infinities, NaN", flush=True)
    _check_quant(x.cuda(), F.QuantInt8Call(x.cuda()))


def test_quant_nan_payloads():
    # NaNs of any payload and sign leave zeros
    x = torch.ones(4, 64)
    bits = x.view(torch.int32)
    bits[0, 3], bits[1, 3], bits[2, 63], bits[3, 0] = 0x7f800001, -1, 0x7fc00055, -0x3fffab
    codes = F.moe_quant_int8(x.cuda())
    torch.cuda.synchronize()
    assert bool((codes["q"] == 0).all()) and bool(codes["scale"].isnan().all())


def test_quant_midpoints():
    # quotients at and one step beside every midpoint of whole numbers, at scales that are no powers of two
    rng = np.random.default_rng(5)
    mid = np.arange(127) + 0.5
    rows = []
    for _ in range(64):
        s = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-12, 12))
        m = (mid[:126] * s).astype(np.float32) * rng.choice([-1, 1], 126).astype(np.float32)
        for step in (-1, 0, 1):
            rows.append(np.concatenate([[127 * s], (m.view(np.int32) + step).view(np.float32)]).astype(np.float32))
    x = torch.from_numpy(np.stack(rows)).cuda()
    print("quant int8: midpoints", flush=True)
    _check_quant(x, F.QuantInt8Call(x))


@pytest.mark.parametrize("hidden,pad,off,dtype", [(256, 64, 8, BF16), (250, 6, 3, FP16), (128, 4, 4, FP32), (130, 1, 1, FP32),
                                                  (3000, 1, 1, BF16), (35000, 3, 5, FP16)])
def test_quant_strides_alignment_and_actual_rows(hidden, pad, off, dtype):
    rows = 40
    x = torch.randn(rows, hidden + pad + off, device="cuda").to(dtype)[:, off:off + hidden]
    for actual in (0, 1, 17, 40, 99, -3):
        q, s = canary((rows, hidden + 10), I8), canary((rows, 3), FP32)
        call = F.QuantInt8Call(x, actual_rows=torch.tensor([actual], device="cuda"), out={"q": q[:, 5:5 + hidden], "scale": s[:, 1]})
        print(f"quant int8 strided {hidden} {dtype} actual {actual}", flush=True)
        n = min(max(actual, 0), rows)
        _check_quant(x, call, n)
        assert untouched(q[n:]) and untouched(s[n:])
        assert untouched(q[:, :5]) and untouched(q[:, 5 + hidden:]) and untouched(s[:, 0]) and untouched(s[:, 2])


def test_quant_rows_packed_with_their_scale():
    x = _rows(3, 9, 64, BF16).cuda()
    packed = canary((9, 68), I8)
    _check_quant(x, F.QuantInt8Call(x, out={"q": packed[:, :64], "scale": packed.view(FP32)[:, 16]}))
    assert not untouched(packed)


def test_quant_empty():
    out = F.moe_quant_int8(torch.empty((0, 16), dtype=BF16, device="cuda"))
    assert out["q"].shape == (0, 16) and out["scale"].shape == (0,)


# ----------------------------------------------------------------------------- norm

def _check_norm(x, gamma, residual, q_dtype, call, rows=None, eps=1e-6):
    out = call.run()
    torch.cuda.synchronize()
    rows = x.shape[0] if rows is None else rows
    f32 = [None if t is None else t[:rows].float().cpu().numpy() for t in (x, residual)]
    s, n = O.rmsnorm(f32[0], gamma.float().cpu().numpy(), f32[1], eps)
    off = norm_error(x.shape[1]) * np.abs(n)
    if residual is not None:
        want = torch.from_numpy(s).to(x.dtype)
        assert torch.equal(out["residual_out"][:rows].cpu(), want)
    if "y" in out:
        close(out["y"][:rows], n, off, x.dtype)
    (quantised_close if q_dtype == I8 else fp8_close)(out["q"][:rows], out["scale"][:rows], n, off)


@pytest.mark.parametrize("q_dtype", [I8, FP8])
@pytest.mark.parametrize("dtype,gamma_dtype", [(FP16, FP16), (FP16, FP32), (BF16, BF16), (BF16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("hidden", HIDDEN)
def test_norm(hidden, dtype, gamma_dtype, q_dtype):
    gamma = (1 + 0.3 * torch.randn(hidden, generator=torch.Generator().manual_seed(hidden))).to(gamma_dtype).cuda()
    for rows, with_residual, with_y in ((1, True, False), (6, False, True), (5, True, True)):
        print(f"norm {rows} x {hidden} {dtype} {gamma_dtype} -> {q_dtype}", flush=True)
        x = _rows(hidden * 10 + rows, rows, hidden, dtype).cuda()
        res = _rows(hidden * 10 + rows + 5, rows, hidden, dtype).cuda() if with_residual else None
        _check_norm(x, gamma, res, q_dtype, F.RmsNormQuantCall(x, gamma, residual=res, q_dtype=q_dtype, with_y=with_y))


@pytest.mark.parametrize("q_dtype", [I8, FP8])
@pytest.mark.parametrize("hidden,pad,off,dtype", [(256, 64, 8, BF16), (250, 6, 3, FP16), (130, 1, 1, FP32), (3000, 1, 1, BF16),
                                                  (35000, 3, 5, FP16)])
def test_norm_strides_alignment_and_actual_rows(hidden, pad, off, dtype, q_dtype):
    rows, wide = 24, hidden + pad + off
    x, res = (torch.randn(rows, w, device="cuda").to(dtype)[:, off:off + hidden] for w in (wide, wide + 2))
    gamma = torch.randn(hidden + 1, device="cuda").to(dtype)[1:]
    cols = 1 if q_dtype == I8 else -(-hidden // 128)
    for actual in (0, 1, 17, 24, 99, -3):
        q, s, y, ro = canary((rows, hidden + 10), q_dtype), canary((rows, cols + 2), FP32), canary((rows, hidden + 3), dtype), canary((rows, hidden + 4), dtype)
        out = {"q": q[:, 5:5 + hidden], "scale": s[:, 1] if q_dtype == I8 else s[:, 1:-1], "y": y[:, 1:1 + hidden],
               "residual_out": ro[:, 3:3 + hidden]}
        call = F.RmsNormQuantCall(x, gamma, residual=res, q_dtype=q_dtype, actual_rows=torch.tensor([actual], device="cuda"), out=out)
        print(f"norm strided {hidden} {dtype} {q_dtype} actual {actual}", flush=True)
        n = min(max(actual, 0), rows)
        _check_norm(x, gamma, res, q_dtype, call, n)
        for t in (q, s, y, ro):
            assert untouched(t[n:])
        assert untouched(q[:, :5]) and untouched(q[:, 5 + hidden:]) and untouched(s[:, :1]) and untouched(s[:, 1 + cols:])
        assert untouched(y[:, :1]) and untouched(y[:, 1 + hidden:]) and untouched(ro[:, :3]) and untouched(ro[:, 3 + hidden:])


@pytest.mark.parametrize("hidden", [96, 1500, 7168, 33000])
def test_norm_in_place(hidden):
    x, res = _rows(1, 5, hidden, BF16).cuda(), _rows(2, 5, hidden, BF16).cuda()
    gamma = torch.ones(hidden, dtype=BF16, device="cuda")
    want = F.moe_rmsnorm_quant(x, gamma, residual=res, with_y=True)
    got = F.moe_rmsnorm_quant(x, gamma, residual=res, with_y=True, out={"residual_out": res})
    torch.cuda.synchronize()
    assert got["residual_out"] is res
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("q_dtype", [I8, FP8])
def test_norm_values_that_are_not_finite(q_dtype):
    x = torch.ones(6, 300)
    x[0, 5], x[1, 6], x[2, 7], x[2, 8] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[3] = 1e25                      # squares past FP32: r is 0
    x[4] = 0.0
    out = F.moe_rmsnorm_quant(x.cuda(), torch.ones(300).cuda(), q_dtype=q_dtype, with_y=True)
    torch.cuda.synchronize()
    y, s = host(out["y"]), host(out["scale"]).reshape(6, -1)
    q = host(out["q"].float())
    assert np.isnan(y[0]).all() and np.isnan(y[2]).all() and np.isnan(s[[0, 2]]).all()
    assert np.isnan(y[1, 6]) and (np.delete(y[1], 6) == 0).all() and np.isnan(s[1, 0])
    assert (y[3] == 0).all() and (y[4] == 0).all() and (q[3] == 0).all() and (q[4] == 0).all()
    if q_dtype == I8:
        assert (q[:3] == 0).all()
    else:
        assert np.isnan(q[0, :128]).all() and np.isnan(q[2]).all()
    one = 1 / np.sqrt(1 + 1e-6)
    assert np.abs(y[5] - one).max() <= norm_error(300)
    assert np.abs(q[5] * np.repeat(s[5], 300 if q_dtype == I8 else 128)[:300] - one).max() <= norm_error(300) + 2.0 ** -23


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-12, 1e-5, 3.0])
def test_norm_epsilon(eps):
    x = torch.cat([_rows(7, 3, 200, FP32) * 1e-4, torch.zeros(1, 200)]).cuda()
    gamma = torch.ones(200).cuda()
    _check_norm(x, gamma, None, I8, F.RmsNormQuantCall(x, gamma, eps=eps, with_y=True), eps=np.float32(eps))


def test_norm_rows_past_4_gib_and_more_rows_than_workgroups():
    # x rows 1 MiB apart, 4100 of them; 2^21 workgroups take the rows past them in turn
    base = torch.zeros(4100 * (1 << 20), dtype=torch.uint8, device="cuda")
    x = base.view(BF16).view(4100, 1 << 19)[:, :24]
    x.copy_(_rows(11, 4100, 24, BF16).cuda())
    gamma = torch.ones(24, dtype=BF16, device="cuda")
    _check_norm(x, gamma, None, I8, F.RmsNormQuantCall(x, gamma, with_y=True))
    _check_quant(x, F.QuantInt8Call(x))
    del base, x
    rows = (1 << 21) + 5
    x = torch.randn((rows, 1040), device="cuda", dtype=BF16)
    q = F.moe_quant_int8(x)
    torch.cuda.synchronize()
    for part in (slice(0, 300), slice(rows - 300, rows)):
        codes, scales = O.quantise_rows(x[part].float().cpu().numpy())
        np.testing.assert_array_equal(q["q"][part].cpu().numpy(), codes)
        np.testing.assert_array_equal(q["scale"][part].cpu().numpy(), scales)


def test_hooks_and_streams():
    x = _rows(1, 300, 2048, BF16).cuda()
    gamma = torch.ones(2048, dtype=BF16, device="cuda")
    for make, hook in ((lambda **k: F.QuantInt8Call(x, **k), "ev_quant"), (lambda **k: F.RmsNormQuantCall(x, gamma, **k), "ev_norm")):
        want = {k: v.clone() for k, v in make().run().items()}
        ev = (HipEvent(), HipEvent())
        call = make(**{hook: ev})
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        call.run(side)
        side.synchronize()
        assert ev[0].elapsed_ms(ev[1]) >= 0
        for k in want:
            assert torch.equal(call.out[k], want[k])

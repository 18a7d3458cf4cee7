"""Results of the INT8 operators at the ends of their types: subnormal numbers, the border to infinity, ties.

Products of one code each with one scale are one FP32 multiplication, rounded once more to the result's type, so the bits have
to be those of the same two steps on the CPU.  So are those of the norm's sum."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import dev

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


def _scales(n):
    """From below the smallest subnormal of FP32 over FP16's and BF16's to the largest FP32, with full significands and
    with those that make ties."""
    rng = np.random.default_rng(4)
    full = rng.uniform(1, 2, n // 2) * 2.0 ** rng.integers(-149, 121, n // 2)
    fp16 = (rng.integers(0, 4096, n // 4) / 2) * 2.0 ** -25
    ties = (1 + rng.integers(0, 512, n - n // 2 - n // 4) / 512) * 2.0 ** rng.integers(-140, 18, n - n // 2 - n // 4)
    s = np.concatenate([full, fp16, ties]).astype(np.float32)
    s[:8] = [65504, 65519.996, 65520, 65536, 3.3895314e38, 3.39e38, 2.0 ** -149, 2.0 ** -126]
    return s


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("rows,tiles", [(4, 0), (1100, 1)])
def test_products(rows, tiles, dtype):
    k, ws = 16, _scales(4093)
    codes = np.array([1, -1, 127, -128, 3, 0, 100, -77], np.int8)
    x = np.zeros((rows, k), np.int8)
    x[:, 5] = np.resize(codes, rows)
    w = np.zeros((1, len(ws), k), np.int8)
    w[0, :, 5] = 1
    call = F.GroupedMatmulInt8Call(dev(x), torch.ones(rows, device="cuda"), dev(w), dev(ws[None]), out_dtype=dtype)
    plan = F.moe_grouped_matmul_int8_plan(call.desc)
    print(f"products at the ends of {dtype} {plan}", flush=True)
    assert plan["lds_tiles"] == tiles
    y = call.run()["y"]
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(x[:, 5:6].astype(np.float32) * ws).to(dtype)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("hidden", [96, 509, 4000, 7167, 17000])
def test_sum_of_the_norm(hidden, dtype):
    rng = np.random.default_rng(hidden)
    top = {FP32: 127, BF16: 127, FP16: 15}[dtype]
    low = {FP32: -149, BF16: -133, FP16: -24}[dtype]
    x, res = (torch.from_numpy((rng.choice([-1, 1], (5, hidden)) * rng.uniform(1, 2, (5, hidden)) * 2.0 ** rng.integers(low, top + 1, (5, hidden)))
                               .astype(np.float32)).to(dtype) for _ in range(2))
    x[0], res[0] = x[0].abs().clamp_min(1), x[0].abs().clamp_min(1)      # sums past the type, not past FP32 in 16 bits
    x[1], res[1] = torch.tensor(2.0 ** low, dtype=dtype), -x[0]
    out = F.moe_rmsnorm_quant(x.cuda(), torch.ones(hidden, dtype=dtype, device="cuda"), residual=res.cuda())
    print(f"sums at the ends of {dtype} {hidden}", flush=True)
    torch.cuda.synchronize()
    assert torch.equal(out["residual_out"].cpu(), (x.float() + res.float()).to(dtype))


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("hidden", [128, 515, 8000])
def test_normed_rows_that_are_subnormal(hidden, dtype):
    # rows of one value v: r = 2^-k exactly for v = 2^k without epsilon's part, so y = gamma rounded once
    low = {FP32: -149, BF16: -133, FP16: -24}[dtype]
    rng = np.random.default_rng(hidden)
    gamma = (rng.uniform(1, 2, hidden) * 2.0 ** rng.integers(low - 2, low + 14, hidden)).astype(np.float32)
    x = torch.full((3, hidden), 2.0 ** 13)
    x[1], x[2] = -2.0 ** 10, 2.0 ** 6
    out = F.moe_rmsnorm_quant(x.to(dtype).cuda(), dev(gamma), eps=2.0 ** -126, with_y=True)
    print(f"subnormal y {dtype} {hidden}", flush=True)
    torch.cuda.synchronize()
    # s gamma, exact, times r, whose sum, division, root and reciprocal are exact for equal powers of two up to 2^24 of them
    want = torch.from_numpy(np.sign(x.numpy()) * gamma).to(dtype)
    assert torch.equal(out["y"].cpu(), want)

"""moe_quant_int8 and moe_rmsnorm_quant at the borders between the shapes of their kernel, with row ends of every
length behind the last whole run of 8: rows held by 16 lanes (up to 128 elements), by a wave (512), by a
workgroup with one run of 8 to a thread (the norm, up to 4096) and two (16384), and rows read twice.

How far the norm may be off, in half-units of 2^-24 (each addition to a sum of positive terms loses one at
most): a thread's own squares, 6 steps in a wave and 4 over 16 waves, half of which reaches the root; then
5 for the division by H and epsilon's addition (half of either), root, reciprocal and two products."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import FP8, canary, quantised_close as fp8_close, untouched
from _int8 import close, quantised_close
from oracle import int8_rows as O

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8

HIDDEN = [9, 10, 11, 12, 13, 14, 15, 121, 128, 129, 130, 131, 132, 133, 134, 135, 505, 512, 513, 1026, 1027, 1028, 1029, 1030, 1031,
          4089, 4096, 4097, 4103, 4104, 9002, 9003, 9004, 9005, 9006, 12288, 16376, 16377, 16383, 16384, 16385, 16386, 16387, 16388,
          16389, 16390, 16391, 16392, 24577]
ROWS = 9


def _error(hidden):
    own = 8 * -(-hidden // 8192) if hidden > 16384 else 16 if hidden > 4096 else 8
    return ((own + 6 + 4) / 2 + 5) * 2.0 ** -24


def _rows(seed, hidden, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((ROWS, hidden), generator=g) * torch.exp(2 * torch.randn((ROWS, 1), generator=g))).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32])
@pytest.mark.parametrize("hidden", HIDDEN)
def test_quant(hidden, dtype):
    x = _rows(hidden, hidden, dtype)
    q, s = canary((ROWS, hidden + 3), I8), canary((ROWS,), FP32)
    print(f"quant int8 {hidden} {dtype}", flush=True)
    F.moe_quant_int8(x, out={"q": q[:, 1:1 + hidden], "scale": s})
    torch.cuda.synchronize()
    codes, scales = O.quantise_rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(q[:, 1:1 + hidden].cpu().numpy(), codes)
    assert untouched(q[:, :1]) and untouched(q[:, 1 + hidden:])


@pytest.mark.parametrize("q_dtype", [I8, FP8])
@pytest.mark.parametrize("dtype,gamma_dtype", [(FP16, FP16), (FP16, FP32), (BF16, BF16), (BF16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("hidden", HIDDEN)
def test_norm(hidden, dtype, gamma_dtype, q_dtype):
    x, res = _rows(hidden, hidden, dtype), _rows(hidden + 1, hidden, dtype)
    gamma = (1 + 0.3 * torch.randn(hidden, generator=torch.Generator().manual_seed(hidden))).to(gamma_dtype).cuda()
    wide = canary((3, ROWS, hidden + 2), dtype)
    q = canary((ROWS, hidden + 3), q_dtype)
    out = {"q": q[:, 1:1 + hidden], "y": wide[0, :, 1:1 + hidden], "residual_out": wide[1, :, 1:1 + hidden]}
    print(f"norm {hidden} {dtype} {gamma_dtype} -> {q_dtype}", flush=True)
    out = F.moe_rmsnorm_quant(x, gamma, residual=res, q_dtype=q_dtype, out=out)
    torch.cuda.synchronize()
    s, n = O.rmsnorm(x.float().cpu().numpy(), gamma.float().cpu().numpy(), res.float().cpu().numpy(), 1e-6)
    off = _error(hidden) * np.abs(n)
    assert torch.equal(out["residual_out"].cpu(), torch.from_numpy(s).to(dtype))
    close(out["y"], n, off, dtype)
    (quantised_close if q_dtype == I8 else fp8_close)(out["q"], out["scale"], n, off)
    for t in (q, wide[0], wide[1]):
        assert untouched(t[:, :1]) and untouched(t[:, 1 + hidden:])
    assert untouched(wide[2])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("hidden", [15, 127, 509, 4095, 7167, 16383, 16387, 33001])
def test_norm_in_place(hidden, dtype):
    x, res = _rows(1, hidden, dtype), _rows(2, hidden, dtype)
    gamma = torch.ones(hidden, dtype=dtype, device="cuda")
    want = F.moe_rmsnorm_quant(x, gamma, residual=res, with_y=True)
    got = F.moe_rmsnorm_quant(x, gamma, residual=res, with_y=True, out={"residual_out": res})
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k

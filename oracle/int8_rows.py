"""The INT8 operators in 64 bits (test infrastructure only): rows with a scale each, the norm
before the experts, and products with scales for each token and channel.

Written from the operators' definitions in include/ffnwb.h.  Where a definition fixes an FP32
rounding (a scale, a quotient, the sum with the residual) it is made here too; the rest is in 64
bits.

Pins (tests/test_oracle_int8_rows.py): quotients around every midpoint, the norm against
torch's own on the CPU, the products against a loop over rows.
"""

import numpy as np

from .expert_ffn import swiglu

TINY = np.float32(2.0 ** -126)


def quantise_rows(x):
    """x [R, H] (values exact in float32) -> (int8 codes [R, H], float32 scales [R])."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        scale = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)  # NaN wins
        scale = np.where(scale < TINY, TINY, scale)
        quotient = (x / scale[:, None]).astype(np.float32)
        codes = np.where(np.isfinite(scale)[:, None], np.rint(quotient), 0)
    return codes.astype(np.int8), scale


def rmsnorm(x, gamma, residual, epsilon):
    """(s [R, H] float32: the rows with their residual, n [R, H] float64: the normed rows)."""
    x = np.asarray(x, dtype=np.float32)
    s = x if residual is None else x + np.asarray(residual, dtype=np.float32)
    with np.errstate(all="ignore"):
        v = s.astype(np.float64)
        r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + epsilon)
        return s, v * np.asarray(gamma, dtype=np.float64) * r


def grouped_matmul(x, x_scale, w, w_scale, group_list=None, epilogue="none"):
    """Values [R, N or F], products [R, N], and whether each row is written.

    group_list: [(key, count), ...] or None for one dense product."""
    rows, n = x.shape[0], w.shape[1]
    p, written = np.zeros((rows, n)), np.zeros(rows, bool)
    at = 0
    for key, count in [(0, rows)] if group_list is None else group_list:
        count = min(max(int(count), 0), rows - at)
        if 0 <= key < w.shape[0] and count:
            part = slice(at, at + count)
            # whole numbers below 2^31: exact in 64-bit floats, whatever the order
            c = x[part].astype(np.float64) @ w[key].astype(np.float64).T
            p[part] = c * np.asarray(x_scale[part], np.float64)[:, None] * np.asarray(w_scale[key], np.float64)
            written[part] = True
        at += count
    return (swiglu(p[:, :n // 2], p[:, n // 2:]) if epilogue == "swiglu" else p), p, written

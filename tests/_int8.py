"""Helpers of the INT8 operators' GPU tests: seeded inputs, and tolerances from the rounding of
the operators' own arithmetic.

* A product's whole-number sum is exact; it is rounded to FP32, and so is each of the two
  products with scales: 3 half-units of 2^-24 of the result, whatever cancels (``PRODUCT``).
* SwiGLU, in half-units of 2^-24 relative: the exponential 2 and its correction 2 (at most as much in the
  sigmoid), its product with the sum 1, the reciprocal 2, two products 2: 9, and 1 for the rest of the
  exponent (``SWIGLU``).  Results that are rounded to 16 bits add |gate| half-units and 1 % for the
  exponent's own rounding, twice (the product with log2(e), and log2(e) itself).
* The norm sums squares in FP32, all terms positive: each addition loses half a unit of the sum
  so far, so the sum is off by (additions one after another) * 2^-24 relative: a thread's own
  elements (at most 32, or H / 1024 of them in rows read twice), 6 steps of a wave, 16 waves.  Half of that
  reaches the square root, then division by H, epsilon's addition, root, reciprocal (half of the
  first two reaches it), and the two products of n: ``norm_error(h)``.
* The scale of a row of n follows its largest value, whose error it shares, with one more
  rounding; a code is within half a step of its quotient, which has one rounding.
"""

import numpy as np
import torch

from _expert import FLOOR, HALF, host
from oracle import expert_ffn, int8_rows as O

PRODUCT = 3 * 2.0 ** -24 * (1 + 2.0 ** -20)
SWIGLU = 10 * 2.0 ** -24


def norm_error(h):
    return ((max(32, h / 1024) + 22) / 2 + 5) * 2.0 ** -24


def codes(rng, shape):
    """INT8 codes over the whole range, -128 among them."""
    return np.clip(np.rint(rng.normal(size=shape) * 50), -128, 127).astype(np.int8)


def matmul_inputs(seed, rows, k, n, experts=1):
    rng = np.random.default_rng(seed)
    return dict(x=codes(rng, (rows, k)), xs=(rng.uniform(0.5, 1.5, rows) / 50).astype(np.float32), w=codes(rng, (experts, n, k)),
                ws=(rng.uniform(0.5, 1.5, (experts, n)) / (50 * np.sqrt(k))).astype(np.float32))


def matmul_reference(c, groups=None, epilogue="none", dtype=torch.bfloat16):
    """(values, how far 32-bit arithmetic may be off, rows written); dtype: of the result."""
    y, p, written = O.grouped_matmul(c["x"], c["xs"], c["w"], c["ws"], groups, epilogue)
    off = PRODUCT * np.abs(p)
    if epilogue == "none":
        return y, off, written
    f = p.shape[1] // 2
    gate, up, dg, du = p[:, :f], p[:, f:], off[:, :f], off[:, f:]
    swiglu = SWIGLU + (0 if dtype in (torch.float32, torch.int8) else 2.02 * np.abs(gate) * 2.0 ** -24)
    return y, 1.1 * dg * (np.abs(up) + du) + np.abs(expert_ffn.silu(gate)) * du + swiglu * np.abs(y), written


def close(got, want, off, dtype):
    got = host(got)
    room = off * (1 + 2 * HALF[dtype]) + HALF[dtype] * np.abs(want) + FLOOR[dtype]
    bad = ~(np.abs(got - want) <= room)
    assert not bad.any(), (int(bad.sum()), got[bad][:3], want[bad][:3], room[bad][:3])


def quantised_close(q, scale, want, off):
    """INT8 rows and scales of finite values that are off by at most `off`."""
    assert q.dtype == torch.int8
    q, scale = host(q), host(scale)
    amax, far = np.abs(want).max(1), off.max(1)
    assert (np.abs(scale - np.maximum(amax / 127, 2.0 ** -126)) <= far / 127 + (amax + far) / 127 * 2.0 ** -24 + 2.0 ** -149).all()
    # half a step of the scale in use, the quotient's rounding (at most 127 * 2^-24 steps), and the value's error
    room = scale[:, None] * (0.5 + 127 * 2.0 ** -24) + off
    bad = ~(np.abs(q * scale[:, None] - want) <= room * (1 + 2.0 ** -40))
    assert not bad.any(), (int(bad.sum()), q[bad][:3], want[bad][:3])
    some = amax > 2.0 ** -100
    assert (np.abs(q[some]).max(1) == 127).all() and np.abs(q).max(initial=0) <= 127

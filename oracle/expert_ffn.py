"""The experts' own work in 64 bits (test infrastructure only): e4m3 rows with a scale for
each 128 elements, products with block-scaled weights, and a whole expert layer.

Written from the operators' definitions in include/ffnwb.h, with values (not storage bits)
in and out; ``e4m3_values`` / ``e4m3_bits`` convert.  Each product also returns ``spread``,
the sum of the absolute values of its terms, from which a test derives how far sums in
32 bits may be off.

Pins (tests/test_oracle_expert_ffn.py): e4m3 against torch's CPU conversion over every code
and around every midpoint, the products against plain dequantised matrix products, the
layer against a loop over tokens and slots.
"""

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def e4m3_values(bits):
    """uint8 e4m3 codes -> float64 (0x7f and 0xff are NaN)."""
    b = np.asarray(bits, dtype=np.uint8).astype(np.int64)
    exponent, mantissa = (b >> 3) & 15, b & 7
    v = np.where(exponent == 0, mantissa * 2.0 ** -9, (8 + mantissa) * 2.0 ** (exponent - 10.0))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b >> 7 == 1, -v, v)


def e4m3_bits(values):
    """Float values of magnitude up to 448 (or NaN) -> uint8 e4m3 codes, nearest, ties to even."""
    v = np.asarray(values, dtype=np.float64)
    mag = np.where(np.isnan(v), 0.0, np.abs(v))
    exponent = np.maximum(np.frexp(np.maximum(mag, 2.0 ** -40))[1] - 1, -6)
    steps = np.rint(mag / 2.0 ** (exponent - 3.0)).astype(np.int64)  # rint: halves to even
    # steps in [8, 16): normal with mantissa steps - 8; 16 carries into the next exponent
    code = np.where(steps < 8, steps, (exponent + 7) * 8 + steps - 8)
    code = np.where(np.isnan(v), 0x7F, code)
    if (code[~np.isnan(v)] > 0x7E).any():
        raise ValueError("magnitude above 448")
    return (code | ((np.signbit(v) & ~np.isnan(v)).astype(np.int64) << 7)).astype(np.uint8)


def quantise_rows(x):
    """x [R, H] (values exact in float32) -> (e4m3 codes [R, H], float32 scales [R, ceil(H / 128)])."""
    x = np.asarray(x, dtype=np.float32)
    rows, hidden = x.shape
    blocks = -(-hidden // BLOCK)
    codes, scales = np.empty((rows, hidden), np.uint8), np.empty((rows, blocks), np.float32)
    tiny = np.float32(2.0 ** -126)
    for i in range(rows):
        for b in range(blocks):
            part = x[i, b * BLOCK:(b + 1) * BLOCK]
            with np.errstate(all="ignore"):
                amax = np.max(np.abs(part))  # NaN wins
                s = np.float32(amax / np.float32(E4M3_MAX))
                s = tiny if s < tiny else s
                scales[i, b] = s
                codes[i, b * BLOCK:(b + 1) * BLOCK] = e4m3_bits((part / s).astype(np.float32))
    return codes, scales


def widen_weights(w, scale):
    """One expert's weights [n, k] times the scale of their 128 x 128 block (None: plain)."""
    w = np.asarray(w, dtype=np.float64)
    if scale is None:
        return w
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), BLOCK, 0), BLOCK, 1)
    return w * s[:w.shape[0], :w.shape[1]]


def widen_rows(x, scale):
    x = np.asarray(x, dtype=np.float64)
    return x * np.repeat(np.asarray(scale, np.float64), BLOCK, 1)[:, :x.shape[1]]


def silu(v):
    with np.errstate(over="ignore", invalid="ignore"):
        return v / (1.0 + np.exp(-v))


def swiglu(gate, up):
    return silu(gate) * up


def grouped_matmul(x, x_scale, w, w_scale, group_list=None, epilogue="none"):
    """Values [R, N or F], spreads of the products [R, N], and whether each row is written.

    group_list: [(key, count), ...] or None for one dense product."""
    rows, n = x.shape[0], w.shape[1]
    y, spread, written = np.zeros((rows, n)), np.zeros((rows, n)), np.zeros(rows, bool)
    at = 0
    for key, count in [(0, rows)] if group_list is None else group_list:
        count = min(max(int(count), 0), rows - at)
        if 0 <= key < w.shape[0] and count:
            a, b = widen_rows(x[at:at + count], x_scale[at:at + count]), widen_weights(w[key], w_scale[key])
            y[at:at + count], spread[at:at + count] = a @ b.T, np.abs(a) @ np.abs(b).T
            written[at:at + count] = True
        at += count
    if epilogue == "swiglu":
        y = swiglu(y[:, :n // 2], y[:, n // 2:])
    return y, spread, written


def layer(x, ids, w13, w13_scale, w2, w2_scale, scales=None, mask=None, relative=0.0, products=0.0):
    """(y, bound): the layer's values [T, H], and how far they may be off when every product
    is off by `products` of its spread and every h by `relative` of itself besides."""
    x = np.asarray(x, dtype=np.float64)
    tokens, slots = ids.shape
    inter = w2.shape[2]
    y, bound = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(tokens):
        for k in range(slots):
            e = int(ids[t, k])
            if not 0 <= e < w13.shape[0] or (mask is not None and not mask[t, k]):
                continue
            c = 1.0 if scales is None else float(scales[t, k])
            a = widen_weights(w13[e], None if w13_scale is None else w13_scale[e])
            b = widen_weights(w2[e], None if w2_scale is None else w2_scale[e])
            p, d = a @ x[t], products * (np.abs(a) @ np.abs(x[t]))
            gate, up = p[:inter], p[inter:]
            h = swiglu(gate, up)
            # |silu'| <= 1.1
            dh = 1.1 * d[:inter] * (np.abs(up) + d[inter:]) + np.abs(silu(gate)) * d[inter:] + relative * np.abs(h)
            y[t] += c * (b @ h)
            bound[t] += abs(c) * (np.abs(b) @ (dh + products * np.abs(h)))
    return y, bound

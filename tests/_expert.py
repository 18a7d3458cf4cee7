"""Helpers of the expert operators' GPU tests: seeded inputs, and tolerances from the
rounding of the operators' own arithmetic.

How far a result may be off, from the definition of the arithmetic:

* products of e4m3 (or 16-bit) values are exact in 32 bits; each addition of a term inside a
  128-element block may lose one unit of 2^-23 of the running sum (a matrix instruction may
  truncate), each later step (scale product, fused multiply-add, sums over waves) half of
  that: ``product_error(k)`` of the sum of the terms' absolute values;
* results in 16 bits may come from the e4m3 matrix instructions, which add products in groups of
  8 adjacent columns and drop the bits of each below 2^-13 of the power of two of the group's
  largest: at most 7 * 2^-13 of the largest product of each group (``dropped_bits``);
* SwiGLU in 32 bits: exp, a sum, a division and a product, 8 half-units of 2^-24 relative;
* a pair of BF16 numbers holds h to 2^-16 relative;
* the last rounding: half a step of the output's type.
"""

import numpy as np
import torch

from oracle import expert_ffn as O

FP8 = torch.float8_e4m3fn
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half of the smallest step, which subnormal results round to
FLOOR = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
SWIGLU = 8 * 2.0 ** -24


def product_error(k):
    return (2 * 128 + -(-k // 128) * 2 + 16) * 2.0 ** -24


def dropped_bits(x, xs, w, ws):
    """[R, N]: what the e4m3 matrix instructions may drop, for codes x [R, K] and one expert's w [N, K]."""
    a, b = np.abs(O.widen_rows(O.e4m3_values(x), xs)), np.abs(O.widen_weights(O.e4m3_values(w), ws))
    k = a.shape[1] // 8
    b = np.nan_to_num(b).reshape(b.shape[0], k, 8).astype(np.float32)
    rows = [(np.nan_to_num(r).reshape(1, k, 8).astype(np.float32) * b).max(2).sum(1) for r in a]
    return 7 * 2.0 ** -13 * np.array(rows, np.float64).reshape(a.shape[0], b.shape[0])


def codes(rng, shape):
    """e4m3 codes of a normal tensor that fills the range."""
    return O.e4m3_bits(np.clip(rng.normal(size=shape) * 130, -448, 448))


def fp8(bits):
    return torch.from_numpy(np.ascontiguousarray(bits)).cuda().view(FP8)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().cpu().to(torch.float64).numpy()


def canary(shape, dtype):
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")[:n].view(dtype).reshape(shape)


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == 0xA5).all())


def matmul_inputs(seed, rows, k, n, experts=1):
    rng = np.random.default_rng(seed)
    return dict(x=codes(rng, (rows, k)), xs=rng.uniform(0.5, 1.5, (rows, -(-k // 128))).astype(np.float32) / 130,
                w=codes(rng, (experts, n, k)),
                ws=(rng.uniform(0.5, 1.5, (experts, -(-n // 128), -(-k // 128))) / (130 * np.sqrt(k))).astype(np.float32))


def matmul_reference(c, groups=None, epilogue="none", narrow=False):
    """(values, how far sums may be off, rows written); narrow: the result is in 16 bits."""
    k, n = c["x"].shape[1], c["w"].shape[1]
    x, w = O.e4m3_values(c["x"]), O.e4m3_values(c["w"])
    p, spread, written = O.grouped_matmul(x, c["xs"], w, c["ws"], groups)
    off = product_error(k) * spread
    if narrow:
        at = 0
        for key, count in [(0, x.shape[0])] if groups is None else groups:
            count = min(max(int(count), 0), x.shape[0] - at)
            if 0 <= key < w.shape[0] and count:
                off[at:at + count] += dropped_bits(x[at:at + count], c["xs"][at:at + count], w[key], c["ws"][key])
            at += count
    if epilogue == "none":
        return p, off, written
    gate, up, dg, du = p[:, :n // 2], p[:, n // 2:], off[:, :n // 2], off[:, n // 2:]
    y = O.swiglu(gate, up)
    return y, 1.1 * dg * (np.abs(up) + du) + np.abs(O.silu(gate)) * du + SWIGLU * np.abs(y), written


def close(got, want, off, dtype):
    got = host(got)
    room = off * (1 + 2 * HALF[dtype]) + HALF[dtype] * np.abs(want) + FLOOR[dtype]
    bad = ~(np.abs(got - want) <= room)
    assert not bad.any(), (int(bad.sum()), got[bad][:3], want[bad][:3], room[bad][:3])


def quantised_close(q, scale, want, off):
    """e4m3 rows and scales of values that are off by `off`: the scale follows the block's
    largest value, each element is within half a step of e4m3 of the value."""
    rows, n = want.shape
    q, scale = host(q), host(scale)
    for b in range(-(-n // 128)):
        part = slice(b * 128, min(n, b * 128 + 128))
        amax, far = np.abs(want[:, part]).max(1), off[:, part].max(1)
        s = scale[:, b]
        assert (np.abs(s - np.maximum(amax / 448, 2.0 ** -126)) <= far / 448 + amax / 448 * 2.0 ** -23).all()
        value = q[:, part] * s[:, None]
        # half a step: 2^-4 of a normal value, 2^-10 scales below; (1 + 2^-4) carries the input's error along
        room = np.maximum(np.abs(want[:, part]) * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 2.0 ** -20) + off[:, part] * (1 + 2.0 ** -4)
        bad = ~(np.abs(value - want[:, part]) <= room)
        assert not bad.any(), (b, int(bad.sum()))


def layer_inputs(seed, tokens, slots, experts, hidden, inter, weights="fp8"):
    rng = np.random.default_rng(seed)
    c = dict(ids=np.stack([rng.permutation(experts)[:slots] if slots <= experts else rng.integers(0, experts, slots)
                           for _ in range(tokens)]).astype(np.int32).reshape(tokens, slots),
             scales=rng.uniform(0.1, 1, (tokens, slots)).astype(np.float32),
             x=rng.normal(size=(tokens, hidden)).astype(np.float32))
    for name, n, k in (("w13", 2 * inter, hidden), ("w2", hidden, inter)):
        if weights == "fp8":
            c[name] = codes(rng, (experts, n, k))
            c[name + "s"] = (rng.uniform(0.5, 1.5, (experts, -(-n // 128), -(-k // 128))) / (130 * np.sqrt(k))).astype(np.float32)
        else:
            c[name] = torch.from_numpy((rng.normal(size=(experts, n, k)) / np.sqrt(k)).astype(np.float32)).to(torch.bfloat16)
            c[name + "s"] = None
    return c


def layer_reference(c, xt, mask=None, scales="own"):
    """(values, how far 32-bit arithmetic may be off); xt: x in its 16-bit type."""
    fp = c["w13s"] is not None
    w13 = O.e4m3_values(c["w13"]) if fp else c["w13"].double().numpy()
    w2 = O.e4m3_values(c["w2"]) if fp else c["w2"].double().numpy()
    k = max(w13.shape[2], w2.shape[2])
    # besides the products: the weighted sum over up to 64 experts and 8 waves
    return O.layer(host(xt), c["ids"], w13, c["w13s"], w2, c["w2s"], c["scales"] if isinstance(scales, str) else scales, mask,
                   relative=SWIGLU + 2.0 ** -16, products=product_error(k) + 80 * 2.0 ** -24)

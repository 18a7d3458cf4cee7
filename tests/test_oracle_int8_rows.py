"""Pins of the INT8 operators' oracle."""

import numpy as np
import torch

from oracle import int8_rows as O


def test_quantise_by_hand():
    codes, scale = O.quantise_rows(np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.49], [0, 0, 0, 0, 0, 0, 0, -0.0],
                                             [254, 1, -1, 3, 5, 2, 0, 0]], np.float32))
    assert scale.tolist() == [1.0, np.float32(2.0 ** -126), 2.0]
    assert codes[0].tolist() == [127, -127, 0, 2, 2, 0, -2, 63]      # halves go to the even neighbour
    assert codes[1].tolist() == [0] * 8
    assert codes[2].tolist() == [127, 0, 0, 2, 2, 1, 0, 0]           # 0.5, -0.5, 1.5, 2.5


def test_quantise_is_within_half_a_step():
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(50, 300)) * np.exp(rng.normal(size=(50, 1)) * 4)).astype(np.float32)
    codes, scale = O.quantise_rows(x)
    assert np.abs(codes).max() == 127 and (np.abs(codes.astype(int)).max(1) == 127).all()
    off = np.abs(codes * scale[:, None].astype(np.float64) - x)
    assert (off <= scale[:, None] * (0.5 + 127 * 2.0 ** -23)).all()


def test_quantise_rows_that_are_not_finite():
    x = np.ones((3, 4), np.float32)
    x[0, 1], x[1, 2], x[2, 0], x[2, 1] = np.nan, np.inf, -np.inf, np.nan
    codes, scale = O.quantise_rows(x)
    assert (codes == 0).all() and np.isnan(scale[0]) and np.isposinf(scale[1]) and np.isnan(scale[2])


def test_norm_against_torch():
    rng = np.random.default_rng(4)
    x, r, g = rng.normal(size=(7, 65)).astype(np.float32), rng.normal(size=(7, 65)).astype(np.float32), rng.normal(size=65)
    s, n = O.rmsnorm(x, g, r, 1e-5)
    assert s.dtype == np.float32 and np.array_equal(s, x + r)
    want = torch.nn.functional.rms_norm(torch.from_numpy(s).double(), (65,), torch.from_numpy(g), 1e-5)
    np.testing.assert_allclose(n, want.numpy(), rtol=1e-12)
    s, n = O.rmsnorm(x, g, None, 1e-5)
    assert np.array_equal(s, x)


def test_products_against_a_loop():
    rng = np.random.default_rng(5)
    x, w = rng.integers(-128, 128, (9, 32)).astype(np.int8), rng.integers(-128, 128, (3, 8, 32)).astype(np.int8)
    xs, ws = rng.uniform(1, 2, 9), rng.uniform(1, 2, (3, 8))
    groups = [(2, 3), (7, 2), (0, -1), (0, 3), (1, 100)]
    y, p, written = O.grouped_matmul(x, xs, w, ws, groups)
    expert = [2, 2, 2, None, None, 0, 0, 0, 1]
    for i, e in enumerate(expert):
        assert written[i] == (e is not None)
        for n in range(8):
            want = 0 if e is None else sum(int(a) * int(b) for a, b in zip(x[i], w[e, n])) * xs[i] * ws[e, n]
            assert abs(y[i, n] - want) <= 1e-12 * abs(want)
    h, p, _ = O.grouped_matmul(x, xs * 1e-4, w, ws, groups, "swiglu")
    g, u = p[0, 1], p[0, 5]
    assert abs(h[0, 1] - g / (1 + np.exp(-g)) * u) <= 1e-12 * abs(h[0, 1])

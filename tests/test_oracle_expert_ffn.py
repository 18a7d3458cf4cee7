"""Pins of the 64-bit oracle of the expert operators."""

import numpy as np
import torch

from oracle import expert_ffn as O


def test_e4m3_codes_match_torch():
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3_values(bits), want)
    fine = bits[(bits & 0x7F) != 0x7F]
    np.testing.assert_array_equal(O.e4m3_bits(O.e4m3_values(fine)), fine)


def test_e4m3_rounding_matches_torch_around_every_midpoint():
    v = np.sort(np.abs(O.e4m3_values(np.arange(0x7F, dtype=np.uint8)))).astype(np.float32)
    mid = (v[1:] + v[:-1]) / 2
    cand = np.concatenate([v, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)),
                           np.random.default_rng(1).uniform(0, 448, 10000).astype(np.float32)])
    cand = np.concatenate([cand, -cand])
    want = torch.from_numpy(cand).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(O.e4m3_bits(cand), want)


def test_quantised_rows_match_torch_and_hand_worked_values():
    x = np.random.default_rng(2).normal(size=(5, 300)).astype(np.float32)
    x[2] *= 1e-30
    x[3, :128] = 0
    codes, scales = O.quantise_rows(x)
    t = torch.nn.functional.pad(torch.from_numpy(x), (0, 84)).view(5, 3, 128)
    s = (t.abs().amax(2) / torch.full((5, 3), 448.0)).clamp_min(2.0 ** -126)
    q = (t / s[:, :, None]).to(torch.float8_e4m3fn).view(5, 384)[:, :300].contiguous()
    np.testing.assert_array_equal(scales, s.numpy())
    np.testing.assert_array_equal(codes, q.view(torch.uint8).numpy())
    # 448 and its half: scale 1, codes of 448 and 224
    codes, scales = O.quantise_rows(np.array([[448.0, 224.0, -1.0]], np.float32))
    assert scales[0, 0] == 1.0 and codes.tolist() == [[0x7E, 0x76, 0xB8]]
    # an infinity: NaN for itself, 0 for the rest; a NaN: all NaN
    codes, scales = O.quantise_rows(np.array([[np.inf, 1.0], [np.nan, 1.0]], np.float32))
    assert np.isinf(scales[0, 0]) and codes[0].tolist() == [0x7F, 0] and np.isnan(scales[1, 0])
    assert codes[1].tolist() == [0x7F, 0x7F]


def test_grouped_matmul_is_the_dequantised_product_of_each_group():
    rng = np.random.default_rng(3)
    x, xs = rng.normal(size=(9, 144)), rng.uniform(0.5, 2, (9, 2))
    w, ws = rng.normal(size=(4, 160, 144)), rng.uniform(0.5, 2, (4, 2, 2))
    y, spread, written = O.grouped_matmul(x, xs, w, ws, [(2, 3), (7, 2), (0, -1), (1, 100)])
    dx, dw = x.copy(), w.copy()
    dx[:, :128] *= xs[:, :1]
    dx[:, 128:] *= xs[:, 1:]
    for e in range(4):
        for i, (r0, r1) in enumerate(((0, 128), (128, 160))):
            for j, (c0, c1) in enumerate(((0, 128), (128, 144))):
                dw[e, r0:r1, c0:c1] *= ws[e, i, j]
    np.testing.assert_allclose(y[:3], dx[:3] @ dw[2].T, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(y[5:], dx[5:] @ dw[1].T, rtol=1e-12, atol=1e-12)
    assert written.tolist() == [True] * 3 + [False] * 2 + [True] * 4
    assert (spread[written] >= np.abs(y[written]) - 1e-12).all()


def test_layer_is_the_weighted_sum_of_the_experts():
    rng = np.random.default_rng(4)
    x, ids = rng.normal(size=(3, 32)), np.array([[0, 1], [1, 1], [-1, 9]])
    w13, w2 = rng.normal(size=(2, 32, 32)), rng.normal(size=(2, 32, 16))
    c, mask = rng.uniform(size=(3, 2)), np.array([[1, 0], [1, 1], [1, 1]], bool)
    y, bound = O.layer(x, ids, w13, None, w2, None, c, mask, relative=1e-3, products=1e-3)

    def expert(e, v):
        g, u = w13[e, :16] @ v, w13[e, 16:] @ v
        return w2[e] @ (g / (1 + np.exp(-g)) * u)

    np.testing.assert_allclose(y[0], c[0, 0] * expert(0, x[0]), rtol=1e-12)
    np.testing.assert_allclose(y[1], (c[1, 0] + c[1, 1]) * expert(1, x[1]), rtol=1e-12)
    assert (y[2] == 0).all() and (bound[2] == 0).all() and (bound[:2] > 0).all()

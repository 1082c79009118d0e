"""Pins of the oracle of the norm and the 4-bit weights: hand-worked values,
closed forms and invariants (no GPU)."""
from fractions import Fraction

import numpy as np
import pytest

import oracle


def test_pack_hand_worked_word():
    codes = np.array([[1, -1, 7, -8, 0, 3, 2, -2] + [0] * 120])
    packed = oracle.q4_pack(codes)
    # low half k0 k2 k4 k6 = 1 7 0 2, high half k1 k3 k5 k7 = F 8 3 E
    assert packed.shape == (1, 64)
    assert packed[0, :4].tolist() == [0x71, 0x20, 0x8F, 0xE3]
    assert not packed[0, 4:].any()


def test_pack_round_trip_and_refusal():
    rng = np.random.default_rng(0)
    codes = rng.integers(-8, 8, (5, 256)).astype(np.int8)
    assert np.array_equal(oracle.q4_unpack(oracle.q4_pack(codes)), codes)
    b = rng.integers(0, 256, (3, 64), dtype=np.uint8)
    assert np.array_equal(oracle.q4_pack(oracle.q4_unpack(b)), b)
    for bad in (8, -9):
        with pytest.raises(ValueError):
            oracle.q4_pack(np.full((1, 128), bad))


def test_shifted_word_holds_neighbours():
    """Shifting a word right by 4i leaves weights 2i and 2i + 1 at the bottom
    of its halves."""
    codes = np.arange(-8, 8).reshape(2, 8).repeat(16, axis=1)[:, :128]
    codes[:, :8] = [[3, -3, 5, -5, 7, -7, 1, -1], [0, 1, 2, 3, 4, 5, 6, 7]]
    w = oracle.q4_pack(codes).view("<u4")[:, 0].tolist()
    for r in range(2):
        for i in range(4):
            assert (w[r] >> 4 * i) & 15 == codes[r, 2 * i] % 16
            assert (w[r] >> (16 + 4 * i)) & 15 == codes[r, 2 * i + 1] % 16


def test_quantize_hand_worked_group():
    w = np.zeros((1, 128))
    w[0, :6] = [3.5, -3.5, 0.75, 0.25, 1.25, -0.26]
    codes, scales = oracle.q4_quantize(w, 128)
    assert scales[0, 0] == 0.5                     # 3.5 / 7
    assert codes[0, :6].tolist() == [7, -7, 2, 0, 2, -1]   # 1.5 and 0.5 and 2.5: ties to even
    codes, scales = oracle.q4_quantize(w, 32)
    assert scales[0].astype(float).tolist() == [0.5, 0, 0, 0] and not codes[0, 32:].any()


def test_quantize_is_nearest_in_rationals():
    rng = np.random.default_rng(1)
    w = rng.standard_normal((2, 128)).astype(np.float32).astype(np.float64)
    codes, scales = oracle.q4_quantize(w, 64)
    for i in range(2):
        for j in range(128):
            s = Fraction(float(scales[i, j // 64]))
            best = min(abs(Fraction(w[i, j]) - c * s) for c in range(-8, 8))
            assert abs(Fraction(w[i, j]) - int(codes[i, j]) * s) == best


def test_quantize_edges():
    w = np.zeros((1, 128))
    w[0, 0] = 1e9
    codes, scales = oracle.q4_quantize(w, 128)
    assert scales[0, 0] == 65504 and codes[0, 0] == 7
    w[0, 1] = np.inf
    codes, scales = oracle.q4_quantize(w, 128)
    assert np.isnan(scales[0, 0]) and not codes.any()


def test_i8_hand_worked_group():
    v = np.zeros((1, 256))
    v[0, :4] = [254, -254, 3, 1]
    v[0, 128] = np.nan
    codes, scales = oracle.i8_quantize(v)
    assert scales[0, 0] == 2 and np.isnan(scales[0, 1])
    assert codes[0, :4].tolist() == [127, -127, 2, 0]      # 1.5 -> 2, 0.5 -> 0
    assert not codes[0, 4:].any()


def test_rms_norm_closed_forms():
    k = 2048
    h = np.zeros((2, k))
    h[0, 5] = 3.0
    h[1] = -2.0
    g = np.linspace(0.5, 1.5, k)
    y = oracle.rms_norm(h, g, 1e-30)
    assert np.allclose(y[0, 5], np.sqrt(k) * g[5]) and np.count_nonzero(y[0]) == 1
    assert np.allclose(y[1], -g)
    s = np.where(np.arange(k) % 3 == 0, -1, 1).astype(np.int8)
    r = oracle.rms_norm(h, g, 1e-30, s)
    assert np.allclose((r ** 2).sum(1), (y ** 2).sum(1))   # orthogonal
    assert np.allclose(np.abs(r[0, :1024]), np.sqrt(k) * g[5] / 32) and not r[0, 1024:].any()


def test_rms_sum_rounds_once_to_the_type():
    a, b = np.array([[2048.0, 1.0]]), np.array([[1.0, 2.0 ** -9]])
    assert oracle.rms_sum(a, b, "f16").tolist() == [[2048.0, 1 + 2.0 ** -9]]
    assert oracle.rms_sum(a, b, "bf16").tolist() == [[2048.0, 1.0]]
    assert oracle.rms_sum(a, b, "f32").tolist() == [[2049.0, 1 + 2.0 ** -9]]
    assert oracle.rms_sum(a, None, "f16").tolist() == a.tolist()


def test_product_is_linear_in_scales_and_tokens():
    rng = np.random.default_rng(2)
    codes = rng.integers(-8, 8, (6, 128))
    s = rng.random((6, 4)).astype(np.float16)
    x = rng.standard_normal((3, 128))
    y = oracle.q4_product(x, codes, s)
    assert np.allclose(y[1, 2], sum(x[1, j] * codes[2, j] * float(s[2, j // 32]) for j in range(128)))
    assert np.allclose(oracle.q4_product(2 * x, codes, s), 2 * y)

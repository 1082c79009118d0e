"""Pins of the oracle's 8-bit floating point rows, lookup and logits: values
worked by hand, torch's own e4m3 type, and planted mistakes that must show."""
import numpy as np
import pytest
import torch

import oracle


def test_e4m3_values_by_hand():
    got = oracle.e4m3_values([0x00, 0x01, 0x07, 0x08, 0x38, 0x3C, 0x40, 0x7E, 0x80, 0xB8, 0xFE])
    assert got.tolist() == [0.0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 1.5, 2.0, 448.0, -0.0, -1.0, -448.0]
    assert np.isnan(oracle.e4m3_values([0x7F, 0xFF])).all()


def test_e4m3_against_torch():
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_values(every.numpy()), want, equal_nan=True)
    # all midpoints, their neighbours, and random numbers
    n = want[:127]
    mid = (n[1:] + n[:-1]) / 2
    v = np.concatenate([mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e3)),
                        np.random.default_rng(0).uniform(0, 448, 5000)]).astype(np.float32)
    v = np.concatenate([v, -v])
    codes = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_codes(v), codes)


def test_quantize_by_hand():
    x = np.zeros((1, 640))
    x[0, :3] = [448.0, 224.0, -1.0]             # scale 1
    x[0, 128:130] = [449.0, 1.0]                # scale 2
    x[0, 256:259] = [np.inf, 3.5, np.nan]       # scale 2^-7 by the finite one: 3.5 * 128 = 448
    x[0, 384] = 3.4e38                          # 1.998 * 2^127 / 448 lies above 2^119
    codes, scales = oracle.f8_quantize(x)
    assert scales.tolist() == [[127, 128, 120, 247, 0]]
    assert codes[0, :3].tolist() == [0x7E, 0x76, 0xB8] and codes[0, 128] == 0x76
    assert codes[0, 256:259].tolist() == [0x7F, 0x7E, 0x7F] and not codes[0, 512:].any()
    v = oracle.f8_values(codes, scales)
    assert v[0, 128] == 448.0 and v[0, 129] == 1.0 and np.isnan(v[0, 256])


def test_values_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((20, 256)) * 10.0 ** np.random.default_rng(2).integers(-30, 30, (20, 1))
    codes, scales = oracle.f8_quantize(x)
    v = oracle.f8_values(codes, scales)
    smallest = np.repeat(2.0 ** (scales.astype(float) - 127), 128, axis=1) * 2.0 ** -10
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) / 16, smallest))


def test_product_and_lookup():
    rng = np.random.default_rng(3)
    x, w = oracle.f8_quantize(rng.standard_normal((3, 256))), oracle.f8_quantize(rng.standard_normal((5, 256)))
    got = oracle.f8_product(x, w)
    a, b = oracle.f8_values(*x), oracle.f8_values(*w)
    assert np.allclose(got, [[sum(p * q for p, q in zip(r, s)) for s in b] for r in a], rtol=1e-12)
    rows = oracle.lookup(b, [4, -1, 5, 0, 4], 3.0)
    assert np.array_equal(rows[0], 3 * b[4]) and not rows[1].any() and not rows[2].any()
    assert np.array_equal(rows[3], 3 * b[0]) and np.array_equal(rows[4], rows[0])


def logits_case():
    logits = np.array([[2.0, -2.0, 1.0, 4.0, 0.5]])
    history = np.array([[0, 1, 3, 3, 9, -1, 3]])
    return dict(logits=logits, history=history, history_lens=[6], prompt_lens=[2], repetition=[2.0],
                presence=[0.25], frequency=[0.5], bias_ids=np.array([[2, 0, 2, 7]]),
                bias_values=np.array([[9.0, 1.0, -3.0, 5.0]]), mask=np.array([[0b01111]]))


def test_logits_by_hand():
    got = oracle.adjust_logits(**logits_case())
    # 0: prompt, 2 / 2 + 1; 1: prompt, -2 * 2; 2: the last bias; 3: 4 / 2 - 2 * 0.5 - 0.25; 4: masked
    assert got.tolist() == [[2.0, -4.0, -2.0, 0.75, -np.inf]]


@pytest.mark.parametrize("change", [dict(history_lens=None), dict(prompt_lens=None), dict(repetition=[1.0]),
                                    dict(presence=[0.0]), dict(frequency=None), dict(mask=None),
                                    dict(bias_values=np.array([[-3.0, 1.0, 9.0, 5.0]]))])
def test_each_part_of_the_logits_shows(change):
    case = logits_case()
    assert not np.array_equal(oracle.adjust_logits(**{**case, **change}), oracle.adjust_logits(**case))

"""Plain fp64 definitions of 8-bit floating point rows with block scales, their
product, embedding lookup, and the adjustment of logits.

TEST INFRASTRUCTURE ONLY, as ternary_ref: it shares no code, table or constant
with the HIP library; NumPy is all it uses.  Codes and scales are uint8 arrays.
Pinned in tests/test_oracle_f8.py.
"""
from __future__ import annotations

import numpy as np


def e4m3_values(codes):
    """fp64 values of e4m3 codes: sign, 4 exponent bits with bias 7, 3 mantissa bits."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    return sign * np.where((c & 0x7F) == 0x7F, np.nan, v)


_NUMBERS = e4m3_values(np.arange(127))       # 0 .. 448, rising


def e4m3_codes(v):
    """Codes nearest to |v| <= 448, ties to the even code; NaN for what is not finite."""
    v = np.asarray(v, np.float64)
    a = np.abs(np.where(np.isfinite(v), v, 0.0))
    hi = np.clip(np.searchsorted(_NUMBERS, a), 1, 126)
    below, above = a - _NUMBERS[hi - 1], _NUMBERS[hi] - a
    c = np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)
    c = np.where(np.signbit(v), c + 128, c)
    return np.where(np.isfinite(v), c, 0x7F).astype(np.uint8)


def f8_quantize(x):
    """Codes and biased scale exponents of fp64 rows."""
    x = np.asarray(x, np.float64)
    m, k = x.shape
    codes, scales = np.zeros((m, k), np.uint8), np.zeros((m, k // 128), np.uint8)
    for i in range(m):
        for g in range(k // 128):
            part = x[i, 128 * g:128 * g + 128]
            a = np.abs(part[np.isfinite(part)]).max(initial=0.0)
            e = -127
            while a > 448 * 2.0 ** e:
                e += 1
            scales[i, g] = e + 127
            codes[i, 128 * g:128 * g + 128] = e4m3_codes(part / 2.0 ** e)
    return codes, scales


def f8_values(codes, scales):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return e4m3_values(codes) * np.repeat(s, 128, axis=1)


def f8_product(x, w):
    """x, w: (codes, scales)."""
    return f8_values(*x) @ f8_values(*w).T


def lookup(values, ids, factor):
    out = np.zeros((len(ids), values.shape[1]))
    for i, t in enumerate(ids):
        if 0 <= t < len(values):
            out[i] = values[t] * factor
    return out


def adjust_logits(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
                  frequency=None, bias_ids=None, bias_values=None, mask=None):
    x = np.array(logits, np.float64)
    m, v = x.shape
    for i in range(m):
        if history is not None:
            h = history.shape[1]
            n = h if history_lens is None else min(max(int(history_lens[i]), 0), h)
            prompt = 0 if prompt_lens is None else int(prompt_lens[i])
            seen, count = set(), {}
            for j in range(n):
                t = int(history[i, j])
                if 0 <= t < v:
                    seen.add(t)
                    if j >= prompt:
                        count[t] = count.get(t, 0) + 1
            for t in seen:
                if repetition is not None:
                    x[i, t] = x[i, t] / float(repetition[i]) if x[i, t] > 0 else x[i, t] * float(repetition[i])
            for t, c in count.items():
                x[i, t] -= c * (0.0 if frequency is None else float(frequency[i]))
                x[i, t] -= 0.0 if presence is None else float(presence[i])
        if bias_ids is not None:
            last = {}
            for j in range(bias_ids.shape[1]):
                if 0 <= bias_ids[i, j] < v:
                    last[int(bias_ids[i, j])] = float(bias_values[i, j])
            for t, b in last.items():
                x[i, t] += b
        if mask is not None:
            for t in range(v):
                if not (int(mask[i, t // 32]) >> (t % 32)) & 1:
                    x[i, t] = -np.inf
    return x

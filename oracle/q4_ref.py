"""Plain fp64 definitions of the RMS norm in front of the linears, its 8-bit
outputs, and 4-bit weights with group scales.

TEST INFRASTRUCTURE ONLY, as ternary_ref: it shares no code, table or constant
with the HIP library; NumPy and the rotation of ternary_ref are all it uses.
Types are named "f32", "f16" and "bf16"; bfloat16 arrays are float32 arrays of
bfloat16 values.  Pinned in tests/test_oracle_q4.py.
"""
from __future__ import annotations

import numpy as np

from .ternary_ref import rotate, round_bf16


def _round_to(v, kind):
    if kind == "bf16":
        return round_bf16(np.asarray(v, np.float32)).astype(np.float64)
    return np.asarray(v).astype({"f32": np.float32, "f16": np.float16}[kind]).astype(np.float64)


def rms_sum(x, residual, kind):
    """x + residual, rounded to the type (fp64 values of it)."""
    h = np.asarray(x, np.float64)
    if residual is None:
        return h
    # the sum is taken in fp32, as the definition's type allows no less
    return _round_to((h + np.asarray(residual, np.float64)).astype(np.float32), kind)


def rms_norm(h, gain, eps, signs=None):
    h = np.asarray(h, np.float64)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    return y if signs is None else rotate(y, signs)


def i8_quantize(v):
    """Codes and fp64 scales of rows v, a group being 128 consecutive values."""
    m, k = v.shape
    codes = np.zeros((m, k), np.int8)
    scales = np.zeros((m, k // 128))
    for i in range(m):
        for g in range(k // 128):
            part = v[i, 128 * g:128 * g + 128]
            if not np.all(np.isfinite(part)):
                scales[i, g] = np.nan
                continue
            a = np.abs(part).max()
            scales[i, g] = a / 127
            if a > 0:
                codes[i, 128 * g:128 * g + 128] = np.rint(127 * part / a)
    return codes, scales


def i8_values(codes, scales):
    return codes.astype(np.float64) * np.repeat(np.asarray(scales, np.float64), 128, axis=1)


def q4_pack(codes):
    """Codes in -8 .. 7 to bytes: of the 8 weights k0 .. k7 of a little-endian
    32-bit word, k(2i) at bits 4i, k(2i + 1) at bits 16 + 4i."""
    codes = np.asarray(codes)
    if codes.min() < -8 or codes.max() > 7:
        raise ValueError("4-bit codes lie in -8 .. 7")
    n, k = codes.shape
    words = np.zeros((n, k // 8), np.uint64)
    for j in range(8):
        at = 4 * (j // 2) + 16 * (j % 2)
        words |= (codes[:, j::8].astype(np.int64) % 16).astype(np.uint64) << np.uint64(at)
    return words.astype("<u4").view(np.uint8).reshape(n, k // 2)


def q4_unpack(packed):
    packed = np.ascontiguousarray(packed)
    n = packed.shape[0]
    words = packed.view("<u4").astype(np.int64)
    codes = np.zeros((n, 8 * words.shape[1]), np.int8)
    for j in range(8):
        d = words // 2 ** (4 * (j // 2) + 16 * (j % 2)) % 16
        codes[:, j::8] = np.where(d > 7, d - 16, d)
    return codes


def q4_quantize(w, group):
    """Codes and binary16 scales of fp64 weight rows."""
    n, k = w.shape
    codes = np.zeros((n, k), np.int8)
    scales = np.zeros((n, k // group), np.float16)
    for i in range(n):
        for g in range(k // group):
            part = w[i, group * g:group * g + group]
            if not np.all(np.isfinite(part)):
                scales[i, g] = np.nan
                continue
            s = np.float16(min(np.abs(part).max() / 7, 65504.0))
            scales[i, g] = s
            if s > 0:
                codes[i, group * g:group * g + group] = np.clip(np.rint(part / float(s)), -8, 7)
    return codes, scales


def q4_values(codes, scales):
    group = codes.shape[1] // scales.shape[1]
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), group, axis=1)


def q4_product(x, codes, scales):
    return np.asarray(x, np.float64) @ q4_values(codes, scales).T

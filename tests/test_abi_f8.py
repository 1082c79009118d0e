"""Host-side refusals of the 8-bit floating point calls, the embedding rows and
the logits (no GPU needed): every call here fails validation on made-up
addresses, so nothing touches a device."""
import math

import pytest
import torch

import tl_hadamard_rotate_amd as tl

A = 0x7F0000000000
STEP = 1 << 33              # far-apart buffers
NULL = 0
B = [A + i * STEP for i in range(14)]


def _quant(x=B[0], m=4, k=1024, xd=1, codes=B[1], scales=B[2]):
    return tl.lib().tl_f8_quantize(x, m, k, xd, codes, scales, NULL)


def _dequant(x=B[0], m=4, k=1024, xd=1, codes=B[1], scales=B[2]):
    return tl.lib().tl_f8_dequantize(codes, scales, m, k, x, xd, NULL)


@pytest.mark.parametrize("call", [_quant, _dequant])
def test_f8_weight_refusals(call):
    for name in ("x", "codes", "scales"):
        assert call(**{name: NULL}) == 1
    assert call(x=B[7] + 8) == 4 and call(codes=B[7] + 8) == 4
    for k in (0, 64, 192, (1 << 20) + 128, -128):
        assert call(k=k) == 2
    assert call(m=0) == 2 and call(m=(1 << 24) + 1) == 2 and call(m=1 << 24, k=8192) == 2
    assert call(xd=3) == 7 and call(xd=4) == 7 and call(xd=-1) == 7
    assert call(codes=B[0] + 16) == 5 and call(scales=B[0] + 4 * 2048 - 16) == 5


def test_f8_quantize_overlap_of_its_outputs():
    assert _quant(scales=B[1] + 4096 - 16) == 5 and _quant(codes=B[2]) == 5


def _gemm(codes=B[0], scales=B[1], x=B[2], xs=B[3], m=4, n=64, k=1024, y=B[4], yd=0, ws=NULL, wb=0):
    return tl.lib().tl_f8_gemm(codes, scales, x, xs, m, n, k, y, yd, ws, wb, NULL)


def test_f8_gemm_refusals():
    for name in ("codes", "scales", "x", "xs", "y"):
        assert _gemm(**{name: NULL}) == 1
    for name in ("codes", "x", "y"):
        assert _gemm(**{name: B[7] + 8}) == 4
    assert _gemm(m=0) == 2 and _gemm(n=0) == 2 and _gemm(k=64) == 2 and _gemm(k=200) == 2
    assert _gemm(m=1 << 24, k=8192) == 2 and _gemm(n=1 << 24, k=8192) == 2 and _gemm(m=1 << 20, n=1 << 20, k=128) == 2
    assert _gemm(yd=3) == 7 and _gemm(yd=4) == 7
    for base in (B[0], B[1], B[2], B[3]):
        assert _gemm(y=base) == 5
    assert _gemm(y=B[0] + 64 * 1024 - 16) == 5


def test_f8_gemm_workspace():
    L = tl.lib()
    for bad in ((0, 64, 1024), (4, 0, 1024), (4, 64, 100), (4, 64, 0), (1 << 24, 64, 8192)):
        assert L.tl_f8_gemm_workspace_bytes(*bad) == -1
    with pytest.raises(tl.TLError):
        tl.f8_gemm_workspace_bytes(4, 64, 100)
    for m in (1, 8, 17, 64, 200, 300, 1000, 4096):
        for n, k in ((1024, 5120), (5120, 17408), (17, 17408), (32003, 5120), (256, 131072)):
            need = L.tl_f8_gemm_workspace_bytes(m, n, k)
            assert 0 <= need <= 1 << 28
            if need:
                assert _gemm(m=m, n=n, k=k) == 8
                assert _gemm(m=m, n=n, k=k, ws=B[6], wb=need - 1) == 8
                assert _gemm(m=m, n=n, k=k, ws=B[6] + 8, wb=need) == 4
                for base in B[:5]:
                    assert _gemm(m=m, n=n, k=k, ws=base, wb=need) == 5


def _q4(codes=B[0], scales=B[1], group=128, ids=B[2], m=4, n=64, k=1024, factor=1.0, out=B[3], od=0):
    return tl.lib().tl_q4_rows(codes, scales, group, ids, m, n, k, factor, out, od, NULL)


def _f8(codes=B[0], scales=B[1], ids=B[2], m=4, n=64, k=1024, factor=1.0, out=B[3], od=0):
    return tl.lib().tl_f8_rows(codes, scales, ids, m, n, k, factor, out, od, NULL)


@pytest.mark.parametrize("call", [_q4, _f8])
def test_rows_refusals(call):
    for name in ("codes", "scales", "ids", "out"):
        assert call(**{name: NULL}) == 1
        if (call, name) != (_f8, "scales"):
            assert call(**{name: B[7] + (2 if name == "ids" else 8)}) == 4
    assert call(m=0) == 2 and call(n=0) == 2 and call(k=64) == 2 and call(k=192) == 2
    assert call(m=1 << 24, k=8192) == 2 and call(n=1 << 24, k=8192) == 2
    assert call(od=3) == 7 and call(od=5) == 7
    for factor in (math.nan, math.inf, -math.inf):
        assert call(factor=factor) == 10
    for base in (B[0], B[1], B[2]):
        assert call(out=base) == 5


def test_q4_rows_group():
    assert _q4(group=16) == 3 and _q4(group=0) == 3


def _adjust(logits=B[0], m=4, v=1000, dt=0, history=B[1], h=10, hl=B[2], pl=B[3], r=B[4], p=B[5], f=B[6],
            ids=B[7], values=B[8], b=5, mask=B[9], out=B[10], od=0):
    return tl.lib().tl_adjust_logits(logits, m, v, dt, history, h, hl, pl, r, p, f, ids, values, b, mask, out, od, NULL)


def test_logits_refusals():
    assert _adjust(logits=NULL) == 1 and _adjust(out=NULL) == 1
    assert _adjust(ids=NULL) == 1 and _adjust(values=NULL) == 1
    off = dict(hl=NULL, pl=NULL, r=NULL, p=NULL, f=NULL)
    for name in off:                                        # each needs a history
        assert _adjust(history=NULL, h=0, **{**off, name: B[11]}) == 1
    assert _adjust(history=NULL, **off) == 2 and _adjust(ids=NULL, values=NULL) == 2    # sizes of nothing
    assert _adjust(m=0) == 2 and _adjust(v=0) == 2 and _adjust(h=-1) == 2 and _adjust(b=-1) == 2
    assert _adjust(v=(1 << 24) + 1) == 2 and _adjust(m=1 << 20, v=1 << 20) == 2
    assert _adjust(h=(1 << 24) + 1) == 2 and _adjust(m=1 << 20, h=1 << 20) == 2 and _adjust(m=1 << 20, b=1 << 20) == 2
    assert _adjust(dt=3) == 7 and _adjust(od=3) == 7 and _adjust(od=-1) == 7
    assert _adjust(logits=B[11] + 8) == 4 and _adjust(out=B[11] + 8) == 4
    for name in ("history", "hl", "pl", "r", "p", "f", "ids", "values", "mask"):
        assert _adjust(**{name: B[11] + 2}) == 4


def test_logits_overlaps():
    assert _adjust(out=B[0] + 16) == 5 and _adjust(out=B[0], od=1) == 5     # in place: the same type only
    for base in B[1:10]:
        assert _adjust(out=base) == 5
    assert _adjust(out=B[9] + 4 * 32 * 4 - 16) == 5                         # the mask's last words


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 1024, dtype=torch.float16)
    codes = torch.zeros(4, 1024, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros(4, 8, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    ids = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: tl.f8_quantize(x), lambda: tl.f8_dequantize(codes, scales),
                 lambda: tl.f8_gemm(codes, scales, codes, scales), lambda: tl.f8_rows(codes, scales, ids),
                 lambda: tl.q4_rows(codes.view(torch.uint8), x, ids), lambda: tl.adjust_logits(x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tl.f8_quantize(x.double()), lambda: tl.f8_quantize([1.0]),
                 lambda: tl.f8_dequantize(codes.view(torch.uint8), scales), lambda: tl.f8_dequantize(codes, [1.0]),
                 lambda: tl.f8_gemm(codes, scales.view(torch.uint8), codes, scales),
                 lambda: tl.adjust_logits(x.int()), lambda: tl.adjust_logits(None)):
        with pytest.raises(TypeError):
            call()

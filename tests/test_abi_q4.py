"""Host-side refusals of the norm and the 4-bit calls (no GPU needed): every
call here fails validation on made-up addresses, so nothing touches a device."""
import math
import subprocess
import sys

import pytest
import torch

import tl_hadamard_rotate_amd as tl

A = 0x7F0000000000
STEP = 1 << 32              # far-apart buffers
NULL = 0
B = [A + i * STEP for i in range(10)]


def _norm(x=B[0], residual=B[1], gain=B[2], signs=NULL, m=4, k=1024, xd=1, eps=1e-6, sum_out=B[4],
          out=B[5], od=1, scales=NULL):
    return tl.lib().tl_rms_norm(x, residual, gain, signs, m, k, xd, eps, sum_out, out, od, scales, NULL)


def test_norm_refusals():
    assert _norm(x=NULL) == 1 and _norm(gain=NULL) == 1 and _norm(out=NULL) == 1
    assert _norm(residual=NULL) == 1                        # sum_out without a residual
    assert _norm(od=3) == 1                                 # 8 bits without scales
    assert _norm(xd=3) == 7 and _norm(xd=4) == 7 and _norm(od=4) == 7 and _norm(od=-1) == 7
    assert _norm(scales=B[6]) == 7                          # scales without 8 bits
    assert _norm(m=0) == 2 and _norm(m=(1 << 24) + 1) == 2 and _norm(m=1 << 24, k=8192) == 2
    assert _norm(k=0) == 2 and _norm(k=12) == 2 and _norm(k=(1 << 20) + 8) == 2
    assert _norm(k=1032, signs=B[3]) == 2                   # rotation: whole blocks
    assert _norm(k=1032, od=3, scales=B[6]) == 2            # 8 bits: whole groups
    for eps in (0.0, -1e-6, math.nan, math.inf, 1e-45):
        assert _norm(eps=eps) == 10
    for name in ("x", "residual", "gain", "sum_out", "out"):
        assert _norm(**{name: B[7] + 8}) == 4
    assert _norm(signs=B[3] + 1) == 4 and _norm(od=3, scales=B[6] + 2) == 4


def test_norm_overlaps():
    nbytes = 4 * 1024 * 2
    for base in (B[0], B[1], B[2], B[4]):                   # out over an input or the sum
        assert _norm(out=base) == 5
        assert _norm(out=base - nbytes + 16) == 5
    assert _norm(signs=B[3], out=B[3] + 1008) == 5
    for base in (B[0], B[1]):                               # the sum in place: exactly or not at all
        assert _norm(sum_out=base + 16) == 5 and _norm(sum_out=base - 16) == 5
        assert _norm(sum_out=base, eps=0.0) == 10           # (an exact match passes to ...)
        assert _norm(sum_out=base, out=base) == 5
    assert _norm(sum_out=B[0], residual=B[0] + 16) == 5     # in place over x, across the residual
    assert _norm(sum_out=B[2]) == 5                         # over the gain
    for base in (B[0], B[1], B[2], B[4], B[5]):
        assert _norm(od=3, scales=base) == 5


def test_norm_of_one_row_refuses_the_sum_over_its_gain():
    """With one row the gain is as long as x: the same buffer as x, residual
    and gain may be read by all three, but not written as the sum in place."""
    for k in (1024, 32768):                                 # one pass, two passes
        assert _norm(m=1, k=k, gain=B[0], sum_out=B[0]) == 5
        assert _norm(m=1, k=k, gain=B[1], sum_out=B[1]) == 5
        assert _norm(m=1, k=k, x=B[0], residual=B[0], gain=B[0], sum_out=B[0]) == 5


def _quant(w=B[0], signs=NULL, n=4, k=1024, wd=0, group=128, packed=B[2], scales=B[3]):
    return tl.lib().tl_q4_quantize(w, signs, n, k, wd, group, packed, scales, NULL)


def _dequant(packed=B[0], scales=B[1], n=4, k=1024, group=128, w=B[2], wd=0):
    return tl.lib().tl_q4_dequantize(packed, scales, n, k, group, w, wd, NULL)


@pytest.mark.parametrize("call", [_quant, _dequant])
def test_q4_weight_refusals(call):
    assert call(w=NULL) == 1 and call(packed=NULL) == 1 and call(scales=NULL) == 1
    assert call(n=0) == 2 and call(k=64) == 2 and call(k=192) == 2 and call(k=(1 << 20) + 128) == 2
    assert call(n=1 << 24, k=8192) == 2
    for group in (0, 16, 96, 256, -32):
        assert call(group=group) == 3
    assert call(wd=3) == 7 and call(wd=9) == 7
    for name in ("w", "packed", "scales"):
        assert call(**{name: B[7] + 4}) == 4
    assert call(packed=B[5], scales=B[5] + 16, w=B[5]) == 5
    assert call(w=B[5], packed=B[5] + 64) == 5 and call(w=B[5], scales=B[5] + 64) == 5


def test_q4_quantize_overlaps_and_rotation():
    assert _quant(signs=B[1], k=1152) == 2
    assert _quant(signs=B[1] + 2) == 4
    assert _quant(signs=B[1], packed=B[1]) == 5 and _quant(signs=B[1], scales=B[1]) == 5
    assert _quant(packed=B[3] - 16) == 5


def _gemv(packed=B[0], scales=B[1], group=128, x=B[2], xd=1, xs=NULL, m=4, n=64, k=1024, y=B[4], yd=0,
          ws=NULL, wb=0):
    return tl.lib().tl_q4_gemv(packed, scales, group, x, xd, xs, m, n, k, y, yd, ws, wb, NULL)


def test_q4_gemv_refusals():
    for name in ("packed", "scales", "x", "y"):
        assert _gemv(**{name: NULL}) == 1
    assert _gemv(xd=3) == 1                                 # 8 bits without scales
    assert _gemv(m=0) == 2 and _gemv(n=0) == 2 and _gemv(k=64) == 2 and _gemv(k=200) == 2
    assert _gemv(m=1 << 24, k=8192) == 2 and _gemv(n=1 << 24, k=8192) == 2
    assert _gemv(m=1 << 20, n=1 << 20, k=128) == 2          # M * N
    assert _gemv(group=16) == 3 and _gemv(group=256) == 3
    assert _gemv(xd=0) == 7 and _gemv(xd=4) == 7 and _gemv(yd=3) == 7 and _gemv(xs=B[3]) == 7
    for name in ("packed", "scales", "x", "y"):
        assert _gemv(**{name: B[7] + 8}) == 4
    assert _gemv(xd=3, xs=B[3] + 2) == 4
    for base in (B[0], B[1], B[2]):
        assert _gemv(y=base) == 5
    assert _gemv(xd=3, xs=B[3], y=B[3]) == 5
    assert _gemv(y=B[0] + 64 * 512 - 16) == 5               # the last packed bytes


def test_q4_gemv_workspace():
    L = tl.lib()
    for m, k in ((1, 128), (1, 5120), (1, 16384), (3, 5120), (16, 1024), (64, 256), (128, 128)):
        for n in (1, 1024, 131072):
            assert L.tl_q4_gemv_workspace_bytes(m, n, k) == 0
    for bad in ((0, 64, 1024), (4, 0, 1024), (4, 64, 100), (4, 64, 0), (1 << 24, 64, 8192)):
        assert L.tl_q4_gemv_workspace_bytes(*bad) == -1
    for m in (8, 17, 64, 300):
        for n, k in ((1024, 5120), (5120, 17408), (17, 17408)):
            need = L.tl_q4_gemv_workspace_bytes(m, n, k)
            assert need >= 0
            if need:
                assert _gemv(m=m, n=n, k=k) == 8
                assert _gemv(m=m, n=n, k=k, ws=B[6], wb=need - 1) == 8
                assert _gemv(m=m, n=n, k=k, ws=B[6] + 8, wb=need) == 4
                assert _gemv(m=m, n=n, k=k, ws=B[4] - 16, wb=need) == 5
                assert _gemv(m=m, n=n, k=k, ws=B[2], wb=need) == 5
    with pytest.raises(tl.TLError):
        tl.q4_gemv_workspace_bytes(4, 64, 100)


def test_q4_gemv_workspace_does_not_grow_with_the_tokens():
    """256 MiB, or what 64 tokens need where that is more."""
    for m, n, k in ((300, 131072, 5120), (4096, 17408, 5120), (4096, 131072, 5120), (1 << 20, 16384, 5120),
                    (1048561, 16384, 1408), (1 << 24, 1024, 4096), (1 << 12, 1 << 20, 65536), (128, 1 << 24, 4096)):
        few = tl.q4_gemv_workspace_bytes(64, n, k)
        need = tl.q4_gemv_workspace_bytes(m, n, k)
        assert 0 <= need <= max(1 << 28, few)


def test_q4_packed_bytes():
    assert tl.q4_packed_bytes(1, 128) == 64 and tl.q4_packed_bytes(17408, 5120) == 17408 * 2560
    for n, k in ((0, 128), (4, 0), (4, 64), (4, 130)):
        assert tl.q4_packed_bytes(n, k) == -1


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 1024, dtype=torch.float16)
    g = torch.ones(1024, dtype=torch.float16)
    for call in (tl.rms_norm, tl.rms_norm_i8):
        with pytest.raises(ValueError):
            call(x, g, 1e-6)
        with pytest.raises(TypeError):
            call(x.long(), g, 1e-6)
        with pytest.raises(TypeError):
            call([1.0], g, 1e-6)
    with pytest.raises(TypeError):
        tl.rms_norm(x, g, 1e-6, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        tl.q4_quantize(x)
    with pytest.raises(TypeError):
        tl.q4_quantize(x.double())
    packed, scales = torch.zeros(4, 512, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.float16)
    for call in (lambda: tl.q4_dequantize(packed, scales), lambda: tl.q4_gemv(packed, scales, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tl.q4_gemv(packed.int(), scales, x)


def test_package_imports_on_a_torch_without_gpu_support():
    """Such a torch lacks the look-ups of device and stream; the package still
    imports, and its calls refuse host tensors as elsewhere."""
    program = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import tl_hadamard_rotate_amd as tl
try:
    tl.rms_norm(torch.zeros(1, 1024), torch.ones(1024), 1e-6)
except ValueError as e:
    print("refused:", e)
"""
    run = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=100,
                         cwd=tl.__file__.rsplit("/", 2)[0])
    assert run.returncode == 0, run.stderr
    assert run.stdout.startswith("refused:")

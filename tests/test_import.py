"""The package on a torch that lacks what only some of its calls need."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in {missing!r}:
    delattr(torch, name)
import tl_hadamard_rotate_amd as tl

assert tl.packed_bytes(16, 1024, tl.FMT_SLOT2) == 4096
rows = torch.zeros(2, 256)
codes, scales = torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
for call in (lambda: tl.rms_norm(rows, rows[0], 1e-6), lambda: tl.q4_quantize(rows), lambda: tl.adjust_logits(rows),
             lambda: tl.gemv(codes, scales.half(), tl.FMT_SLOT2, rows.half())):
    try:
        call()
    except ValueError as e:             # host tensors: the calls are there, and check
        assert "device" in str(e), e
    else:
        raise AssertionError("a host tensor was taken")
for call in (lambda: tl.f8_quantize(rows), lambda: tl.f8_dequantize(codes, scales),
             lambda: tl.f8_gemm(codes, scales, codes, scales), lambda: tl.f8_rows(codes, scales, codes[0].int()),
             lambda: tl.F8Linear(codes, scales)(rows)):
    try:
        call()
    except RuntimeError as e:
        assert "float8" in str(e), e
    else:
        raise AssertionError("an 8-bit call went on without its types")
print("done")
"""


@pytest.mark.parametrize("missing", [["float8_e8m0fnu"], ["float8_e8m0fnu", "float8_e4m3fn"]])
def test_a_torch_without_8_bit_types(missing):
    res = subprocess.run([sys.executable, "-c", PROGRAM.format(missing=missing)], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and res.stdout.strip() == "done", res.stderr

"""The top of fp32's range in 8-bit floating point: what the header says of it, by the
oracle here and by the library on the GPU."""
import numpy as np
import pytest
import torch

import oracle
import tl_hadamard_rotate_amd as tl

TOP = 1.9375 * 2.0 ** 127               # half way from code 240 to 256 under the scale 2^120; ties to 256
LARGEST = float(np.finfo(np.float32).max)
BELOW = float(np.nextafter(np.float32(TOP), np.float32(0)))


def rows():
    x = np.zeros((6, 128), np.float64)
    x[0, :2] = [LARGEST, 1.0]
    x[1, :3] = [3.4e38, -LARGEST, 2.0 ** 126]
    x[2, :2] = [TOP, -TOP]
    x[3, :2] = [BELOW, -BELOW]
    x[4, :2] = [1.75 * 2.0 ** 127, 2.0 ** 120]
    x[5, :2] = [float("inf"), BELOW]
    return x


def values(x):
    """fp32 values of the rounded rows: 2^128 and more is infinity."""
    with np.errstate(over="ignore"):
        return oracle.f8_values(*oracle.f8_quantize(x)).astype(np.float32)


def test_largest_values_of_the_definition():
    v = values(rows())
    assert v[0, 0] == np.inf and v[1, 0] == np.inf and v[1, 1] == -np.inf and v[1, 2] == 2.0 ** 126
    assert v[2, 0] == np.inf and v[2, 1] == -np.inf
    assert v[3, 0] == 1.875 * 2.0 ** 127 == -v[3, 1]
    assert v[4, 0] == 1.75 * 2.0 ** 127 and np.isnan(v[5, 0]) and v[5, 1] == v[3, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_largest_values_of_the_library(gpu, out):
    x = torch.from_numpy(rows()).float()
    codes, scales = tl.f8_quantize(x.to(gpu))
    want = torch.from_numpy(values(x.double().numpy()))
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(1, 2, 3), b.nan_to_num(1, 2, 3))  # noqa: E731
    assert same(tl.f8_dequantize(codes, scales, out_dtype=out).float().cpu(), want)
    ids = torch.arange(len(x), dtype=torch.int32, device=gpu)
    # infinity before the factor, which takes ordinary numbers anywhere
    factor = 2.0 ** -100
    assert same(tl.f8_rows(codes, scales, ids, factor, out_dtype=out).float().cpu(), want * factor)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_largest_values_in_a_product(gpu, m, out):
    """Below 2^128 a weight counts; 2^128 is infinity."""
    n, k = 4200, 640
    w = torch.zeros(n, k)
    w[::2, 200], w[1::2, 200] = BELOW, LARGEST
    x = torch.zeros(m, k)
    x[:, 200] = 2.0 ** -120
    got = tl.f8_gemm(*tl.f8_quantize(w.to(gpu)), *tl.f8_quantize(x.to(gpu)), out_dtype=out)
    assert bool((got[:, ::2] == 240).all()) and bool((got[:, 1::2] == float("inf")).all())

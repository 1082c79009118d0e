"""Host-side refusals of the 8-bit floating point product with sums of fewer bits (no
GPU needed): the statuses of the ordinary product, on made-up addresses."""
import pytest

import tl_hadamard_rotate_amd as tl

A = 0x7F0000000000
B = [A + i * (1 << 33) for i in range(10)]
GOOD = dict(codes=B[0], scales=B[1], x=B[2], xs=B[3], m=200, n=512, k=17408, y=B[4], yd=1, ws=0, wb=0)


def status(name, **change):
    a = {**GOOD, **change}
    return getattr(tl.lib(), name)(a["codes"], a["scales"], a["x"], a["xs"], a["m"], a["n"], a["k"], a["y"], a["yd"],
                                   a["ws"], a["wb"], 0)


@pytest.mark.parametrize("change,want", [
    (dict(codes=0), 1), (dict(scales=0), 1), (dict(x=0), 1), (dict(xs=0), 1), (dict(y=0), 1),
    (dict(m=0), 2), (dict(n=0), 2), (dict(k=64), 2), (dict(k=200), 2), (dict(m=1 << 24), 2), (dict(n=(1 << 24) + 1), 2),
    (dict(codes=B[7] + 8), 4), (dict(x=B[7] + 8), 4), (dict(y=B[7] + 2), 4),
    (dict(y=B[0]), 5), (dict(y=B[1]), 5), (dict(y=B[2]), 5), (dict(y=B[3]), 5),
    (dict(yd=3), 7), (dict(yd=-1), 7), (dict(), 8), (dict(ws=B[6], wb=1), 8),
    (dict(ws=B[6] + 8, wb=1 << 28), 4), (dict(ws=B[0], wb=1 << 28), 5), (dict(ws=B[4], wb=1 << 28), 5)])
def test_refusals(change, want):
    assert status("tl_f8_gemm_approx", **change) == want == status("tl_f8_gemm", **change)

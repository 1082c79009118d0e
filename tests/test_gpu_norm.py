"""The RMS norm (residual, gain, rotation, 8-bit outputs) against its fp64
definition.

Tolerances, u = 2^-24 (an fp32 rounding): the sum of K squares is taken by at
least 64 lanes in parallel, so no term passes more than K/64 + 16 additions;
its relative error is at most half that on the root, and the division by K,
eps, the root, its reciprocal and the products add 8 roundings:
    norm = ((K/64 + 16) / 2 + 8) u            relative, on every value.
The rotation's ten levels of sums, and the products in front, add at most
12 u * sum |y| / 32 over the block; the row's factor is common to its values, so
its error stays relative to the rotated value.  The output adds half a step of its type
(relative eps / 2, or half the smallest step of binary16)."""
import numpy as np
import pytest
import torch

import oracle
import tl_hadamard_rotate_amd as tl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(m, k, kind, gpu, seed=0, residual=True, rot=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (scale * draw(m, k)).to(TYPES[kind])
    r = (3 * scale * draw(m, k)).to(TYPES[kind]) if residual else None
    gain = (1 + 0.2 * draw(k)).to(TYPES[kind])
    s = (2 * torch.randint(0, 2, (k,), generator=g) - 1).to(torch.int8) if rot else None
    dev = lambda t: None if t is None else t.to(gpu)  # noqa: E731
    return dev(x), dev(r), dev(gain), dev(s)


def norm_rel(k):
    return ((k / 64 + 16) / 2 + 8) * U


def bounds(want, y, k, out, rot):
    """Elementwise bound of |got - want|; y: the values before the rotation."""
    tol = norm_rel(k) * np.abs(want)
    if rot:
        b = np.abs(y).reshape(y.shape[0], -1, 1024).sum(-1) / 32
        tol = tol + 12 * U * np.repeat(b, 1024, axis=1)
    if out is not None:
        tol = tol + torch.finfo(out).eps / 2 * (np.abs(want) + tol) + \
            (2.0 ** -25 if out == torch.float16 else 2.0 ** -149)
    return tol


def reference(x, r, gain, s, kind, eps=EPS):
    h = oracle.rms_sum(host(x), None if r is None else host(r), kind)
    y = oracle.rms_norm(h, host(gain), eps)
    return h, y, y if s is None else oracle.rotate(y, s.cpu().numpy())


SHAPES = [(1, 8), (3, 24), (1, 136), (5, 1000), (2, 1024), (1, 5120), (7, 5120), (3, 17408),
          (2, 16392), (1, 24576), (1, 24584), (1, 33024), (300, 1032)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("m,k", SHAPES)
def test_norm(gpu, m, k, kind, out):
    for residual in (False, True):
        x, r, gain, _ = make(m, k, kind, gpu, seed=m + k, residual=residual)
        got = tl.rms_norm(x, gain, EPS, residual=r, out_dtype=TYPES[out])
        h, y, want = reference(x, r, gain, None, kind)
        if residual:
            got, total = got
            assert total.dtype == x.dtype and np.array_equal(host(total), h)
        assert got.dtype == TYPES[out]
        assert np.all(np.abs(host(got) - want) <= bounds(want, y, k, TYPES[out], False))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,k", [(1, 1024), (1, 5120), (6, 5120), (3, 17408), (33, 2048), (1, 36864)])
def test_norm_rotated(gpu, m, k, kind):
    for out in TYPES:
        x, r, gain, s = make(m, k, kind, gpu, seed=m + k, rot=True)
        got, total = tl.rms_norm(x, gain, EPS, residual=r, signs=s, out_dtype=TYPES[out])
        h, y, want = reference(x, r, gain, s, kind)
        assert np.array_equal(host(total), h)
        assert np.all(np.abs(host(got) - want) <= bounds(want, y, k, TYPES[out], True))


def i8_check(q, scales, want, y, k, exact=None):
    """Codes equal the definition's away from the ties that the error bound
    reaches, and lie one apart there at most.  Without the rotation they are
    equal everywhere: h * gain, given as ``exact``, has at most 48 bits, and the
    row's factor cancels in them."""
    rot = exact is None
    codes, sc = oracle.i8_quantize(want)
    if not rot:
        codes = oracle.i8_quantize(exact)[0]
    a = np.repeat(sc * 127, 128, axis=1)
    assert np.all(np.abs(host(scales) - sc) <= (norm_rel(k) + 4 * U) * sc +
                  (bounds(want, y, k, None, rot).reshape(len(want), -1, 128).max(-1) / 127 if rot else 0))
    got = host(q)
    if not rot:
        assert np.array_equal(got, codes)
        return
    tol = bounds(want, y, k, None, True)
    t = 127 * want / a
    slack = 127 * (tol + np.abs(want) / a * np.repeat(
        tol.reshape(len(want), -1, 128).max(-1), 128, axis=1)) / a + 4 * U * 127
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= slack
    assert np.array_equal(got[~near], codes[~near])
    assert np.all(np.abs(got[near] - codes[near]) <= 1)
    assert near.mean() < 0.02


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (1, 5120), (16, 5120), (2, 17408), (65, 1152), (1, 33024)])
def test_norm_i8(gpu, m, k, kind):
    x, r, gain, _ = make(m, k, kind, gpu, seed=m + k)
    q, scales, total = tl.rms_norm_i8(x, gain, EPS, residual=r)
    h, y, want = reference(x, r, gain, None, kind)
    assert np.array_equal(host(total), h)
    i8_check(q, scales, want, y, k, h * host(gain))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,k", [(1, 1024), (5, 5120), (2, 17408)])
def test_norm_i8_rotated(gpu, m, k, kind):
    x, r, gain, s = make(m, k, kind, gpu, seed=m + k, rot=True)
    q, scales, total = tl.rms_norm_i8(x, gain, EPS, residual=r, signs=s)
    h, y, want = reference(x, r, gain, s, kind)
    i8_check(q, scales, want, y, k)


def test_i8_ties_go_to_even(gpu):
    """Values n/2 with the group's largest at 127 (or 127/2, 2^-70 times
    that): every odd n is a tie."""
    for f in (1.0, 0.5, 2.0 ** -70):
        v = torch.arange(-127, 128, dtype=torch.float64) / 2
        row = torch.cat([v[:127], v[-1:] * 2, v[127:254], -v[-1:] * 2]) * f
        x = row.float()[None].to(gpu)
        q, scales = tl.rms_norm_i8(x, torch.ones(256, device=gpu), 1e-30)
        want = np.rint(row.numpy() / f * 1.0)
        want[[127, 255]] = [127, -127]
        assert np.array_equal(host(q)[0], want)


@pytest.mark.parametrize("rot", [False, True])
def test_i8_codes_do_not_depend_on_a_power_of_two(gpu, rot):
    """A gain of 2^-110 leaves every rounding as it was: the same codes, scales
    times 2^-110 (their values then lie below 1e-30)."""
    x, _, _, s = make(3, 2048, "f32", gpu, residual=False, rot=rot)
    one = torch.ones(2048, device=gpu)
    q, sc = tl.rms_norm_i8(x, one, EPS, signs=s)
    tiny, tiny_sc = tl.rms_norm_i8(x, one * 2.0 ** -110, EPS, signs=s)
    assert torch.equal(q, tiny) and torch.equal(sc * 2.0 ** -110, tiny_sc)


def test_zero_rows_and_groups(gpu):
    x, _, gain, s = make(4, 2048, "f16", gpu, residual=False, rot=True)
    x[1] = 0
    x[2, 128:256] = 0
    y = tl.rms_norm(x, gain, EPS, out_dtype=torch.float32)
    assert not host(y)[1].any() and not host(y)[2, 128:256].any()
    q, scales = tl.rms_norm_i8(x, gain, EPS)
    assert not host(q)[1].any() and not host(scales)[1].any() and host(scales)[2, 1] == 0
    q, scales = tl.rms_norm_i8(x, gain, EPS, signs=s)
    assert not host(q)[1].any() and not host(scales)[1].any()


@pytest.mark.parametrize("kind", list(TYPES))
def test_nonfinite_values_stay_in_their_rows(gpu, kind):
    x, r, gain, s = make(5, 2048, kind, gpu, rot=True)
    clean = tl.rms_norm(x, gain, EPS, residual=r, signs=s)[0]
    clean8 = tl.rms_norm_i8(x, gain, EPS, residual=r)
    x[1, 7], x[3, 1500] = float("nan"), float("inf")
    got = tl.rms_norm(x, gain, EPS, residual=r, signs=s)[0]
    keep = [0, 2, 4]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[3, 1024:]).any()
    plain = host(tl.rms_norm(x, gain, EPS, residual=r, out_dtype=torch.float32)[0])
    assert np.isnan(plain[1]).all() and np.isnan(plain[3, 1500])
    assert not np.delete(plain[3], 1500).any()                 # 1 / sqrt(inf) = 0
    q, scales, _ = tl.rms_norm_i8(x, gain, EPS, residual=r)
    assert torch.equal(q[keep], clean8[0][keep]) and torch.equal(scales[keep], clean8[1][keep])
    assert torch.isnan(scales[1]).all() and torch.isnan(scales[3, 11]) and not q[3, 1408:1536].any()


@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("k", [2048, 36864])
def test_i8_codes_of_rows_without_finite_norms(gpu, k, rot):
    """A NaN makes its whole row NaN; an infinity, or squares whose sum passes
    fp32, make the rest of the row 0: codes 0 in every group, scales NaN or 0."""
    x, _, gain, s = make(5, k, "f32", gpu, residual=False, rot=rot)
    clean = tl.rms_norm_i8(x, gain, EPS, signs=s)
    x[1, 7], x[2, 1500] = float("nan"), float("inf")
    x[3] *= 1e25
    q, scales = tl.rms_norm_i8(x, gain, EPS, signs=s)
    assert torch.equal(q[[0, 4]], clean[0][[0, 4]]) and torch.equal(scales[[0, 4]], clean[1][[0, 4]])
    assert not q[1:4].any()
    sc = host(scales)
    hit = np.zeros(k // 128, bool)
    hit[8:16 if rot else 8] = True
    hit[11] = True
    assert np.isnan(sc[1]).all() and not sc[3].any()
    assert np.isnan(sc[2, hit]).all() and not sc[2, ~hit].any()


@pytest.mark.parametrize("xf,gf,eps", [(1e15, 1e25, EPS), (1e-17, 1e-25, 2.0 ** -126)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("m,k", [(3, 2048), (2, 17408), (1, 33024)])
def test_products_with_the_gain_past_fp32(gpu, m, k, kind, xf, gf, eps):
    """Outputs that fit although h * gain passes fp32, or lies below its
    normal numbers."""
    x, _, gain, _ = make(m, k, kind, gpu, seed=k, residual=False)
    x, gain = (x.double() * xf).to(x.dtype), (gain.double() * gf).to(x.dtype)
    h, y, want = reference(x, None, gain, None, kind, eps=eps)
    for out in ("f32", "bf16"):
        got = tl.rms_norm(x, gain, eps, out_dtype=TYPES[out])
        assert np.all(np.abs(host(got) - want) <= bounds(want, y, k, TYPES[out], False))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gf", [2.0 ** -49, 2.0 ** 49])
@pytest.mark.parametrize("xf,eps", [(1e16, EPS), (1e-17, 2.0 ** -126)])
def test_gains_within_the_stated_range(gpu, kind, gf, xf, eps):
    """Rotated and 8-bit outputs at the ends of the gains that tl.h states."""
    for rot in (False, True):
        x, _, gain, s = make(3, 2048, kind, gpu, residual=False, rot=rot)
        x, gain = (x.double() * xf).to(x.dtype), (gain.double() * gf).to(x.dtype)
        h, y, want = reference(x, None, gain, s, kind, eps=eps)
        got = tl.rms_norm(x, gain, eps, signs=s, out_dtype=torch.float32)
        assert np.all(np.abs(host(got) - want) <= bounds(want, y, 2048, torch.float32, rot))
        i8_check(*tl.rms_norm_i8(x, gain, eps, signs=s), want, y, 2048, None if rot else h * host(gain))


@pytest.mark.parametrize("k", [5120, 17408, 36864])
@pytest.mark.parametrize("rot", [False, True])
def test_rows_alone_are_the_same_bits(gpu, k, rot):
    """A row's outputs, sum, codes and scales do not depend on the rows beside
    it or on their number."""
    x, r, gain, s = make(9, k, "bf16", gpu, rot=rot)
    many = (*tl.rms_norm(x, gain, EPS, residual=r, signs=s), *tl.rms_norm_i8(x, gain, EPS, residual=r, signs=s))
    for i in (0, 4, 8):
        a, b = x[i:i + 1].clone(), r[i:i + 1].clone()
        one = (*tl.rms_norm(a, gain, EPS, residual=b, signs=s), *tl.rms_norm_i8(a, gain, EPS, residual=b, signs=s))
        for got, want in zip(one, many):
            assert torch.equal(got, want[i:i + 1])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("m,k", [(2, 24576), (2, 25600), (1, 36864)])
def test_norm_i8_rotated_long_rows(gpu, m, k, kind):
    x, r, gain, s = make(m, k, kind, gpu, seed=m + k, rot=True)
    q, scales, total = tl.rms_norm_i8(x, gain, EPS, residual=r, signs=s)
    h, y, want = reference(x, r, gain, s, kind)
    assert np.array_equal(host(total), h)
    i8_check(q, scales, want, y, k)


def test_large_and_tiny_values(gpu):
    """binary16 rows near its largest and smallest numbers, eps of the smallest
    normal number."""
    for scale in (1e4, 1e-6):
        x, _, gain, _ = make(3, 1536, "f16", gpu, residual=False, scale=scale)
        got = tl.rms_norm(x, gain, 2.0 ** -126, out_dtype=torch.float32)
        h, y, want = reference(x, None, gain, None, "f16", eps=2.0 ** -126)
        assert np.all(np.abs(host(got) - want) <= bounds(want, y, 1536, torch.float32, False))


def test_sum_in_place(gpu):
    for target in ("x", "residual"):
        for k, rot in ((5120, True), (33024, False), (36864, True)):
            x, r, gain, s = make(3, k, "f16", gpu, rot=rot)
            want, total = tl.rms_norm(x, gain, EPS, residual=r, signs=s)
            where = x if target == "x" else r
            got, same = tl.rms_norm(x, gain, EPS, residual=r, signs=s, sum_out=where)
            assert same is where and torch.equal(where, total) and torch.equal(got, want)


@pytest.mark.parametrize("kind", list(TYPES))
def test_sum_rounds_to_nearest_even(gpu, kind):
    """The stored sum is the rounded sum, bit for bit: ordinary values, halves
    of the last bit, subnormal and overflowing sums, infinities and NaN."""
    t, m, k = TYPES[kind], 8, 1024
    g = torch.Generator().manual_seed(5)
    bits = {2: torch.int16, 4: torch.int32}[t.itemsize]
    any_bits = lambda: torch.randint(-2 ** 31, 2 ** 31, (m, k), generator=g).to(bits).view(t)  # noqa: E731
    x, r = any_bits(), any_bits()
    x[0], r[0] = 1.0, 0.5 * torch.finfo(t).eps * torch.arange(k).to(t)          # ties of every kind
    x[1], r[1] = x[1].sign() * torch.finfo(t).tiny, r[1].sign() * torch.finfo(t).tiny * 0.5
    x[2, :512], r[2, :512] = torch.finfo(t).max, torch.finfo(t).max
    x[3], r[3] = x[3].float().nan_to_num(1.0).clamp(-8, 8).to(t), r[3].float().nan_to_num(1.0).clamp(-8, 8).to(t)
    got = torch.empty(m, k, dtype=t, device=gpu)
    tl.rms_norm(x.to(gpu), torch.ones(k, dtype=t, device=gpu), EPS, residual=r.to(gpu), sum_out=got)
    want = (x.float() + r.float()).to(t)
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    assert torch.equal(got.view(bits)[ok], want.view(bits)[ok])


def test_residual_may_be_x_itself(gpu):
    x, _, gain, _ = make(2, 5120, "bf16", gpu, residual=False)
    got, total = tl.rms_norm(x, gain, EPS, residual=x)
    want = tl.rms_norm(2 * x, gain, EPS)
    assert torch.equal(total, 2 * x) and torch.equal(got, want)


def test_neighbouring_memory_is_left_alone(gpu):
    m, k = 3, 1152
    x, r, gain, _ = make(m, k, "f16", gpu)
    big = [torch.full((m * k + 512,), 7.0, dtype=torch.float16, device=gpu) for _ in range(2)]
    out, total = (b[256:256 + m * k].view(m, k) for b in big)
    tl.rms_norm(x, gain, EPS, residual=r, out=out, sum_out=total)
    q = torch.full((m * k + 512,), 7, dtype=torch.int8, device=gpu)
    sc = torch.full((m * 9 + 64,), 7.0, device=gpu)
    tl.rms_norm_i8(x, gain, EPS, residual=r, out=q[256:256 + m * k].view(m, k),
                   scales=sc[32:32 + m * 9].view(m, 9))
    for b in (*big, q):
        assert (b[:256] == 7).all() and (b[256 + m * k:] == 7).all()
    assert (sc[:32] == 7).all() and (sc[32 + m * 9:] == 7).all()


def test_refused_call_writes_nothing(gpu):
    x, r, gain, _ = make(2, 1032, "f16", gpu)
    out = torch.full((2, 1032), 7.0, dtype=torch.float16, device=gpu)
    s = torch.ones(1032, dtype=torch.int8, device=gpu)
    with pytest.raises(tl.TLError, match="TL_ERR_SHAPE"):
        tl.rms_norm(x, gain, EPS, signs=s, out=out)
    with pytest.raises(tl.TLError, match="TL_ERR_VALUE"):
        tl.rms_norm(x, gain, 0.0, out=out)
    with pytest.raises(tl.TLError, match="TL_ERR_ALIAS"):
        tl.rms_norm(x, gain, EPS, residual=r, out=r)
    with pytest.raises(ValueError):
        tl.rms_norm(x[:, :1024], gain[:1024], EPS)          # a view with a stride
    with pytest.raises(ValueError):
        tl.rms_norm(x, gain, EPS, sum_out=out)
    with pytest.raises(TypeError):
        tl.rms_norm(x, gain.float(), EPS)
    assert (out == 7).all()


def test_repeats_and_rows_alone_are_the_same_bits(gpu):
    x, r, gain, s = make(9, 5120, "bf16", gpu, rot=True)
    a = tl.rms_norm(x, gain, EPS, residual=r, signs=s)[0]
    assert torch.equal(a, tl.rms_norm(x, gain, EPS, residual=r, signs=s)[0])
    one = tl.rms_norm(x[4:5].clone(), gain, EPS, residual=r[4:5].clone(), signs=s)[0]
    tol = host(torch.maximum(a[4:5].abs(), one.abs())) * 2.0 ** -10 + 2.0 ** -14
    assert np.all(np.abs(host(a[4:5]) - host(one)) <= tol)


def test_other_stream_and_graph_replays(gpu):
    x, r, gain, s = make(8, 5120, "f16", gpu, rot=True)
    want = tl.rms_norm(x, gain, EPS, residual=r, signs=s)
    want8 = tl.rms_norm_i8(x, gain, EPS, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tl.rms_norm(x, gain, EPS, residual=r, signs=s)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, total = torch.zeros_like(x), torch.zeros_like(x)
    q, sc = torch.zeros_like(want8[0]), torch.zeros_like(want8[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.rms_norm(x, gain, EPS, residual=r, signs=s, out=out, sum_out=total)
        tl.rms_norm_i8(x, gain, EPS, residual=r, out=q, scales=sc, sum_out=total)
    for i in range(4):
        x.copy_(torch.randn_like(x) * (i + 1))
        want = tl.rms_norm(x, gain, EPS, residual=r, signs=s)
        want8 = tl.rms_norm_i8(x, gain, EPS, residual=r)
        out.zero_(), total.zero_(), q.zero_(), sc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(total, want[1])
        assert torch.equal(q, want8[0]) and torch.equal(sc, want8[1])


def test_offsets_past_32_bits(gpu):
    """More than 2^32 elements: the first and last rows against the same rows
    alone; the rows between repeat them."""
    k, m = 8192, (1 << 19) + 3
    gain = torch.ones(k, dtype=torch.float16, device=gpu)
    x = torch.ones(m, k, dtype=torch.float16, device=gpu)
    x[0], x[-1] = torch.randn(k, device=gpu), torch.randn(k, device=gpu)
    y = tl.rms_norm(x, gain, EPS)
    ends = tl.rms_norm(x[[0, 1, -1]].contiguous(), gain, EPS)
    assert torch.equal(y[[0, 1, -1]], ends)
    assert bool((y[1:-1] == ends[1, 0]).all())


@pytest.mark.parametrize("k,rot", [(24, False), (128, False), (1024, True)])
def test_more_rows_than_workgroups(gpu, k, rot):
    """Rows past 2^20 are a workgroup's second: every row repeats one of 1021,
    and so do its outputs."""
    m, some = (1 << 20) + 5, 1021
    x, _, gain, s = make(some, k, "f16", gpu, residual=False, rot=rot)
    rows = torch.arange(m, device=gpu) % some
    want = tl.rms_norm(x, gain, EPS, signs=s)
    assert torch.equal(tl.rms_norm(x[rows], gain, EPS, signs=s), want[rows])
    if k % 128 == 0:
        want = tl.rms_norm_i8(x, gain, EPS, signs=s)
        got = tl.rms_norm_i8(x[rows], gain, EPS, signs=s)
        assert torch.equal(got[0], want[0][rows]) and torch.equal(got[1], want[1][rows])


def test_norm_feeds_the_ternary_product(gpu):
    """Norm with the rotation, then tl_gemv on its output, against the norm,
    rotation and product in 64 bits."""
    m, k, n = 4, 5120, 768
    x, r, gain, s = make(m, k, "f16", gpu, seed=3, rot=True)
    rng = np.random.default_rng(3)
    codes = rng.integers(-1, 2, (n, k)).astype(np.int8)
    scales = np.abs(0.02 * rng.standard_normal((n, k // 128))).astype(np.float16)
    packed = tl.pack(torch.from_numpy(codes).to(gpu), tl.FMT_SLOT2)
    x_rot, total = tl.rms_norm(x, gain, EPS, residual=r, signs=s)
    y = tl.gemv(packed, torch.from_numpy(scales).to(gpu), tl.FMT_SLOT2, x_rot)
    _, _, want = reference(x, r, gain, s, "f16")
    assert oracle.rel_l2(host(y), oracle.matvec(codes, scales, want)) < 2e-3

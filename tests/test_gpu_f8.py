"""8-bit floating point rows: rounding, values and the product, against their
fp64 definitions.

Tolerance of the product, u = 2^-24.  float32 outputs, and few tokens: products
are exact in fp32; a term passes through at most 32 additions within its matrix
instruction, one for each later one (K / 32) and at most 24 where parts of K are
joined; an addition that truncates is off by 2 u of its result, so
    |got - want| <= 2 u (K/32 + 56) * sum_k |x w|.
Other outputs of more tokens come from the 8-bit matrix instructions, which align
the products of 8 neighbouring k to the largest exponent among them and drop what
lies 14 bits below: at most 2^-13 of the largest for each of 8,
    + 2^-10 * sum over eights of max |x w|.
The output adds half a step of its type."""
import numpy as np
import pytest
import torch

import oracle
import tl_hadamard_rotate_amd as tl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EXACT_TOKENS = 16           # up to here every output type sums exact products in fp32


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def raw(t):
    return t.detach().view(torch.uint8).cpu().numpy()


def e8(a, gpu):
    return torch.from_numpy(a).to(gpu).view(torch.float8_e8m0fnu)


def e4(a, gpu):
    return torch.from_numpy(a).to(gpu).view(torch.float8_e4m3fn)


# ------------------------------------------------------------ rows

def check_rounding(x, gpu):
    codes, scales = tl.f8_quantize(x.to(gpu))
    want = oracle.f8_quantize(x.double().numpy())
    assert np.array_equal(raw(codes), want[0]) and np.array_equal(raw(scales), want[1])
    return codes, scales, want


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (17, 1152), (2, 5120), (1, 17408)])
def test_quantize_is_exact(gpu, m, k, kind):
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(m, k, generator=g))
    codes, scales, want = check_rounding(x.to(TYPES[kind]), gpu)
    for out in ("f32", "f16", "bf16"):
        back = tl.f8_dequantize(codes, scales, out_dtype=TYPES[out])
        exact = torch.from_numpy(oracle.f8_values(*want).astype(np.float32)).to(TYPES[out])
        assert torch.equal(back.cpu(), exact)


def test_quantize_ties_and_limits(gpu):
    n = oracle.e4m3_values(np.arange(127))
    x = np.zeros((10, 128), np.float32)
    x[0, :126], x[0, 126] = (n[1:] + n[:-1]) / 2, 448           # every tie
    x[1] = -np.nextafter(x[0], np.float32(0))
    x[2] = np.nextafter(x[0], np.float32(1e3))
    x[2, 126] = 448                                             # (just past it the scale doubles)
    x[3, :2] = [np.nextafter(np.float32(448), np.float32(1e3)), 1]
    x[4, :3] = [3.4e38, -3e38, 1e30]
    x[5, :3] = [1e-45, -3e-45, 1e-40]                           # below the smallest scale's values
    x[6, :4] = [2.0 ** -119, 1.9 * 2.0 ** -119, 1.75 * 2.0 ** -119, 2.0 ** -126]
    x[7, :2] = [-0.0, 0.0]
    x[8, :2] = [1.7500001, 1.75]
    check_rounding(torch.from_numpy(x), gpu)


def test_quantize_what_is_not_finite(gpu):
    x = torch.randn(4, 384)
    clean = tl.f8_quantize(x.to(gpu))
    y = x.clone()
    y[1, 130], y[1, 200], y[2, 5], y[3, 256:] = float("inf"), float("nan"), float("-inf"), float("nan")
    codes, scales, _ = check_rounding(y, gpu)
    back = host(tl.f8_dequantize(codes, scales, out_dtype=torch.float32))
    assert np.array_equal(np.isnan(back), ~torch.isfinite(y).numpy())
    assert np.array_equal(raw(scales)[0], raw(clean[1])[0])


def test_every_code_and_scale_decodes(gpu):
    codes = np.tile(np.arange(256, dtype=np.uint8), 128).reshape(1, -1)
    scales = np.arange(256, dtype=np.uint8).reshape(1, 256)
    for out in ("f32", "f16", "bf16"):
        got = tl.f8_dequantize(e4(codes, gpu), e8(scales, gpu), out_dtype=TYPES[out]).cpu()
        with np.errstate(over="ignore"):
            want = oracle.f8_values(codes, scales).astype(np.float32)
        assert torch.equal(torch.nan_to_num(got.float(), nan=1.25),
                           torch.nan_to_num(torch.from_numpy(want).to(TYPES[out]).float(), nan=1.25))


# ------------------------------------------------------------ product

def make(m, n, k, seed=0, outliers=True, spread=1):
    """(x, w) as (codes, scales) of the oracle, scales of neighbouring blocks apart."""
    rng = np.random.default_rng(seed)
    x, w = rng.standard_normal((m, k)), 0.02 * rng.standard_normal((n, k))
    if outliers:
        x[rng.random((m, k)) < 0.01] *= 20
    x *= np.repeat(2.0 ** rng.integers(-spread, spread + 1, (m, k // 128)), 128, axis=1)
    w *= np.repeat(2.0 ** rng.integers(-spread, spread + 1, (n, k // 128)), 128, axis=1)
    return quick(x), quick(w)


def quick(x):
    """The oracle's rounding through torch's type (pinned against each other)."""
    m, k = x.shape
    b = x.reshape(m, -1, 128)
    f, p = np.frexp(np.abs(b).max(-1))
    e = np.where(f <= 0.875, p - 9, p - 8)
    e = np.where(f == 0, -127, e)
    c = torch.from_numpy((b / 2.0 ** e[..., None]).reshape(m, k).astype(np.float32)).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).numpy(), (e + 127).astype(np.uint8)


def call(x, w, dtype, gpu, **kw):
    return tl.f8_gemm(e4(w[0], gpu), e8(w[1], gpu), e4(x[0], gpu), e8(x[1], gpu), out_dtype=dtype, **kw)


def tolerance(x, w, out):
    a, b = np.abs(oracle.f8_values(*x)), np.abs(oracle.f8_values(*w))
    k = a.shape[1]
    tol = 2 * U * (k / 32 + 56) * (a @ b.T)
    if out != torch.float32 and len(a) > EXACT_TOKENS:
        p = torch.zeros(len(a), len(b), dtype=torch.float64)
        ta, tb = torch.from_numpy(a), torch.from_numpy(b)
        for g in range(0, k, 8):
            top = torch.zeros_like(p)
            for j in range(g, g + 8):
                torch.maximum(top, ta[:, j, None] * tb[None, :, j], out=top)
            p += top
        tol = tol + 2.0 ** -10 * p.numpy()
    return tol


def check(x, w, out, gpu, **kw):
    got = host(call(x, w, out, gpu, **kw))
    want = oracle.f8_product(x, w)
    tol = tolerance(x, w, out)
    if out != torch.float32:
        tol = tol + torch.finfo(out).eps / 2 * np.abs(want) + (2.0 ** -25 if out == torch.float16 else 0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 16, 256), (1, 1000, 5120), (2, 33, 384), (3, 17, 1152),
                                   (8, 130, 17408), (15, 64, 9216), (16, 515, 640), (17, 48, 2048),
                                   (31, 100, 1280), (33, 257, 5120), (45, 96, 3328), (64, 80, 4096)])
def test_few_tokens(gpu, m, n, k, out):
    x, w = make(m, n, k, seed=m + n + k, spread=6)
    check(x, w, TYPES[out], gpu)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(65, 17, 128), (66, 300, 256), (128, 128, 384), (129, 257, 640), (200, 1, 896),
                                   (255, 511, 1152), (256, 256, 512), (257, 259, 2176), (300, 1030, 1280),
                                   (513, 70, 5120), (20, 4200, 640), (33, 9000, 384), (64, 5003, 1152),
                                   (100, 2100, 896), (128, 4100, 256), (200, 1500, 5248), (40, 40, 5376),
                                   (66, 8371, 256), (90, 2741, 4480)])
def test_many_tokens(gpu, m, n, k, out):
    x, w = make(m, n, k, seed=m + n + k, spread=4)
    check(x, w, TYPES[out], gpu)


@pytest.mark.parametrize("m,n,k", [(1, 40, 131072), (70, 24, 40960)])
def test_long_rows(gpu, m, n, k):
    x, w = make(m, n, k, seed=7)
    check(x, w, torch.float32, gpu)


@pytest.mark.parametrize("n,k", [(270, 1408), (4130, 1408), (270, 5248)])
@pytest.mark.parametrize("m", [1, 20, 64, 100, 300])
def test_codes_count_and_none_is_missed(gpu, m, n, k):
    """Small whole numbers: every sum is exact, so one product lost, counted
    twice or taken from another place shows."""
    rng = np.random.default_rng(m)
    values = np.array([-2, -1, 0, 1, 2])
    xc, wc = rng.integers(0, 5, (m, k)), rng.integers(0, 5, (n, k))
    code = oracle.e4m3_codes(values.astype(float))
    s = np.full((max(m, n), k // 128), 127, np.uint8)
    got = host(call((code[xc], s[:m]), (code[wc], s[:n]), torch.float32, gpu))
    want = (torch.from_numpy(values[xc]).double() @ torch.from_numpy(values[wc]).double().T).numpy()
    assert np.array_equal(got, want)
    got = host(call((code[xc], s[:m]), (code[wc], s[:n]), torch.float16, gpu))
    assert np.array_equal(got, want)            # |sums| stay below 2048


@pytest.mark.parametrize("m", [1, 20, 100, 300])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1152, 5376])
def test_every_scale_reaches_its_block(gpu, m, out, k):
    """One block of each row counts, under a scale of its own."""
    n = 130
    rng = np.random.default_rng(m)
    xv, wv = np.zeros((m, k)), np.zeros((n, k))
    xs, ws = rng.integers(110, 140, (m, k // 128)).astype(np.uint8), rng.integers(110, 140, (n, k // 128)).astype(np.uint8)
    at = rng.integers(0, k // 128, n)
    xv[:, ::128] = 1.0
    for i in range(n):
        wv[i, 128 * at[i]] = 1.0
    got = host(call((oracle.e4m3_codes(xv), xs), (oracle.e4m3_codes(wv), ws), TYPES[out], gpu))
    want = 2.0 ** (xs[:, at].astype(float) + ws[np.arange(n), at] - 254.0)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("m", [1, 30, 100, 300])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("k", [512, 5248])
def test_nan_and_zero_stay_in_their_rows(gpu, m, out, k):
    n = 150
    x, w = make(m, n, k, seed=m)
    x, w = (x[0].copy(), x[1].copy()), (w[0].copy(), w[1].copy())
    w[0][3, 300] = 0x7F
    w[1][140, 2] = 255                                  # the NaN scale
    x[0][m // 2, 7] = 0xFF
    w[0][9], w[1][9] = 0, 0
    got = host(call(x, w, TYPES[out], gpu))
    nan = np.zeros((m, n), bool)
    nan[:, 3] = nan[:, 140] = nan[m // 2] = True
    assert np.array_equal(np.isnan(got), nan)
    assert not got[~nan[:, 9], 9].any()
    check_rows = [i for i in range(m) if i != m // 2][:4]
    if check_rows:
        cols = [j for j in range(n) if j not in (3, 140)]
        xx, ww = (x[0][check_rows], x[1][check_rows]), (w[0][cols], w[1][cols])
        want = oracle.f8_product(xx, ww)
        tol = 2 * tolerance(xx, ww, torch.float32) + 2.0 ** -10 * np.abs(oracle.f8_values(*xx)) @ np.abs(oracle.f8_values(*ww)).T
        tol += 2.0 ** -11 * np.abs(want) + 2.0 ** -25
        assert np.all(np.abs(got[np.ix_(check_rows, cols)] - want) <= tol)


@pytest.mark.parametrize("m,n,k", [(1, 1000, 5120), (12, 500, 17408), (40, 96, 2048), (100, 300, 1280), (300, 520, 2048),
                                   (40, 96, 6016), (100, 4100, 1280), (300, 520, 6016)])
def test_same_bits_again_and_alone(gpu, m, n, k):
    """From call to call, and whatever the other tokens hold."""
    x, w = make(m, n, k, seed=m)
    for out in (torch.float32, torch.bfloat16):
        got = call(x, w, out, gpu)
        assert torch.equal(got, call(x, w, out, gpu))
        other = (x[0].copy(), x[1].copy())
        other[0][:m - 1] = 0x38
        assert torch.equal(got[m - 1], call(other, w, out, gpu)[m - 1])


@pytest.mark.parametrize("k", [640, 5248])
@pytest.mark.parametrize("m", [1, 33, 90, 260])
def test_nothing_behind_the_rows_is_written(gpu, m, k):
    x, w = make(m, 33, k, seed=m)
    for out in (torch.float32, torch.float16):
        big = torch.full((m + 3, 33), 7.0, dtype=out, device=gpu)
        call(x, w, out, gpu, out=big[:m])
        assert bool((big[m:] == 7).all()) and torch.equal(big[:m], call(x, w, out, gpu))


def test_workspace_contents_do_not_matter(gpu):
    for m, n, k in ((13, 512, 17408), (200, 512, 17408), (300, 520, 5120)):
        x, w = make(m, n, k, seed=m)
        need = tl.f8_gemm_workspace_bytes(m, n, k)
        got = call(x, w, torch.float16, gpu)
        ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=gpu)
        assert torch.equal(got, call(x, w, torch.float16, gpu, workspace=ws))


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(9, 40, 17408), (40, 150, 7040), (130, 130, 9984), (300, 300, 12800),
                                   (600, 5200, 7040), (520, 700, 17408),
                                   # tiles of every shape, whole and cut
                                   (33, 2084, 256), (81, 2741, 4480), (101, 2697, 3712), (65, 8371, 256),
                                   (585, 3219, 256), (18, 5477, 3200), (19, 1241, 5504), (17, 16869, 256),
                                   (33, 5462, 6400), (34, 5585, 4224), (33, 17109, 256), (67, 10982, 6400),
                                   (131, 16163, 256), (130, 8329, 9856), (391, 5554, 5504), (389, 16929, 256),
                                   (1100, 16700, 5248)])
def test_long_sums_of_whole_numbers(gpu, m, n, k, out):
    """Every place of long rows counts, in whole and in cut tiles: codes of -1, 0 and
    1, sparse enough that sums stay exact in every type, under scales whose product
    is 1 and which differ from block to block."""
    rng = np.random.default_rng(k)
    xv, wv = rng.integers(-1, 2, (m, k)), rng.integers(-1, 2, (n, k))
    xv[rng.random((m, k)) < 0.9] = 0
    e = rng.integers(-20, 21, k // 128)
    code = np.array([0xB8, 0, 0x38], np.uint8)
    xs, ws = np.tile((127 + e).astype(np.uint8), (m, 1)), np.tile((127 - e).astype(np.uint8), (n, 1))
    got = host(call((code[xv + 1], xs), (code[wv + 1], ws), TYPES[out], gpu))
    want = torch.from_numpy(xv).float() @ torch.from_numpy(wv).float().T        # whole numbers below 2^24
    assert np.array_equal(got, want.to(TYPES[out]).double().numpy())


@pytest.mark.parametrize("m", [1, 16, 40, 100, 300])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1280, 5504])
def test_scales_far_from_one(gpu, m, out, k):
    """Blocks of 2^-117 times 2^110 and the like: products stay ordinary numbers."""
    n = 140
    x, w = make(m, n, k, seed=m, outliers=False)
    for e in (-108, 117):
        xs = (x[1].astype(int) + e).clip(10, 245).astype(np.uint8)      # (codes of 2^-9 .. 448: within 2^-126 .. 2^127)
        ws = (w[1].astype(int) - e).clip(10, 245).astype(np.uint8)
        check((x[0], xs), (w[0], ws), TYPES[out], gpu)


@pytest.mark.parametrize("k", [640, 5248])
@pytest.mark.parametrize("m", [1, 12, 40, 300])
def test_rows_cut_out_of_others(gpu, m, k):
    """Any run of rows is rows again: scales then start at odd addresses."""
    n = 50
    x, w = make(m + 3, n + 3, k, seed=m)
    xc, xs, wc, ws = e4(x[0], gpu), e8(x[1], gpu), e4(w[0], gpu), e8(w[1], gpu)
    for out in (torch.float32, torch.float16):
        got = tl.f8_gemm(wc[3:], ws[3:], xc[3:], xs[3:], out_dtype=out)
        want = tl.f8_gemm(wc[3:].clone(), ws[3:].clone(), xc[3:].clone(), xs[3:].clone(), out_dtype=out)
        assert torch.equal(got, want)
    v = tl.f8_dequantize(wc, ws, out_dtype=torch.float32)
    assert torch.equal(tl.f8_dequantize(wc[3:], ws[3:], out_dtype=torch.float32), v[3:])
    ids = torch.arange(n, dtype=torch.int32, device=gpu)
    assert torch.equal(tl.f8_rows(wc[3:], ws[3:], ids, out_dtype=torch.float32), v[3:])
    c2, s2 = torch.full_like(wc.view(torch.uint8), 9), torch.full_like(ws.view(torch.uint8), 9)
    tl.f8_quantize(v[3:], c2.view(torch.float8_e4m3fn)[3:], s2.view(torch.float8_e8m0fnu)[3:])
    c1, s1 = tl.f8_quantize(v)
    assert bool((c2[:3] == 9).all() and (s2[:3] == 9).all())
    assert torch.equal(c2[3:], c1.view(torch.uint8)[3:]) and torch.equal(s2[3:], s1.view(torch.uint8)[3:])


def test_quantize_past_32_bits(gpu):
    """The last rows of more than 2^32 values."""
    m, k = 32800, 131072
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=gpu)
    x[m - 2] = 3.0
    x[m - 1, -1] = -448.0
    codes, scales = tl.f8_quantize(x)
    del x
    assert not codes[:m - 2].view(torch.uint8).any() and not scales[:m - 2].view(torch.uint8).any()
    back = tl.f8_dequantize(codes, scales)
    assert bool((back[m - 2] == 3).all()) and float(back[m - 1, -1]) == -448 and not back[m - 1, :-1].any()
    assert not back[:m - 2].any()


@pytest.mark.parametrize("m", [1, 16, 40, 300, 1100])
def test_weights_past_32_bits(gpu, m):
    """The last of more than 2^32 weights (and, for 1100 tokens, of as many outputs)."""
    n, k = (1 << 22) + 37, 1024
    codes = torch.zeros(n, k, dtype=torch.uint8, device=gpu)
    scales = torch.full((n, k // 128), 127, dtype=torch.uint8, device=gpu)
    rows = torch.tensor([0, 5, 1 << 21, n - 300, n - 38, n - 2, n - 1], device=gpu)
    g = torch.Generator().manual_seed(m)
    wv, xv = torch.randint(-1, 2, (len(rows), k), generator=g), torch.randint(-1, 2, (m, k), generator=g)
    code = torch.tensor([0xB8, 0, 0x38], dtype=torch.uint8)
    codes[rows] = code[wv + 1].to(gpu)
    xs = torch.full((m, k // 128), 127, dtype=torch.uint8, device=gpu)
    for out in (torch.float16, torch.float32) if m < 1100 else (torch.float16,):
        y = tl.f8_gemm(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu),
                       code[xv + 1].to(gpu).view(torch.float8_e4m3fn), xs.view(torch.float8_e8m0fnu), out_dtype=out)
        assert torch.equal(y[:, rows].float().cpu(), xv.float() @ wv.float().T)
        y[:, rows] = 0
        assert not y[0].any() and not y[m - 1].any() and not y[m // 2].any()


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("m,n,k", [(3, 515, 1024), (40, 96, 2048), (100, 1024, 7168), (300, 5200, 7040)])
def test_captured_and_replayed(gpu, m, n, k, out):
    """Two graphs over one workspace, one after the other, with other calls between."""
    x, w = make(m, n, k, seed=m)
    other = make(m, n, k, seed=m + 1)[0]
    xc, xs, wc, ws = e4(x[0], gpu), e8(x[1], gpu), e4(w[0], gpu), e8(w[1], gpu)
    room = torch.empty(max(16, tl.f8_gemm_workspace_bytes(m, n, k)), dtype=torch.uint8, device=gpu)
    run = lambda **kw: tl.f8_gemm(wc, ws, xc, xs, out_dtype=TYPES[out], **kw)  # noqa: E731
    want = run()
    graphs, outs = [], []
    for given in (room, room, None):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = run(workspace=given)
        graphs.append(g)
        outs.append(y)
    for i in range(3):
        src = (other if i == 1 else x)
        xc.view(torch.uint8).copy_(torch.from_numpy(src[0]))
        xs.view(torch.uint8).copy_(torch.from_numpy(src[1]))
        now = run()
        for g, y in zip(graphs, outs):
            y.zero_()
            g.replay()
            room.fill_(0xFF)
        torch.cuda.synchronize()
        assert all(torch.equal(y, now) for y in outs) and torch.equal(now, want) == (i != 1)


def test_linear_rounds_and_multiplies(gpu):
    g = torch.Generator().manual_seed(5)
    wf, xf = 0.02 * torch.randn(300, 1280, generator=g), torch.randn(9, 1280, generator=g)
    layer = tl.F8Linear(*tl.f8_quantize(wf.to(gpu)))
    for m in (1, 9):
        x = xf[:m].to(torch.bfloat16)
        want = oracle.f8_product(oracle.f8_quantize(x.double().numpy()), oracle.f8_quantize(wf.double().numpy()))
        got = host(layer(x.to(gpu)))
        assert np.allclose(got, want, rtol=1e-5, atol=1e-5 * np.abs(want).max())


def test_refusals_of_device_tensors(gpu):
    x, w = make(2, 32, 256)
    wc, ws, xc, xs = e4(w[0], gpu), e8(w[1], gpu), e4(x[0], gpu), e8(x[1], gpu)
    with pytest.raises(ValueError):
        tl.f8_gemm(wc, ws, xc[:, :128].contiguous(), xs[:, :1].contiguous())
    with pytest.raises(ValueError):
        tl.f8_gemm(wc, ws[:, :1].contiguous(), xc, xs)
    with pytest.raises(ValueError):
        tl.f8_gemm(wc, ws, xc, xs, out=torch.empty(32, 2, device=gpu))
    with pytest.raises(TypeError):
        tl.f8_gemm(wc, ws, xc, xs, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        tl.f8_dequantize(wc.t(), ws)
    with pytest.raises(ValueError):
        tl.f8_quantize(torch.zeros(2, 200, device=gpu))
    with pytest.raises(tl.TLError):
        tl.f8_quantize(torch.zeros(0, 128, device=gpu))

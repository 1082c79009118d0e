"""4-bit weights: rounding, values and the product with few tokens, against
their fp64 definitions.

Tolerance of the product, u = 2^-24: products of codes and activations are
exact; the sum within a group of G passes a term through at most G additions,
the scales and the sum over the groups add at most K/32 + 16 roundings, so
    |got - want| <= (G + K/32 + 16) u * sum_k |x w|,
whatever the order; 8-bit activations have exact group sums and scales of their
own (two more roundings).  bfloat16 activations below 2^-28 of the largest of
their 128 are off by at most 2^-29 of it: under 2^-28 * max |x| * sum |w|.  The output
adds half a step of its type."""
import numpy as np
import pytest
import torch

import oracle
import tl_hadamard_rotate_amd as tl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------ weights

def check_rounding(w64, group, packed, scales):
    codes, sc = oracle.q4_quantize(w64, group)
    assert np.array_equal(scales.cpu().numpy().view(np.uint16) & 0x7FFF, sc.view(np.uint16) & 0x7FFF)
    assert np.array_equal(packed.cpu().numpy(), oracle.q4_pack(codes))
    return codes, sc


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 128), (3, 384), (17, 1152), (5, 5120)])
def test_quantize_is_exact(gpu, n, k, group, kind):
    g = torch.Generator().manual_seed(n + k)
    w = (0.02 * torch.randn(n, k, generator=g)).to(TYPES[kind])
    packed, scales = tl.q4_quantize(w.to(gpu), group)
    codes, sc = check_rounding(w.double().numpy(), group, packed, scales)
    for out in ("f32", "f16", "bf16"):
        back = tl.q4_dequantize(packed, scales, out_dtype=TYPES[out])
        want = torch.from_numpy(oracle.q4_values(codes, sc).astype(np.float32)).to(TYPES[out])
        assert torch.equal(back.cpu(), want)


def test_quantize_ties_zeros_and_limits(gpu):
    w = np.zeros((6, 128), np.float32)
    w[0, :15] = np.arange(-7, 8) / 2 * 0.5           # scale 1/4 ... halves are ties
    w[0, 20] = 1.75
    w[1, :4] = [1e9, -1e9, 1e4, 3e4]                 # the scale is held at 65504
    w[2, :3] = [1e-7, -1e-7, 3e-8]                   # scale below the smallest binary16: 0
    w[3, :5] = [6e-8 * 7, 6e-8, -9e-8, 3e-8, -3e-8]  # subnormal scale
    w[5, :2] = [-8.0, 7.0]
    packed, scales = tl.q4_quantize(torch.from_numpy(w).to(gpu), 128)
    codes, sc = check_rounding(w.astype(np.float64), 128, packed, scales)
    assert sc[1, 0] == 65504 and sc[2, 0] == 0 and sc[4, 0] == 0 and 0 < sc[3, 0] < 6e-7
    assert not codes[2].any() and codes[1, 0] == 7 and codes[1, 1] == -8


def test_quantize_nonfinite_groups(gpu):
    w = torch.randn(3, 256)
    clean = tl.q4_quantize(w.to(gpu), 64)
    w[1, 70], w[2, 200] = float("inf"), float("nan")
    packed, scales = tl.q4_quantize(w.to(gpu), 64)
    back = host(tl.q4_dequantize(packed, scales))
    assert np.isnan(back[1, 64:128]).all() and np.isnan(back[2, 192:]).all()
    same = np.ones((3, 256), bool)
    same[1, 64:128] = same[2, 192:] = False
    assert np.array_equal(back[same], host(tl.q4_dequantize(*clean))[same])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 1024), (6, 5120)])
def test_quantize_rotated(gpu, n, k, group):
    """The rotation is fp32 (12 roundings of sum |w| / 32 over the block): the
    values lie within half a step of the rotated weights, the scale within its
    own rounding of the largest over 7."""
    g = torch.Generator().manual_seed(k + group)
    w = 0.02 * torch.randn(n, k, generator=g)
    s = (2 * torch.randint(0, 2, (k,), generator=g) - 1).to(torch.int8)
    packed, scales = tl.q4_quantize(w.to(gpu), group, signs=s.to(gpu))
    rot = oracle.fold_weights(w.double().numpy(), s.numpy())
    err = 12 * U * np.abs(w.double().numpy()).reshape(n, -1, 1024).sum(-1).max() / 32
    top = np.abs(rot).reshape(n, -1, group).max(-1)
    sc = host(scales)
    assert np.all(np.abs(sc - top / 7) <= top / 7 * 2.0 ** -11 + err)
    step = np.repeat(sc, group, axis=1)
    back = host(tl.q4_dequantize(packed, scales, out_dtype=torch.float32))
    # (the largest may exceed 7 steps by the rounding of the scale)
    assert np.all(np.abs(back - rot) <= step * (0.5 + 7 * 2.0 ** -11) + err)


def test_every_packed_byte_decodes(gpu):
    b = torch.arange(256, dtype=torch.uint8).repeat(2)[None].repeat(3, 1).contiguous()
    b[1] = b[1].flip(0)
    scales = torch.ones(3, 8, dtype=torch.float16)
    got = host(tl.q4_dequantize(b.to(gpu), scales.to(gpu), out_dtype=torch.float32))
    assert np.array_equal(got, oracle.q4_unpack(b.numpy()))


# ------------------------------------------------------------ product

def make(m, n, k, kind, group, gpu, seed=0, outliers=True):
    rng = np.random.default_rng(seed)
    codes = np.clip(np.rint(2.6 * rng.standard_normal((n, k))), -8, 7).astype(np.int8)
    scales = (0.004 + 0.008 * rng.random((n, k // group))).astype(np.float16)
    x = rng.standard_normal((m, k))
    if outliers:
        x[rng.random((m, k)) < 0.01] *= 20
    xs = None
    if kind == "i8":
        q, s = oracle.i8_quantize(x)
        q[0, :3] = -128
        x, xs = torch.from_numpy(q).to(gpu), torch.from_numpy(s.astype(np.float32)).to(gpu)
    else:
        x = torch.from_numpy(x.astype(np.float32)).to(TYPES[kind]).to(gpu)
    packed = torch.from_numpy(oracle.q4_pack(codes)).to(gpu)
    return x, xs, packed, torch.from_numpy(scales).to(gpu), codes, scales


def values(x, xs):
    return host(x) if xs is None else oracle.i8_values(x.cpu().numpy(), xs.cpu().numpy())


def check_product(got, x, xs, codes, scales, out):
    v = values(x, xs)
    want = oracle.q4_product(v, codes, scales)
    w = np.abs(oracle.q4_values(codes, scales))
    k, group = codes.shape[1], codes.shape[1] // scales.shape[1]
    tol = (group + k / 32 + 16) * U * (np.abs(v) @ w.T)
    if x.dtype == torch.bfloat16:
        top = np.abs(v).reshape(len(v), -1, 128).max(-1)
        tol += 2.0 ** -28 * (np.repeat(top, 128, axis=1) @ w.T)
    if out != torch.float32:
        tol += torch.finfo(out).eps / 2 * (np.abs(want) + tol) + 2.0 ** -25
    bad = np.abs(host(got) - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], host(got)[bad][:5], want[bad][:5], tol[bad][:5])


SIZES = [(1, 1, 128), (1, 16, 128), (1, 17, 256), (2, 15, 384), (3, 33, 1152), (4, 1000, 640),
         (5, 64, 1024), (8, 100, 5120), (15, 130, 1152), (16, 257, 2048), (1, 1024, 5120),
         (1, 520, 17408), (16, 40, 17408)]
MANY = [(17, 33, 384), (31, 64, 1024), (32, 100, 1152), (33, 257, 640), (48, 129, 5120), (64, 256, 2048),
        (64, 50, 17408), (65, 17, 256), (130, 70, 1024), (300, 1, 128)]


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", SIZES + MANY)
def test_product(gpu, m, n, k, group, kind):
    x, xs, packed, scales, codes, sc = make(m, n, k, kind, group, gpu, seed=m + n + k)
    out = [torch.float32, torch.float16, torch.bfloat16][(m + n) % 3]
    got = tl.q4_gemv(packed, scales, x, x_scales=xs, out_dtype=out)
    assert got.shape == (m, n) and got.dtype == out
    check_product(got, x, xs, codes, sc, out)


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("m,n,k", [(1, 6144, 5120), (8, 17408, 5120), (16, 5120, 17408), (37, 6144, 5120),
                                   (64, 5120, 17408)])
def test_product_at_projection_sizes(gpu, m, n, k, kind):
    x, xs, packed, scales, codes, sc = make(m, n, k, kind, 128, gpu, seed=1)
    check_product(tl.q4_gemv(packed, scales, x, x_scales=xs), x, xs, codes, sc, torch.float32)


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("m,group", [(1, 128), (5, 64), (20, 32), (64, 128)])
def test_product_of_the_longest_rows(gpu, m, group, kind):
    x, xs, packed, scales, codes, sc = make(m, 19, 1 << 20, kind, group, gpu, seed=m)
    check_product(tl.q4_gemv(packed, scales, x, x_scales=xs), x, xs, codes, sc, torch.float32)


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
def test_one_hot_activations_give_the_weights(gpu, kind):
    """y of a one-hot token is one column of the weights, exactly; every token
    and column position is tried."""
    k, n = 384, 40
    rng = np.random.default_rng(5)
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    sc = (2.0 ** rng.integers(-6, 3, (n, k // 32))).astype(np.float16)
    packed, scales = torch.from_numpy(oracle.q4_pack(codes)).to(gpu), torch.from_numpy(sc).to(gpu)
    x = torch.eye(k, device=gpu)
    xs = None
    if kind == "i8":
        x, xs = x.to(torch.int8), torch.ones(k, k // 128, device=gpu)
    else:
        x = x.to(TYPES[kind])
    want = oracle.q4_values(codes, sc).T
    for m in (1, 16, 48, k):
        for t in range(0, k, m):
            rows = slice(t, t + m)
            got = tl.q4_gemv(packed, scales, x[rows].contiguous(),
                             x_scales=None if xs is None else xs[rows].contiguous())
            assert np.array_equal(host(got), want[rows])


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("m", [2, 16, 40])
def test_tokens_do_not_touch_each_other(gpu, m, kind):
    """A NaN or infinity in one token leaves the others' bits alone."""
    x, xs, packed, scales, codes, sc = make(m, 100, 1152, kind, 64, gpu)
    clean = tl.q4_gemv(packed, scales, x, x_scales=xs)
    for value in (float("nan"), float("inf")):
        bad = (x if xs is None else xs).clone()
        bad[m // 2, 3] = value
        got = tl.q4_gemv(packed, scales, bad if xs is None else x, x_scales=None if xs is None else bad)
        keep = [i for i in range(m) if i != m // 2]
        assert torch.equal(got[keep], clean[keep])
        assert not torch.isfinite(got[m // 2]).any()


def test_zero_activations_and_scales(gpu):
    for kind in ("f16", "bf16", "i8"):
        x, xs, packed, scales, _, _ = make(3, 50, 512, kind, 32, gpu)
        x[1] = 0
        if xs is not None:
            xs[1] = 0
        scales[7] = 0
        y = tl.q4_gemv(packed, scales, x, x_scales=xs)
        assert not y[1].any() and not y[:, 7].any() and y[0, 0] != 0


def test_wide_range_of_bfloat16_activations(gpu):
    """Activations from 1e-30 to 1e30 in one row, each group of one size or
    mixed: exact down to 2^-28 of the group's largest."""
    x, _, packed, scales, codes, sc = make(3, 60, 1024, "bf16", 128, gpu, outliers=False)
    f = torch.tensor([1e-30, 1e30, 1e-3, 1.0, 1e10, 1e-20, 1e3, 1e-38], device=gpu)
    for rows, value in ((0, f.repeat_interleave(128)), (1, f.repeat(128)), (2, 10 * f[2])):
        x[rows] = (x[rows].float() * value).to(torch.bfloat16)
    check_product(tl.q4_gemv(packed, scales, x), x, None, codes, sc, torch.float32)


def test_largest_and_smallest_binary16(gpu):
    x, _, packed, scales, codes, sc = make(2, 60, 512, "f16", 64, gpu, outliers=False)
    x[0] = torch.sign(x[0]) * 65504
    x[1] = torch.sign(x[1]) * 2.0 ** -24
    check_product(tl.q4_gemv(packed, scales, x), x, None, codes, sc, torch.float32)


@pytest.mark.parametrize("m", [1, 5, 16, 23, 64])
def test_neighbouring_memory_is_left_alone(gpu, m):
    n, k = 37, 384
    for kind in ("f16", "i8"):
        x, xs, packed, scales, codes, sc = make(m, n, k, kind, 32, gpu)
        for out in (torch.float32, torch.float16):
            pad = 64
            big = torch.full((m * n + 2 * pad,), 7.0, dtype=out, device=gpu)
            y = big[pad:pad + m * n].view(m, n)
            tl.q4_gemv(packed, scales, x, x_scales=xs, out_dtype=out, out=y)
            check_product(y, x, xs, codes, sc, out)
            assert (big[:pad] == 7).all() and (big[pad + m * n:] == 7).all()


@pytest.mark.parametrize("m", [24, 64])
def test_workspace_bounds(gpu, m):
    """The workspace's stated size is enough, its contents do not matter, and
    nothing behind it is written."""
    n, k = 512, 17408
    x, _, packed, scales, codes, sc = make(m, n, k, "f16", 128, gpu)
    need = tl.q4_gemv_workspace_bytes(m, n, k)
    big = torch.full((need + 512,), 255, dtype=torch.uint8, device=gpu)
    y = tl.q4_gemv(packed, scales, x, workspace=big[:need])
    check_product(y, x, None, codes, sc, torch.float32)
    assert (big[need:] == 255).all()
    if need:
        with pytest.raises(tl.TLError, match="TL_ERR_WORKSPACE"):
            tl.q4_gemv(packed, scales, x, workspace=big[:need - 16])


def test_refused_calls(gpu):
    x, _, packed, scales, _, _ = make(2, 32, 512, "f16", 64, gpu)
    q = x.to(torch.int8)
    s = torch.ones(2, 4, device=gpu)
    y = torch.full((2, 32), 7.0, device=gpu)
    for bad in (lambda: tl.q4_gemv(packed, scales, x[:, :256], out=y),
                lambda: tl.q4_gemv(packed, scales[:, :3].contiguous(), x, out=y),
                lambda: tl.q4_gemv(packed, scales[:16], x, out=y),
                lambda: tl.q4_gemv(packed, scales, x, x_scales=s, out=y),
                lambda: tl.q4_gemv(packed, scales, q, out=y),
                lambda: tl.q4_gemv(packed, scales, q, x_scales=s[:, :2].contiguous(), out=y),
                lambda: tl.q4_gemv(packed, scales, x.t().contiguous().t(), out=y),
                lambda: tl.q4_gemv(packed, scales, x.cpu(), out=y),
                lambda: tl.q4_gemv(packed, scales, x, out=y[:1]),
                lambda: tl.q4_gemv(packed, scales, x.float(), out=y),
                lambda: tl.q4_gemv(packed, scales, x, out_dtype=torch.int8),
                lambda: tl.q4_quantize(x.float(), group=96),
                lambda: tl.q4_quantize(x[:, :200].float().contiguous()),
                lambda: tl.q4_dequantize(packed, scales, out=x)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(tl.TLError):        # no tokens (torch gives an empty view no address)
        tl.q4_gemv(packed, scales, x[:0], out=y[:0])
    with pytest.raises(tl.TLError, match="TL_ERR_ALIGN"):
        tl.q4_gemv(packed, scales, torch.zeros(1025, dtype=torch.float16, device=gpu)[1:].view(2, 512), out=y)
    assert (y == 7).all()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("m", [1, 16, 40])
def test_streams_graph_replays_and_repeats(gpu, m, kind):
    n, k = 1000, 5120
    x, xs, packed, scales, _, _ = make(m, n, k, kind, 128, gpu)
    want = tl.q4_gemv(packed, scales, x, x_scales=xs)
    assert torch.equal(want, tl.q4_gemv(packed, scales, x, x_scales=xs))
    # two calls that may run at once, each with a workspace of its own
    sides, ys = [torch.cuda.Stream() for _ in range(2)], []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ys.append(tl.q4_gemv(packed, scales, x, x_scales=xs))
    for s in sides:
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ys[0], want) and torch.equal(ys[1], want)
    y = torch.zeros_like(want)
    ws = torch.empty(max(1, tl.q4_gemv_workspace_bytes(m, n, k)), dtype=torch.uint8, device=gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.q4_gemv(packed, scales, x, x_scales=xs, out=y, workspace=ws)
    for i in range(4):
        if kind == "i8":
            x.copy_(torch.randint(-127, 128, x.shape, device=gpu))
        else:
            x.copy_(torch.randn_like(x))
        want = tl.q4_gemv(packed, scales, x, x_scales=xs)
        y.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_offsets_past_32_bits(gpu):
    """More than 2^32 packed bytes and 2^33 weights: rows at both ends against
    the same rows alone."""
    k, n = 16384, (1 << 19) + 5
    packed = torch.zeros(n, k // 2, dtype=torch.uint8, device=gpu)
    scales = torch.ones(n, k // 128, dtype=torch.float16, device=gpu)
    ends = [0, 1, 17, n - 18, n - 2, n - 1]
    packed[ends] = torch.randint(0, 256, (len(ends), k // 2), device=gpu).to(torch.uint8)
    codes = oracle.q4_unpack(packed[ends].cpu().numpy())
    one = np.ones((len(ends), k // 128), np.float16)
    for m in (1, 20):
        x = torch.randn(m, k, device=gpu).to(torch.float16)
        y = tl.q4_gemv(packed, scales, x)
        check_product(y[:, ends], x, None, codes, one, torch.float32)
        assert int((y != 0).any(0).sum()) == len(ends)
    back = tl.q4_dequantize(packed, scales)                 # 2^33 values
    assert np.array_equal(host(back[ends]), codes)
    again, s = tl.q4_quantize(back)
    assert int((again != 0).any(1).sum()) == len(ends)
    c2, s2 = oracle.q4_quantize(codes.astype(np.float64), 128)
    assert np.array_equal(again[ends].cpu().numpy(), oracle.q4_pack(c2))
    assert np.array_equal(s[ends].cpu().numpy(), s2)


def test_more_tokens_than_one_launch(gpu):
    """One token more than a launch takes: it is alone in the last one, whose
    split is still that of all tokens."""
    m, n, k = 65535 * 16 + 1, 16384, 1408
    g = torch.Generator(device=gpu).manual_seed(3)
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device=gpu, dtype=torch.uint8)
    scales = torch.rand(n, k // 32, generator=g, device=gpu).add_(0.5).half()
    x = torch.randint(-127, 128, (m, k), generator=g, device=gpu, dtype=torch.int8)
    xs = torch.rand(m, k // 128, generator=g, device=gpu).add_(0.5).div_(4096)
    y = tl.q4_gemv(packed, scales, x, xs, out_dtype=torch.float16)
    some = [0, 63, 64, 500000, m - 2, m - 1]
    check_product(y[some], x[some], xs[some], oracle.q4_unpack(packed.cpu().numpy()), scales.cpu().numpy(),
                  torch.float16)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_more_tokens_than_the_workspace_holds(gpu, kind):
    """A prompt whose parts' sums are done in turn, the last turn of few
    tokens: tokens at the ends of the turns, nothing written behind the
    workspace, replays of a graph."""
    m, n, k = 1601, 17408, 5120
    g = torch.Generator(device=gpu).manual_seed(4)
    packed = torch.randint(0, 256, (n, k // 2), generator=g, device=gpu, dtype=torch.uint8)
    scales = torch.rand(n, k // 128, generator=g, device=gpu).add_(0.5).half()
    xs = None
    if kind == "i8":
        x = torch.randint(-127, 128, (m, k), generator=g, device=gpu, dtype=torch.int8)
        xs = torch.rand(m, k // 128, generator=g, device=gpu).add_(0.5).div_(4096)
    else:
        x = torch.randn(m, k, generator=g, device=gpu).half()
    need = tl.q4_gemv_workspace_bytes(m, n, k)
    assert 0 < need <= 1 << 28
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=gpu)
    y = torch.empty(m, n, device=gpu)
    tl.q4_gemv(packed, scales, x, xs, out=y, workspace=ws[:need])
    assert (ws[need:] == 255).all()
    rows = torch.cat([torch.arange(0, n, 997, device=gpu), torch.tensor([n - 1], device=gpu)])
    some = [0, 1, 63, 64, 511, 512, 575, 576, 639, 640, 767, 768, 769, 1023, 1024, 1535, 1536, m - 2, m - 1]
    check_product(y[some][:, rows], x[some], None if xs is None else xs[some],
                  oracle.q4_unpack(packed[rows].cpu().numpy()), scales[rows].cpu().numpy(), torch.float32)
    # every token: 128 at a time, another split.  Each result is off by (128 + k/32 + 16) u
    # = 1.9e-5 of sum |x w|, which is about 0.64 sqrt(k) = 46 deviations of y, the largest
    # of a batch at least 3: together under 2 * 1.9e-5 * 46 / 3 = 6e-4 of the largest
    for i in range(0, m, 128):
        part = tl.q4_gemv(packed, scales, x[i:i + 128], None if xs is None else xs[i:i + 128])
        assert torch.allclose(part, y[i:i + 128], rtol=1e-3, atol=1e-3 * float(part.abs().max()))
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.q4_gemv(packed, scales, x, xs, out=y, workspace=ws[:need])
    for _ in range(3):
        y.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ------------------------------------------------------------ together

@pytest.mark.parametrize("rot", [False, True])
@pytest.mark.parametrize("m", [1, 16, 40])
def test_norm_rounding_and_product_together(gpu, m, rot):
    """A block's step as it is used: residual and norm to 8 bits, the product
    with weights rounded (and rotated) by the library.  Against the definition
    in 64 bits on the library's own codes to the product's bound; against the
    unrounded norm and weights within the errors of 8 and 4 bits: a step's
    rounding is uniform, so its deviation is step / sqrt(12), and the steps
    are the largest of 128 over 127 and over 7."""
    k, n = 5120, 300
    g = torch.Generator().manual_seed(m)
    x, r = (torch.randn(m, k, generator=g).half().to(gpu) for _ in range(2))
    gain = (1 + 0.1 * torch.randn(k, generator=g)).half().to(gpu)
    w = (0.02 * torch.randn(n, k, generator=g)).to(gpu)
    s = (2 * torch.randint(0, 2, (k,), generator=g) - 1).to(torch.int8).to(gpu) if rot else None
    packed, scales = tl.q4_quantize(w, 128, signs=s)
    q, qs, total = tl.rms_norm_i8(x, gain, 1e-6, residual=r, signs=s)
    layer = tl.Q4Linear(packed, scales, s)
    y = layer(q, qs)
    codes = oracle.q4_unpack(packed.cpu().numpy())
    check_product(y, q, qs, codes, scales.cpu().numpy(), torch.float32)
    h = oracle.rms_sum(host(x), host(r), "f16")
    assert np.array_equal(host(total), h)
    full = oracle.rms_norm(h, host(gain), 1e-6) @ host(w).T     # the rotation cancels
    # largest of 128 normal values: at most about 4 deviations
    rel = np.sqrt((4 / 7) ** 2 / 12 + (4 / 127) ** 2 / 12)
    assert oracle.rel_l2(host(y), full) < 1.5 * rel
    # the float16 way through the same layer
    v = tl.rms_norm(x, gain, 1e-6, residual=r)[0]
    assert oracle.rel_l2(host(layer(v)), full) < 1.5 * rel

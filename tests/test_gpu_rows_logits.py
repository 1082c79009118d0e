"""Embedding rows and the adjustment of logits against their fp64 definitions,
and the whole run from token to logits.

Rows: code * scale is exact in fp32, the factor's product rounds once there and
once to the output.  Logits: at most six fp32 operations, each off by half a step
of a magnitude of at most m = |x| max(r, 1 / r) + |f n| + |p| + |b|, so
|got - want| <= 6 * 2^-24 * m plus half a step of the output's type."""
import numpy as np
import pytest
import torch

import oracle
import tl_hadamard_rotate_amd as tl

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------ rows

def table(form, n, k, gpu, seed=0):
    """(arguments of the call, fp64 values) of a table of the form."""
    w = (0.02 * torch.randn(n, k, generator=torch.Generator().manual_seed(seed)))
    if form == "f8":
        codes, scales = tl.f8_quantize(w.to(gpu))
        return (codes, scales), oracle.f8_values(codes.view(torch.uint8).cpu().numpy(), scales.view(torch.uint8).cpu().numpy())
    packed, scales = tl.q4_quantize(w.to(gpu), int(form[3:]))
    return (packed, scales), oracle.q4_values(oracle.q4_unpack(packed.cpu().numpy()), scales.cpu().numpy())


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["f8", "q4_32", "q4_64", "q4_128"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (7, 50, 384), (33, 1000, 1152), (2, 300, 5120), (600, 77, 128),
                                   (4099, 60, 2176)])
def test_rows(gpu, m, n, k, form, out):
    args, values = table(form, n, k, gpu, seed=n)
    call = tl.f8_rows if form == "f8" else tl.q4_rows
    ids = np.random.default_rng(m).integers(-3, n + 3, m).astype(np.int32)
    ids[0] = n - 1                      # the last row; then repeated and outside ones
    if m > 6:
        ids[1:6] = [n - 1, -1, n, 2 ** 31 - 1, -2 ** 31]
    factor = 5120 ** 0.5
    got = host(call(*args, torch.from_numpy(ids).to(gpu), factor, out_dtype=TYPES[out]))
    want = oracle.lookup(values, ids.tolist(), float(np.float32(factor)))
    tol = (HALF["f32"] + (HALF[out] if out != "f32" else 0)) * np.abs(want) * 1.001 + (2.0 ** -25 if out == "f16" else 0)
    assert np.all(np.abs(got - want) <= tol)
    assert not got[(ids < 0) | (ids >= n)].any()
    # without a factor the values themselves
    plain = call(*args, torch.from_numpy(ids).to(gpu), out_dtype=TYPES[out])
    assert torch.equal(plain.cpu(), torch.from_numpy(oracle.lookup(values, ids.tolist(), 1.0)).float().to(TYPES[out]))


def test_rows_leave_what_is_behind_them(gpu):
    args, _ = table("f8", 20, 256, gpu)
    big = torch.full((9, 256), 3.0, dtype=torch.float16, device=gpu)
    tl.f8_rows(*args, torch.tensor([1, 2, 99, 3], dtype=torch.int32, device=gpu), out=big[:4])
    assert bool((big[4:] == 3).all()) and not big[2].any() and bool(big[3].any())


def test_rows_past_32_bits(gpu):
    """The last rows of a table of more than 2^32 values."""
    n, k = 40000, 131072
    codes = torch.zeros(n, k, dtype=torch.uint8, device=gpu)
    scales = torch.full((n, k // 128), 127, dtype=torch.uint8, device=gpu)
    codes[n - 1] = 0x38
    codes[n - 2, -1] = 0x40
    ids = torch.tensor([0, n - 1, n - 2, n], dtype=torch.int32, device=gpu)
    got = tl.f8_rows(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), ids, 2.0)
    assert not got[0].any() and bool((got[1] == 2).all()) and not got[3].any()
    assert float(got[2, -1]) == 4 and not got[2, :-1].any()


# ------------------------------------------------------------ logits

def case(m, v, h, b, mask, seed):
    rng = np.random.default_rng(seed)
    c = {"logits": 3 * rng.standard_normal((m, v))}
    if h:
        c["history"] = (v * rng.random((m, h)) ** 4).astype(np.int32)
        c["history"][rng.random((m, h)) < 0.05] = -1
        c["history"][0, 0] = v                                  # just outside
        c["history_lens"] = rng.integers(0, h + 1, m).astype(np.int32)
        c["history_lens"][0] = h
        c["prompt_lens"] = rng.integers(0, h + 1, m).astype(np.int32)
        c["repetition"] = (0.7 + rng.random(m)).astype(np.float32)
        c["presence"] = rng.standard_normal(m).astype(np.float32)
        c["frequency"] = (0.2 * rng.random(m)).astype(np.float32)
        if m > 1:
            c["history_lens"][1] = 0
    if b:
        c["bias_ids"] = rng.integers(-2, v + 2, (m, b)).astype(np.int32)
        c["bias_ids"][:, b // 2] = c["bias_ids"][:, 0]          # named twice
        c["bias_values"] = (4 * rng.standard_normal((m, b))).astype(np.float32)
    if mask:
        c["mask"] = rng.integers(0, 2 ** 32, (m, (v + 31) // 32), dtype=np.uint64).astype(np.uint32)
        c["mask"][m - 1] = 0 if m > 1 else c["mask"][0]         # a row that allows nothing
    return c


def to_device(c, kind, gpu):
    t = {}
    for name, a in c.items():
        if name == "logits":
            t[name] = torch.from_numpy(a).to(TYPES[kind]).to(gpu)
        else:
            t[name] = torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(gpu)
    return t


def check(got, c, kind, out):
    c = dict(c, logits=torch.from_numpy(c["logits"]).to(TYPES[kind]).double().numpy())
    want = oracle.adjust_logits(**c)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    mag = np.abs(c["logits"])
    if "history" in c:
        col = lambda n: np.abs(c[n].astype(np.float64))[:, None] if n in c else 0.0  # noqa: E731
        r = col("repetition") if "repetition" in c else 1.0
        mag = mag * np.maximum(r, 1 / r) + col("frequency") * c["history"].shape[1] + col("presence")
    if "bias_values" in c:
        mag = mag + np.abs(c["bias_values"]).max()
    fine = np.isfinite(want)
    tol = 6 * 2.0 ** -24 * mag[fine] + HALF[out] * np.abs(want[fine]) + (2.0 ** -25 if out == "f16" else 0)
    assert np.all(np.abs(got[fine] - want[fine]) <= tol)


@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"),
                                      ("f16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("m,v,h,b,mask", [(1, 1, 1, 1, True), (1, 33, 5, 3, True), (3, 1000, 40, 0, False),
                                          (2, 8191, 300, 17, True), (2, 8193, 0, 9, True), (4, 20007, 900, 0, True),
                                          (1, 40000, 3000, 64, False), (3, 32003, 0, 0, True), (2, 77, 0, 0, False)])
def test_logits(gpu, m, v, h, b, mask, kind, out):
    c = case(m, v, h, b, mask, seed=v + h)
    t = to_device(c, kind, gpu)
    check(host(tl.adjust_logits(**t, out_dtype=TYPES[out])), c, kind, out)
    if kind == out:                                            # in place
        want = tl.adjust_logits(**t)
        tl.adjust_logits(**t, out=t["logits"])
        assert torch.equal(t["logits"], want)


@pytest.mark.parametrize("given", [("repetition",), ("presence",), ("frequency",), ("history_lens",), ("prompt_lens",), ()])
def test_each_penalty_alone(gpu, given):
    c = case(3, 500, 60, 0, False, seed=4)
    c = {n: a for n, a in c.items() if n in ("logits", "history") + given}
    check(host(tl.adjust_logits(**to_device(c, "f32", gpu))), c, "f32", "f32")


def test_a_token_repeated_throughout(gpu):
    """Every place of a long history names one token; lengths past its ends."""
    v, h = 9000, 20000
    c = {"logits": np.ones((3, v)), "history": np.full((3, h), 8999, np.int32),
         "history_lens": np.array([h, 2 ** 31 - 1, -5], np.int32), "prompt_lens": np.array([0, 1, 2 ** 31 - 1], np.int32),
         "repetition": np.full(3, 2, np.float32), "presence": np.zeros(3, np.float32),
         "frequency": np.full(3, 2.0 ** -10, np.float32)}
    got = host(tl.adjust_logits(**to_device(c, "f32", gpu)))
    assert got[0, 8999] == 0.5 - h * 2.0 ** -10 and got[1, 8999] == 0.5 - (h - 1) * 2.0 ** -10 and got[2, 8999] == 1
    assert np.array_equal(got[:, :8999], np.ones((3, 8999)))


def test_the_longest_histories_and_bias_lists(gpu):
    """Counts and places beyond 16 bits."""
    v, h, b = 20000, 70000, 70000
    c = case(2, v, h, b, True, seed=9)
    c["history"][0, ::2], c["history_lens"][0], c["prompt_lens"][0] = 7, h, 11
    c["frequency"][:] = 2.0 ** -12
    c["bias_ids"][1, :], c["bias_ids"][1, -1] = 3, 4
    check(host(tl.adjust_logits(**to_device(c, "f32", gpu))), c, "f32", "f32")


@pytest.mark.parametrize("m,v,h,b", [(1100, 501, 50, 3), (260, 30011, 700, 0), (520, 9001, 0, 40), (35, 250007, 300, 20)])
def test_many_sequences(gpu, m, v, h, b):
    c = case(m, v, h, b, True, seed=m)
    check(host(tl.adjust_logits(**to_device(c, "bf16", gpu), out_dtype=torch.float32)), c, "bf16", "f32")


def test_what_is_not_finite(gpu):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf, -inf, nan, 1.0, nan, inf, -inf, -3.4e38]], device=gpu)
    every = torch.arange(8, dtype=torch.int32, device=gpu)[None]
    got = tl.adjust_logits(x, history=every, repetition=torch.tensor([2.0], device=gpu),
                           presence=torch.tensor([1.0], device=gpu), mask=torch.tensor([[0b10001111]], dtype=torch.int32, device=gpu))
    assert torch.equal(got[0, [0, 1, 3, 4, 5, 6, 7]].cpu(), torch.tensor([inf, -inf, -0.5, -inf, -inf, -inf, -inf]))
    assert bool(got[0, 2].isnan())


def test_empty_history_and_biases(gpu):
    x = torch.randn(2, 300, device=gpu)
    none = torch.empty(2, 0, dtype=torch.int32, device=gpu)
    one = torch.ones(2, device=gpu)
    got = tl.adjust_logits(x, history=none, repetition=2 * one, bias_ids=none, bias_values=none.float())
    assert torch.equal(got, x)
    with pytest.raises(ValueError):
        tl.adjust_logits(x, repetition=one)
    with pytest.raises(TypeError):
        tl.adjust_logits(x, bias_ids=none)
    with pytest.raises(ValueError):
        tl.adjust_logits(x, mask=none)
    with pytest.raises(TypeError):
        tl.adjust_logits(x, history=none.long())


def test_many_rows(gpu):
    """More rows than a grid's second dimension holds."""
    m, v = 70000, 40
    x = torch.zeros(m, v, dtype=torch.float16, device=gpu)
    ids = (torch.arange(m, dtype=torch.int32, device=gpu) % v)[:, None].contiguous()
    got = tl.adjust_logits(x, bias_ids=ids, bias_values=torch.ones(m, 1, device=gpu))
    assert torch.equal(got, torch.zeros_like(x).scatter_(1, ids.long(), 1))


def test_as_many_rows_as_may_be(gpu):
    """A lane or more for each of 2^24 rows, and more lanes than one launch has."""
    m = 1 << 24
    x = torch.arange(m, dtype=torch.float32, device=gpu)[:, None]
    ids = (torch.arange(m, dtype=torch.int32, device=gpu) % 2)[:, None].contiguous()
    got = tl.adjust_logits(x, bias_ids=ids, bias_values=torch.ones(m, 1, device=gpu))
    assert torch.equal(got[:, 0], x[:, 0] + (ids[:, 0] == 0))


def test_logits_past_32_bits(gpu):
    m, v = 4100, 1 << 20
    x = torch.zeros(m, v, dtype=torch.float16, device=gpu)
    ids = torch.full((m, 2), v - 1, dtype=torch.int32, device=gpu)
    ids[:, 0] = torch.arange(m, device=gpu)
    mask = torch.full((m, v // 32), -1, dtype=torch.int32, device=gpu)
    mask[m - 1, 7] = ~1
    tl.adjust_logits(x, bias_ids=ids, bias_values=torch.tensor([[1.0, 2.0]], device=gpu).repeat(m, 1), mask=mask, out=x)
    at = torch.arange(m, device=gpu)
    assert bool((x[:, v - 1] == 2).all()) and bool((x[at, at] == 1).all()) and float(x[m - 1, 224]) == -float("inf")
    x[:, v - 1], x[at, at], x[m - 1, 224] = 0, 0, 0
    assert not any(bool(x[i:i + 512].any()) for i in range(0, m, 512))


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_logits_larger_than_the_caches(gpu, out):
    """Rows that start at every alignment of the type."""
    m, v = 530, 131075
    x = (torch.arange(m * v, device=gpu, dtype=torch.int32) % 251).view(m, v).to(torch.bfloat16)
    big = torch.full((m + 1, v), 7.0, dtype=TYPES[out], device=gpu)
    ids = torch.stack([torch.arange(m, device=gpu), torch.full((m,), v - 1, device=gpu)], 1).int().contiguous()
    tl.adjust_logits(x, bias_ids=ids, bias_values=torch.full((m, 2), 4.0, device=gpu), out_dtype=TYPES[out], out=big[:m])
    want = x.float().scatter_add_(1, ids.long(), torch.full((m, 2), 4.0, device=gpu)).to(TYPES[out])
    assert torch.equal(big[:m], want) and bool((big[m] == 7).all())


def test_rows_past_one_launch(gpu):
    """More lanes of 8 values than a launch has."""
    m, n, k = 1 << 24, 1000, 1152
    args, _ = table("f8", n, k, gpu)
    ids = torch.arange(m, dtype=torch.int32, device=gpu) % (n + 1)
    got = tl.f8_rows(*args, ids)
    want = torch.cat([tl.f8_dequantize(*args), torch.zeros(1, k, dtype=torch.float16, device=gpu)])
    for at in list(range(0, m, m // 7)) + [m - 4096, (1 << 31) // (k // 8) - 2048]:
        assert torch.equal(got[at:at + 4096], want[ids[at:at + 4096].long()]), at


# ------------------------------------------------------------ the run

def run_of_calls(embedding, head, gain, ids, history, mask, bufs=None):
    """Token ids to adjusted logits: embedding, norm, 8-bit rows, head, penalties."""
    h = tl.f8_rows(*embedding, ids, 32.0, out_dtype=torch.bfloat16)
    y = tl.rms_norm(h, gain, 1e-6, out_dtype=torch.bfloat16)
    logits = tl.f8_gemm(*head, *tl.f8_quantize(y), out_dtype=torch.float32)
    m = ids.shape[0]
    return tl.adjust_logits(logits, history=history, repetition=torch.full((m,), 1.25, device=ids.device),
                            mask=mask, out=logits)


@pytest.mark.parametrize("m", [1, 5, 70])
def test_from_token_to_logits(gpu, m):
    n, k = 515, 1024
    rng = np.random.default_rng(m)
    embedding, values = table("f8", n, k, gpu, seed=1)
    head, weights = table("f8", n, k, gpu, seed=2)
    gain = torch.ones(k, dtype=torch.bfloat16, device=gpu)
    ids = rng.integers(0, n, m).astype(np.int32)
    history = rng.integers(0, n, (m, 12)).astype(np.int32)
    mask = rng.integers(0, 2 ** 32, (m, (n + 31) // 32), dtype=np.uint64).astype(np.uint32)
    dev = [torch.from_numpy(a.view(np.int32)).to(gpu) for a in (ids, history, mask)]
    got = run_of_calls(embedding, head, gain, *dev)
    h = torch.from_numpy(oracle.lookup(values, ids.tolist(), 32.0)).to(torch.bfloat16).double().numpy()
    # codes depend on the norm's own rounding: taken from the call, the rest from the definitions
    y = tl.rms_norm(torch.from_numpy(h).to(torch.bfloat16).to(gpu), gain, 1e-6, out_dtype=torch.bfloat16)
    x = oracle.f8_values(*oracle.f8_quantize(y.double().cpu().numpy()))
    want = oracle.adjust_logits(x @ weights.T, history=history, repetition=np.full(m, 1.25), mask=mask)
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(host(got)))
    tol = 2 * 2.0 ** -24 * (k / 32 + 60) * 1.25 * (np.abs(x) @ np.abs(weights).T)
    assert np.all(np.abs(host(got)[fine] - want[fine]) <= tol[fine])

    # captured, replayed with the program's own work in between, on another stream
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run_of_calls(embedding, head, gain, *dev)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = run_of_calls(embedding, head, gain, *dev)
    for i in range(3):
        ids2 = torch.from_numpy(rng.integers(0, n, m).astype(np.int32)).to(gpu)
        dev[0].copy_(ids2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, run_of_calls(embedding, head, gain, *dev)), i


def test_two_streams_at_once(gpu):
    embedding, _ = table("q4_64", 400, 1024, gpu)
    head, _ = table("f8", 2000, 1024, gpu)
    x = [torch.randn(m, 1024, device=gpu) for m in (3, 200)]
    want = [tl.f8_gemm(*head, *tl.f8_quantize(a), out_dtype=torch.float16) for a in x]
    ids = torch.arange(400, dtype=torch.int32, device=gpu)
    rows = tl.q4_rows(*embedding, ids, 2.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(3):
        got = []
        for s, a in zip(streams, x):
            with torch.cuda.stream(s):
                got.append((tl.f8_gemm(*head, *tl.f8_quantize(a), out_dtype=torch.float16),
                            tl.q4_rows(*embedding, ids, 2.0)))
        torch.cuda.synchronize()
        for (y, r), w in zip(got, want):
            assert torch.equal(y, w) and torch.equal(r, rows)

"""The two ends of a model around the ternary linears, as cases to time and compare.

Token ids become rows of the embedding, the last hidden rows meet the head, and
the head's logits are adjusted before a token is drawn:

  rows      ``q4_rows`` and ``f8_rows``: embedding lookup with a scaling factor
            in tables of 4-bit codes or of 8-bit floating point
  quantize  ``f8_quantize`` then ``f8_dequantize``: rows (weights or
            activations) to 8-bit floating point (e4m3) with a power-of-two
            scale for each block of 128, and back to the values these stand for
  product   ``f8_gemm``: product of rows and weights in that form, from one
            token to a prompt
  logits    ``adjust_logits``: penalties for repeated tokens, biases and a
            grammar's mask

Shapes are those of the library's benchmark (K = 5120 and 17408 inputs; k/v,
gate/up and down projections) and generic vocabularies and odd sizes.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
LARGEST_WEIGHT = 131072 * 5120             # the listed head
LARGEST_PRODUCT = 4096 * 17408 * 5120      # the listed prompt
LARGEST_QUANTIZE = 17408 * 5120            # the listed projection
LARGEST_ROWS = 4096 * 5120                 # the listed prompt's embedding
LARGEST_LOGITS = 64 * 131072               # the listed batch


def listed():
    return [
        # the embedding of one new token: latency counts
        {"name": "rows token q4", "op": "rows", "form": "q4", "m": 1, "n": 131072, "k": 5120,
         "group": 128, "out": "f16"},
        # a prompt's embedding, padded, for a bfloat16 stream
        {"name": "rows prompt f8", "op": "rows", "form": "f8", "m": 4096, "n": 131072, "k": 5120,
         "out": "bf16"},
        # one token's activations in front of a product
        {"name": "quantize token", "op": "quantize", "m": 1, "k": 5120, "x": "f16"},
        # a projection's weights, when a model is loaded
        {"name": "quantize gate weights", "op": "quantize", "m": 17408, "k": 5120, "x": "f32"},
        # k/v projection of one token: the smallest product
        {"name": "product token kv", "op": "product", "m": 1, "n": 1024, "k": 5120, "out": "f32"},
        # the head of one token
        {"name": "product token head", "op": "product", "m": 1, "n": 131072, "k": 5120, "out": "f32"},
        # down projection of thirteen decoding sequences
        {"name": "product batch down", "op": "product", "m": 13, "n": 5120, "k": 17408, "out": "bf16"},
        # scoring a text: the head of every position, a vocabulary that divides by nothing
        {"name": "product ragged head", "op": "product", "m": 1000, "n": 32003, "k": 5120, "out": "f16"},
        # gate/up projection of a prompt
        {"name": "product prompt gate", "op": "product", "m": 4096, "n": 17408, "k": 5120, "out": "bf16"},
        # one sequence about to draw its next token
        {"name": "logits token", "op": "logits", "m": 1, "v": 131072, "x": "f32", "out": "f32",
         "history": 2048, "biases": 16, "mask": True},
        # decoding sequences with long histories
        {"name": "logits batch", "op": "logits", "m": 64, "v": 131072, "x": "bf16", "out": "f32",
         "history": 8192, "biases": 300, "mask": True},
        # an odd vocabulary and count of sequences, no grammar
        {"name": "logits ragged", "op": "logits", "m": 37, "v": 32003, "x": "f16", "out": "f16",
         "history": 777, "biases": 0, "mask": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rows", "quantize", "product", "product", "logits"])
    k = 128 * _log(rng, 1, 136)
    if op == "rows":
        n = min(_log(rng, 64, 131072), LARGEST_WEIGHT // k)
        c = {"op": op, "form": rng.choice(["q4", "f8"]), "m": min(_log(rng, 1, 4096), LARGEST_ROWS // k),
             "n": n, "k": k, "out": rng.choice(["f16", "bf16", "f32"])}
        if c["out"] == "f32":
            c["m"] = max(1, c["m"] // 2)
        if c["form"] == "q4":
            c["group"] = rng.choice([32, 64, 128])
        return c
    if op == "quantize":
        return {"op": op, "m": min(_log(rng, 1, 65536), LARGEST_QUANTIZE // k), "k": k,
                "x": rng.choice(["f32", "f16", "bf16"])}
    if op == "product":
        m = _log(rng, 1, 4096)
        n = min(_log(rng, 16, 131072), LARGEST_WEIGHT // k, LARGEST_PRODUCT // (m * k))
        if m * n > 4096 * 17408:
            n = 4096 * 17408 // m
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["f32", "f16", "bf16"])}
    v = _log(rng, 1000, 262144)
    m = min(_log(rng, 1, 256), max(1, LARGEST_LOGITS // v))
    return {"op": op, "m": m, "v": v, "x": rng.choice(["f32", "f16", "bf16"]),
            "out": rng.choice(["f32", "f32", "f16", "bf16"]),
            "history": rng.choice([0, _log(rng, 1, 8192), _log(rng, 1, 8192)]),
            "biases": rng.choice([0, _log(rng, 1, 512)]), "mask": rng.random() < 0.6}


def work(case):
    op, m = case["op"], case["m"]
    if op == "logits":
        v = case["v"]
        moved = m * v * (BYTES[case["x"]] + BYTES[case["out"]]) + 4 * m * case["history"] + 20 * m
        moved += 8 * m * case["biases"] + (m * ((v + 31) // 32) * 4 if case["mask"] else 0)
        return {"bytes": moved, "flops": 6 * m * v}
    k = case["k"]
    if op == "rows":
        row = k + k // 128 if case["form"] == "f8" else k // 2 + 2 * (k // case["group"])
        distinct = min(m, case["n"])
        return {"bytes": distinct * row + 4 * m + m * k * BYTES[case["out"]], "flops": 2 * m * k}
    if op == "quantize":    # codes and scales are written by one call and read by the other
        return {"bytes": m * k * (BYTES[case["x"]] + 2) + 2 * m * (k + k // 128), "flops": 4 * m * k}
    n = case["n"]
    return {"bytes": (m + n) * (k + k // 128) + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}


# ---------------------------------------------------------------- inputs

def _activations(g, m, k):
    """N(0, 1) with one element in a hundred twenty times larger."""
    x = torch.randn(m, k, generator=g, device=DEVICE)
    big = torch.rand(m, k, generator=g, device=DEVICE) < 0.01
    return torch.where(big, 20 * x, x)


def _power(e):
    """float32 powers of two, by their bits (pow need not be exact); 0 for -127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_quantize(x):
    """e4m3 codes of float32 rows and the biased exponents of their blocks' scales:
    the smallest power of two under which the block's largest is at most 448."""
    m, k = x.shape
    b = x.view(m, k // 128, 128)
    f, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(f <= 0.875, p - 9, p - 8)
    e = torch.where(f == 0, -127, e).clamp(-127, 127)
    c = (b * _power(-e).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return c.view(m, k), (e + 127).to(torch.uint8)


def _quantized(g, n, k, spread):
    """Random rows in 8-bit form, made a piece at a time."""
    codes = torch.empty(n, k, dtype=torch.float8_e4m3fn, device=DEVICE)
    scales = torch.empty(n, k // 128, dtype=torch.uint8, device=DEVICE)
    rows = max(1, (1 << 27) // k)
    for i in range(0, n, rows):
        r = min(rows, n - i)
        x = _activations(g, r, k) if spread is None else spread * torch.randn(r, k, generator=g, device=DEVICE)
        codes[i:i + r], scales[i:i + r] = _plain_quantize(x)
    return codes, scales.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    st = dict(case)
    op, m = case["op"], case["m"]

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEVICE, dtype=torch.int32)

    if op == "rows":
        n, k = case["n"], case["k"]
        if case["form"] == "f8":
            st["codes"], st["scales"] = _quantized(g, n, k, 0.02)
        else:
            st["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEVICE, dtype=torch.uint8)
            s = torch.rand(n, k // case["group"], generator=g, device=DEVICE).mul_(0.008).add_(0.004)
            st["scales"] = s.to(torch.float16)
        # frequent tokens have low ids; a padded end where there is room for one
        u = torch.rand(m, generator=g, device=DEVICE)
        st["ids"] = (n * u ** 3).long().clamp(0, n - 1).to(torch.int32)
        if m >= 32:
            st["ids"][m - m // 16:] = -1
        st["factor"] = math.sqrt(k)
        st["y"] = torch.empty(m, k, dtype=DTYPES[case["out"]], device=DEVICE)
        return st
    if op == "quantize":
        k = case["k"]
        x = 0.02 * torch.randn(m, k, generator=g, device=DEVICE) if m > 4096 else _activations(g, m, k)
        st["x"] = x.to(DTYPES[case["x"]])
        st["codes"] = torch.empty(m, k, dtype=torch.float8_e4m3fn, device=DEVICE)
        st["scales"] = torch.empty(m, k // 128, dtype=torch.float8_e8m0fnu, device=DEVICE)
        st["back"] = torch.empty(m, k, dtype=torch.bfloat16, device=DEVICE)
        return st
    if op == "product":
        n, k = case["n"], case["k"]
        st["codes"], st["scales"] = _quantized(g, n, k, 0.02)
        st["xq"], st["xs"] = _quantized(g, m, k, None)
        st["y"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device=DEVICE)
        return st
    v, h, b = case["v"], case["history"], case["biases"]
    st["logits"] = (3 * torch.randn(m, v, generator=g, device=DEVICE)).to(DTYPES[case["x"]])
    for name in ("history_ids", "history_lens", "prompt_lens", "repetition", "presence", "frequency",
                 "bias_ids", "bias_values", "mask_words"):
        st[name] = None
    if h:
        u = torch.rand(m, h, generator=g, device=DEVICE)
        st["history_ids"] = (v * u ** 4).long().clamp(0, v - 1).to(torch.int32)
        st["history_lens"] = ints(h // 2, h + 1, m)
        st["history_lens"][0] = h
        st["prompt_lens"] = ints(0, h // 2 + 1, m)
        if m > 2:
            st["history_lens"][2] = 0
        st["repetition"] = 1 + 0.3 * torch.rand(m, generator=g, device=DEVICE)
        st["presence"] = 0.5 * torch.rand(m, generator=g, device=DEVICE)
        st["frequency"] = 0.1 * torch.rand(m, generator=g, device=DEVICE)
    if b:       # fewer than the width in some rows: the rest is padded
        st["bias_ids"] = ints(0, v, m, b)
        st["bias_ids"][m // 2, b // 2:] = -1
        st["bias_values"] = 5 * torch.randn(m, b, generator=g, device=DEVICE)
    if case["mask"]:   # a grammar allows little, but every other row nearly all
        words = torch.randint(-2 ** 31, 2 ** 31, (3, m, (v + 31) // 32), generator=g, device=DEVICE)
        tight, loose = words[0] & words[1] & words[2], words[0] | words[1] | words[2]
        tight[::2] = loose[::2]
        st["mask_words"] = tight.to(torch.int32)
    st["y"] = torch.empty(m, v, dtype=DTYPES[case["out"]], device=DEVICE)
    return st


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import tl_hadamard_rotate_amd as tl
    op = st["op"]
    if op == "rows":
        call = tl.q4_rows if st["form"] == "q4" else tl.f8_rows
        return call(st["codes"], st["scales"], st["ids"], st["factor"], out_dtype=st["y"].dtype, out=st["y"])
    if op == "quantize":
        tl.f8_quantize(st["x"], codes=st["codes"], scales=st["scales"])
        return tl.f8_dequantize(st["codes"], st["scales"], out_dtype=torch.bfloat16, out=st["back"])
    if op == "product":
        return tl.f8_gemm(st["codes"], st["scales"], st["xq"], st["xs"], out_dtype=st["y"].dtype, out=st["y"])
    return tl.adjust_logits(st["logits"], history=st["history_ids"], history_lens=st["history_lens"],
                            prompt_lens=st["prompt_lens"], repetition=st["repetition"],
                            presence=st["presence"], frequency=st["frequency"],
                            bias_ids=st["bias_ids"], bias_values=st["bias_values"],
                            mask=st["mask_words"], out_dtype=st["y"].dtype, out=st["y"])


# ---------------------------------------------------------------- the plain forms

def _plain_values(codes, scales):
    """float32 values of rows in 8-bit form."""
    n, k = codes.shape
    e = scales.view(torch.uint8).to(torch.int32) - 127
    return (codes.float().view(n, k // 128, 128) * _power(e).unsqueeze(-1)).view(n, k)


def _plain_q4_values(packed, scales):
    """float32 values of packed 4-bit weights: of the 8 weights k0 .. k7 of a
    32-bit word, the even ones lie in its low half, the odd ones in its high half."""
    n, groups = scales.shape
    shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=packed.device)
    nibbles = (packed.view(torch.int32).unsqueeze(-1) >> shifts) & 15
    codes = ((nibbles ^ 8) - 8).float().view(n, groups, -1)
    return (codes * scales.float().unsqueeze(-1)).view(n, -1)


def run(state):
    if own:
        return _own(state)
    st = state
    op, m = st["op"], st["m"]
    if op == "rows":
        n = st["codes"].shape[0]
        known = (st["ids"] >= 0) & (st["ids"] < n)
        at = torch.where(known, st["ids"], 0).long()
        values = _plain_q4_values if st["form"] == "q4" else _plain_values
        codes = st["codes"] if st["form"] == "q4" else st["codes"].view(torch.uint8)
        scales = st["scales"] if st["form"] == "q4" else st["scales"].view(torch.uint8)
        codes, scales = codes[at], scales[at]
        if st["form"] == "f8":
            codes = codes.view(torch.float8_e4m3fn)
        return torch.where(known[:, None], values(codes, scales) * st["factor"], 0.0).to(st["y"].dtype)
    if op == "quantize":
        return _plain_values(*_plain_quantize(st["x"].float())).to(torch.bfloat16)
    if op == "product":
        y = torch.empty_like(st["y"])
        x = _plain_values(st["xq"], st["xs"])
        n, k = st["codes"].shape
        rows = max(1, (1 << 28) // k)
        for i in range(0, n, rows):
            y[:, i:i + rows] = (x @ _plain_values(st["codes"][i:i + rows], st["scales"][i:i + rows]).t()).to(y.dtype)
        return y
    v = st["v"]
    x = st["logits"].float()
    if st["history_ids"] is not None:
        ids, h = st["history_ids"].long(), st["history"]
        at = torch.arange(h, device=ids.device)[None]
        told = at < st["history_lens"][:, None]
        answered = told & (at >= st["prompt_lens"][:, None])
        count = torch.zeros(2, m, v, device=ids.device)
        count[0].scatter_add_(1, ids, told.float())
        count[1].scatter_add_(1, ids, answered.float())
        r = st["repetition"][:, None]
        x = torch.where(count[0] > 0, torch.where(x > 0, x / r, x * r), x)
        x = x - st["frequency"][:, None] * count[1] - st["presence"][:, None] * (count[1] > 0)
    if st["bias_ids"] is not None:      # of a token named twice the last value counts
        ids = st["bias_ids"].long()
        place = torch.arange(1, ids.shape[1] + 1, device=ids.device).expand(m, -1)
        last = torch.zeros(m, v, dtype=torch.long, device=ids.device)
        last.scatter_reduce_(1, ids.clamp(min=0), torch.where(ids >= 0, place, 0), "amax")
        value = st["bias_values"].gather(1, (last - 1).clamp(min=0))
        x = x + torch.where(last > 0, value, 0.0)
    if st["mask_words"] is not None:
        bits = (st["mask_words"][..., None] >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1
        x = torch.where(bits.view(m, -1)[:, :v] != 0, x, -math.inf)
    return x.to(st["y"].dtype)


# ---------------------------------------------------------------- the definition, in 64 bits

def _two(e):
    return ((e.long() + 1023) * 2 ** 52).view(torch.float64)


def _exact_values(codes, scales):
    b = codes.view(torch.uint8).to(torch.int64)
    mantissa, e = b % 8, b // 8 % 16
    v = torch.where(e > 0, (8 + mantissa) * _two(e - 10), mantissa * 2.0 ** -9)
    v = torch.where(b >= 128, -v, v)
    return v * torch.repeat_interleave(_two(scales.view(torch.uint8).long() - 127), 128, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "rows":
        y = torch.zeros(m, case["k"], dtype=torch.float64, device=DEVICE)
        codes = st["codes"].view(torch.uint8)
        scales = st["scales"] if case["form"] == "q4" else st["scales"].view(torch.uint8)
        for i in range(0, m, 512):
            ids = st["ids"][i:i + 512].long()
            there = (ids >= 0).nonzero().flatten()
            c, s = codes[ids[there]], scales[ids[there]]
            if case["form"] == "f8":
                w = _exact_values(c, s)
            else:
                b = c.to(torch.int16).reshape(len(there), -1, 4)
                w = torch.empty(*b.shape[:2], 8, dtype=torch.float64, device=DEVICE)
                for j, at in enumerate((0, 4, 1, 5)):    # byte j holds two weights of one parity
                    w[..., at] = (b[..., j] % 16 + 8) % 16 - 8.0
                    w[..., at + 2] = (b[..., j] // 16 + 8) % 16 - 8.0
                w = w.reshape(len(there), -1) * torch.repeat_interleave(s.double(), case["group"], dim=1)
            y[i + there] = w * case["k"] ** 0.5
        return y
    if op == "quantize":
        x = st["x"].double().reshape(-1, 128)
        top = x.abs().max(-1, keepdim=True).values
        e = torch.ceil(torch.log2(top / 448))
        e = torch.where(_two(e) * 448 < top, e + 1, e)
        e = torch.where(_two(e - 1) * 448 >= top, e - 1, e)
        v = x / _two(e)
        step = torch.full_like(v, 2.0 ** -9)
        for i in range(-5, 9):      # steps of the values from 2^i up
            step = torch.where(v.abs() >= 2.0 ** i, 2.0 ** (i - 3), step)
        lower = torch.floor(v / step)
        rest = v / step - lower
        up = (rest > 0.5) | ((rest == 0.5) & (lower % 2 != 0))
        return ((lower + up) * step * _two(e)).reshape(st["x"].shape)
    if op == "product":
        n, k = case["n"], case["k"]
        x = _exact_values(st["xq"], st["xs"])
        y = torch.empty(m, n, dtype=torch.float64, device=DEVICE)
        rows = max(16, (1 << 26) // k)
        for i in range(0, n, rows):
            y[:, i:i + rows] = x @ _exact_values(st["codes"][i:i + rows], st["scales"][i:i + rows]).t()
        return y
    v = case["v"]
    y = st["logits"].double()
    for i in range(m):
        if case["history"]:
            told = st["history_ids"][i, :st["history_lens"][i]]
            seen = told.unique().long()
            r = st["repetition"][i].double()
            y[i, seen] = torch.where(y[i, seen] > 0, y[i, seen] / r, y[i, seen] * r)
            ids, n = told[st["prompt_lens"][i]:].unique(return_counts=True)
            y[i, ids.long()] -= n * st["frequency"][i].double() + st["presence"][i].double()
        if case["biases"]:
            named = {t: b for t, b in zip(st["bias_ids"][i].tolist(), st["bias_values"][i].tolist()) if t >= 0}
            if named:
                ids = torch.tensor(list(named), device=DEVICE)
                y[i, ids] += torch.tensor(list(named.values()), dtype=torch.float64, device=DEVICE)
        if case["mask"]:
            words = st["mask_words"][i].long()
            allowed = torch.stack([words // 2 ** j % 2 for j in range(32)], 1).flatten()[:v]
            y[i][allowed == 0] = -math.inf
    return y

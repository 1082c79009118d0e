"""The operators around the ternary linear layer, as cases to time and compare.

Three operators, and the chain of the first two:

  norm   ``rms_norm``: residual addition, root-mean-square norm and gain, with
         the signed 1024-block Hadamard rotation of the following ternary
         linear as an option
  q4     ``q4_gemv``: product with 4-bit weights and group scales, from
         binary16 or bfloat16 activations
  chain  ``rms_norm_i8`` then ``q4_gemv``: the norm writes 8-bit activations
         with a scale per 128, the product reads them
  round  ``q4_quantize`` then ``q4_dequantize``: weight rows to 4-bit codes and
         scales, and back to the values these stand for

Shapes are those of the library's benchmark (K = 5120 and 17408 inputs; q, k/v,
gate/up and down projections) and generic vocabularies and odd sizes.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}
EPS = 1e-6
LARGEST_WEIGHT = 131072 * 5120      # the listed head
LARGEST_ROUND = 17408 * 5120        # the listed projection to quantise
LARGEST_NORM = 4096 * 5120          # the listed prompt


def listed():
    return [
        # one new token before a block's rotated projections: latency counts
        {"name": "norm token rotated", "op": "norm", "m": 1, "k": 5120, "x": "f16", "out": "f16",
         "res": True, "rot": True},
        # a batch of decoding sequences, wide rows of the down projection, odd count, fp32 stream
        {"name": "norm batch wide f32", "op": "norm", "m": 37, "k": 17408, "x": "f32", "out": "f16",
         "res": False, "rot": True},
        # a whole prompt in the bfloat16 stream, before linears without a rotation
        {"name": "norm prompt bf16", "op": "norm", "m": 4096, "k": 5120, "x": "bf16", "out": "bf16",
         "res": True, "rot": False},
        # a prompt before ternary linears
        {"name": "norm prompt rotated", "op": "norm", "m": 2048, "k": 5120, "x": "f16", "out": "f16",
         "res": True, "rot": True},
        # k/v projection of one token: the smallest product
        {"name": "q4 token kv", "op": "q4", "m": 1, "n": 1024, "k": 5120, "x": "f16", "out": "f32",
         "group": 128},
        # the head of one token
        {"name": "q4 token head", "op": "q4", "m": 1, "n": 131072, "k": 5120, "x": "f16", "out": "f32",
         "group": 128},
        # down projection of eight sequences, bfloat16 activations
        {"name": "q4 batch down bf16", "op": "q4", "m": 8, "n": 5120, "k": 17408, "x": "bf16",
         "out": "f32", "group": 64},
        # a vocabulary that divides by nothing, many sequences, short groups
        {"name": "q4 batch ragged head", "op": "q4", "m": 45, "n": 32003, "k": 5120, "x": "f16",
         "out": "f16", "group": 32},
        # norm and q projection of one token through 8-bit activations
        {"name": "chain token q", "op": "chain", "m": 1, "n": 6144, "k": 5120, "x": "f16", "out": "f16",
         "group": 128, "rot": True},
        # norm and gate/up of sixteen sequences through 8-bit activations
        {"name": "chain batch gate", "op": "chain", "m": 16, "n": 17408, "k": 5120, "x": "bf16",
         "out": "f16", "group": 128, "rot": False},
        # quantising one projection, and a small odd one with short groups
        {"name": "round gate", "op": "round", "n": 17408, "k": 5120, "w": "f32", "group": 128},
        {"name": "round small odd", "op": "round", "n": 1001, "k": 1152, "w": "bf16", "group": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "q4", "chain", "round"])
    if op == "norm":
        rot = rng.random() < 0.5
        k = 1024 * _log(rng, 1, 17) if rot else 8 * _log(rng, 1, 2176)
        m = min(_log(rng, 1, 4096), LARGEST_NORM // k)
        x = rng.choice(["f16", "bf16", "f32"])
        out = rng.choice(["f16", "bf16", "f32"])
        if x == "f32" or out == "f32":
            m = min(m, LARGEST_NORM // k // 2)
        return {"op": op, "m": max(1, m), "k": k, "x": x, "out": out, "res": rng.random() < 0.7,
                "rot": rot}
    if op == "round":
        k = 128 * _log(rng, 1, 136)
        return {"op": op, "n": min(_log(rng, 8, 65536), LARGEST_ROUND // k), "k": k,
                "w": rng.choice(["f32", "f16", "bf16"]), "group": rng.choice([32, 64, 128])}
    m = _log(rng, 1, 64)
    rot = op == "chain" and rng.random() < 0.5
    k = 1024 * _log(rng, 1, 17) if rot else 128 * _log(rng, 1, 136)
    n = min(_log(rng, 16, 131072), LARGEST_WEIGHT // k // (1 + m // 8))
    c = {"op": op, "m": m, "n": n, "k": k, "x": rng.choice(["f16", "bf16"]),
         "out": "f16" if op == "chain" else rng.choice(["f32", "f16"]),
         "group": rng.choice([32, 64, 128])}
    if op == "chain":
        c["rot"] = rot
    return c


def work(case):
    op = case["op"]
    if op == "round":
        n, k = case["n"], case["k"]
        packed = n * k // 2 + 2 * n * (k // case["group"])
        return {"bytes": n * k * (BYTES[case["w"]] + 2) + 2 * packed, "flops": 6 * n * k}
    m, k, e = case["m"], case["k"], BYTES[case["x"]]
    norm = k * e + (k if case.get("rot") else 0)
    flops = m * k * (26 if case.get("rot") else 6)
    if op == "norm":
        moved = m * k * (e * (3 if case["res"] else 1) + BYTES[case["out"]])
        return {"bytes": moved + norm, "flops": flops}
    n = case["n"]
    product = n * k // 2 + 2 * n * (k // case["group"]) + m * n * BYTES[case["out"]]
    if op == "q4":
        return {"bytes": product + m * k * e, "flops": 2 * m * n * k}
    return {"bytes": product + 3 * m * k * e + norm, "flops": 2 * m * n * k + flops}


# ---------------------------------------------------------------- inputs

def _hadamard(dtype):
    """Sylvester's matrix over 32: the sign of (i, j) is the parity of i & j."""
    i = torch.arange(1024, device=DEVICE)
    bits = ((i[:, None] >> torch.arange(10, device=DEVICE)) & 1).to(dtype)
    return (1 - 2 * torch.remainder(bits @ bits.t(), 2)) / 32


def _activations(g, m, k, dtype):
    """N(0, 1) with one element in a hundred twenty times larger."""
    x = torch.randn(m, k, generator=g, device=DEVICE)
    big = torch.rand(m, k, generator=g, device=DEVICE) < 0.01
    return torch.where(big, 20 * x, x).to(dtype)


def _packed(codes):
    """4-bit codes, packed: of the 8 weights k0 .. k7 of a 32-bit word, the even
    ones in its low half and the odd ones in its high half, first lowest."""
    n, k = codes.shape
    c = codes.view(n, k // 8, 8) & 15
    b = c[..., [0, 4, 1, 5]] | c[..., [2, 6, 3, 7]] << 4
    return b.view(torch.uint8).reshape(n, k // 2)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op == "round":
        w = torch.randn(case["n"], case["k"], generator=g, device=DEVICE).mul_(0.02)
        st["w"] = w.to(DTYPES[case["w"]])
        st["packed"] = torch.empty(case["n"], case["k"] // 2, dtype=torch.uint8, device=DEVICE)
        st["scales"] = torch.empty(case["n"], case["k"] // case["group"], dtype=torch.float16,
                                   device=DEVICE)
        st["back"] = torch.empty(case["n"], case["k"], dtype=torch.float16, device=DEVICE)
        return st
    m, k, dtype = case["m"], case["k"], DTYPES[case["x"]]
    st["x"] = _activations(g, m, k, dtype)
    if op != "q4":
        st["gain"] = (1 + 0.1 * torch.randn(k, generator=g, device=DEVICE)).to(dtype)
        st["residual"] = st["sum"] = st["signs"] = st["hadamard"] = None
        if op == "chain" or case["res"]:
            st["residual"] = (3 * torch.randn(m, k, generator=g, device=DEVICE)).to(dtype)
            st["sum"] = torch.empty(m, k, dtype=dtype, device=DEVICE)
        if case["rot"]:
            bits = torch.randint(0, 2, (k,), generator=g, device=DEVICE)
            st["signs"] = (2 * bits - 1).to(torch.int8)
            st["hadamard"] = _hadamard(torch.float64 if op == "chain" else torch.float32)
    if op == "norm":
        st["y"] = torch.empty(m, k, dtype=DTYPES[case["out"]], device=DEVICE)
        return st
    if op == "chain":
        st["q"] = torch.empty(m, k, dtype=torch.int8, device=DEVICE)
        st["q_scales"] = torch.empty(m, k // 128, dtype=torch.float32, device=DEVICE)
    # codes of normally distributed weights, the largest of a group near the
    # end of the range
    n = case["n"]
    st["packed"] = torch.empty(n, k // 2, dtype=torch.uint8, device=DEVICE)
    for i in range(0, n, 16384):
        c = torch.randn(min(16384, n - i), k, generator=g, device=DEVICE).mul_(2.6)
        st["packed"][i:i + 16384] = _packed(c.round_().clamp_(-8, 7).to(torch.int8))
    s = torch.rand(n, k // case["group"], generator=g, device=DEVICE).mul_(0.008).add_(0.004)
    st["scales"] = s.to(torch.float16)
    st["y"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device=DEVICE)
    return st


# ---------------------------------------------------------------- the framework's calls

def _own(st):
    import tl_hadamard_rotate_amd as tl
    op = st["op"]
    if op == "norm":
        tl.rms_norm(st["x"], st["gain"], EPS, residual=st["residual"], signs=st["signs"],
                    out_dtype=st["y"].dtype, sum_out=st["sum"], out=st["y"])
        return st["y"] if st["sum"] is None else (st["y"], st["sum"])
    if op == "q4":
        return tl.q4_gemv(st["packed"], st["scales"], st["x"], out_dtype=st["y"].dtype, out=st["y"])
    if op == "chain":
        tl.rms_norm_i8(st["x"], st["gain"], EPS, residual=st["residual"], signs=st["signs"],
                       sum_out=st["sum"], out=st["q"], scales=st["q_scales"])
        tl.q4_gemv(st["packed"], st["scales"], st["q"], x_scales=st["q_scales"],
                   out_dtype=st["y"].dtype, out=st["y"])
        return st["y"], st["sum"]
    tl.q4_quantize(st["w"], st["group"], packed=st["packed"], scales=st["scales"])
    return tl.q4_dequantize(st["packed"], st["scales"], out_dtype=torch.float16, out=st["back"])


# ---------------------------------------------------------------- the plain forms

def _plain_norm(st, wide):
    """(the residual sum in the stream's type, the normalised and perhaps
    rotated rows in `wide` bits)."""
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(h.dtype)
    f = h.to(wide)
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * st["gain"].to(wide)
    if st["signs"] is not None:
        m, k = y.shape
        y = ((y * st["signs"].to(wide)).view(m * (k // 1024), 1024) @ st["hadamard"]).view(m, k)
    return h, y


def _plain_values(packed, scales):
    """float32 values of packed 4-bit weights."""
    n, groups = scales.shape
    shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=packed.device)
    nibbles = (packed.view(torch.int32).unsqueeze(-1) >> shifts) & 15
    codes = ((nibbles ^ 8) - 8).float().view(n, groups, -1)
    return (codes * scales.float().unsqueeze(-1)).view(n, -1)


def run(state):
    if own:
        return _own(state)
    st = state
    op = st["op"]
    if op == "norm":
        h, y = _plain_norm(st, torch.float32)
        y = y.to(st["y"].dtype)
        return y if st["residual"] is None else (y, h)
    if op == "q4":
        w = _plain_values(st["packed"], st["scales"])
        return (st["x"].float() @ w.t()).to(st["y"].dtype)
    if op == "chain":
        h, y = _plain_norm(st, torch.float64)     # codes are decided at borders
        y = y.view(y.shape[0], -1, 128)
        top = y.abs().amax(-1, keepdim=True)
        q = torch.round(127 * y / top)
        a = (q.float() * (top / 127).float()).view(h.shape)
        w = _plain_values(st["packed"], st["scales"])
        return (a @ w.t()).to(st["y"].dtype), h
    n, k = st["w"].shape
    w = st["w"].double().view(n, -1, st["group"])
    s = (w.abs().amax(-1, keepdim=True) / 7).to(torch.float16)
    c = torch.round(w / s.double()).clamp(-8, 7).to(torch.int8)
    c = torch.where(s == 0, torch.zeros_like(c), c)
    return (c.float() * s.float()).to(torch.float16).view(n, k)


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "round":
        w = st["w"].double().reshape(-1, case["group"])
        top = w.abs().max(-1).values
        s = (top / 7).to(torch.float16).double().unsqueeze(-1)
        v = w / torch.where(s > 0, s, torch.ones_like(s))
        c = torch.floor(v + 0.5)
        c = torch.where((v + 0.5 == c) & (c % 2 != 0), c - 1, c)
        return (torch.clamp(c, min=-8, max=7) * s).reshape(st["w"].shape)
    m, k = case["m"], case["k"]
    a = st["x"].double()
    h = a
    if op != "q4":
        if st["residual"] is not None:
            h = (a + st["residual"].double()).to(st["x"].dtype).double()
        a = h / ((h ** 2).sum(1, keepdim=True) / k + EPS) ** 0.5 * st["gain"].double()
        if case["rot"]:     # Sylvester's recursion: sums and differences of the halves, the quarters, ...
            a = a * st["signs"].double()
            half = 512
            while half:
                a = a.reshape(-1, 512 // half, 2, half)
                a = torch.stack((a[:, :, 0] + a[:, :, 1], a[:, :, 0] - a[:, :, 1]), 2)
                half //= 2
            a = a.reshape(m, k) / 32
    if op == "norm":
        return a if st["residual"] is None else (a, h)
    if op == "chain":
        g = a.reshape(-1, 128)
        step = g.abs().max(-1, keepdim=True).values / 127
        a = (torch.round(g / step) * step).reshape(m, k)
    n = case["n"]
    y = torch.empty(m, n, dtype=torch.float64, device=a.device)
    rows = max(16, (1 << 27) // k)
    for i in range(0, n, rows):
        b = st["packed"][i:i + rows].to(torch.int16).reshape(-1, k // 8, 4)
        w = torch.empty(*b.shape[:2], 8, dtype=torch.float64, device=a.device)
        for j, at in enumerate((0, 4, 1, 5)):    # byte j holds two weights of one parity
            w[..., at] = (b[..., j] % 16 + 8) % 16 - 8.0
            w[..., at + 2] = (b[..., j] // 16 + 8) % 16 - 8.0
        w = w.reshape(-1, k // case["group"], case["group"]) * st["scales"][i:i + rows].double().unsqueeze(-1)
        y[:, i:i + rows] = a @ w.reshape(-1, k).t()
    return y if op == "q4" else (y, h)

"""Cases and plain forms of the operators around the quantized product.

Three operators, as a W8A8 decoder block runs them one after the other:

  quant_matmul            y = (x_codes . w_codes^T) * scale_x * scale_w + bias, the sum exact
  post_norm_add_rms_norm_dynamic_quant
                          p  = h / Rms(h) * gamma_post
                          x' = round16(x + residual_scale * gate * p)
                          in = (x' / Rms(x') * gamma + beta) * smooth
                          scale = rowmax|in| / Q, codes = round(in / scale); or round16(in), no codes
  glu_dynamic_quant       in = act(x[:, :n]) * x[:, n:] * smooth, then scale and codes as above

``run`` computes the plain form (elementary torch operations) or, where ``own`` is true, calls the
library.  Codes come back as the values they stand for, codes * scale, in the inputs' type.  The
plain forms of the two quantizing operators are in 64 bits: every output of theirs is the side of
a rounding border (16 bits, 8 bits, 4 bits) that a value falls on.  The plain product is in 64 bits
because its sums pass 2^24.
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_Q = {"int8": 127.0, "int4": 7.0}
_EPS = 1e-6


def listed():
    """The listed cases; the comment of each says what it stands for."""
    return [
        # one token through a square projection: the latency of a decode step
        dict(name="matmul_1x4096x4096", op="matmul", m=1, n=4096, k=4096, out="bf16", bias=False),
        # a decode batch through the wide projection of an MLP: the weights' bytes
        dict(name="matmul_16x16384x4096", op="matmul", m=16, n=16384, k=4096, out="bf16", bias=False),
        # a ragged chunk of a prompt, with bias, in half precision
        dict(name="matmul_333x5120x7168_bias", op="matmul", m=333, n=5120, k=7168, out="fp16", bias=True),
        # sizes that are multiples of nothing
        dict(name="matmul_129x1023x1001", op="matmul", m=129, n=1023, k=1001, out="fp32", bias=True),
        # a prefill batch: bound by the tensor cores
        dict(name="matmul_8192x7168x4096", op="matmul", m=8192, n=7168, k=4096, out="bf16", bias=False),
        # a decode step's norms
        dict(name="norms_1x4096", op="norms", m=1, n=4096, dtype="bf16", q="int8", gate="channel",
             beta=False, smooth=True),
        # a prefill batch's norms, a gate for each channel
        dict(name="norms_8192x4096", op="norms", m=8192, n=4096, dtype="bf16", q="int8",
             gate="channel", beta=False, smooth=True),
        # a gate for each sequence (conditioned blocks), a 16-bit result for an unquantized layer
        dict(name="norms_4096x7168_16bit", op="norms", m=4096, n=7168, dtype="bf16", q="none",
             gate="sequence", beta=True, smooth=False),
        # packed INT4, no gate
        dict(name="norms_1000x5120_int4", op="norms", m=1000, n=5120, dtype="fp16", q="int4",
             gate="none", beta=False, smooth=False),
        # a decode step's activation
        dict(name="glu_8x16384", op="glu", m=8, n=16384, dtype="bf16", q="int8", act="silu", smooth=True),
        # a prefill batch's activation
        dict(name="glu_4096x16384", op="glu", m=4096, n=16384, dtype="bf16", q="int8", act="silu",
             smooth=True),
        # a row length that 16-byte loads do not divide
        dict(name="glu_777x5001_gelu", op="glu", m=777, n=5001, dtype="fp16", q="int8", act="gelu_tanh",
             smooth=False),
    ]


def _log_size(rng, lo, hi):
    """A size spread over its logarithm; a third of them rounded to 128, the rest as they come."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 256 and rng.random() < 0.34:
        v = (v + 64) // 128 * 128
    return max(lo, min(hi, v))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["matmul", "norms", "glu"])
    if op == "matmul":
        while True:
            m, n, k = _log_size(rng, 1, 8192), _log_size(rng, 256, 16384), _log_size(rng, 256, 16384)
            if rng.random() < 0.7:  # weights of real layers are multiples of 16
                n, k = (n + 15) // 16 * 16, (k + 15) // 16 * 16
            if m * n * k <= 8192 * 7168 * 4096 and n * k <= 16384 * 8192:
                break
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "fp16", "fp32"]),
                    bias=rng.random() < 0.5)
    cap = 8192 * 4096 if op == "norms" else 4096 * 16384
    while True:
        m, n = _log_size(rng, 1, 8192), _log_size(rng, 256, 16384)
        if rng.random() < 0.7:
            n = (n + 7) // 8 * 8
        if m * n <= cap:
            break
    dtype = rng.choice(["bf16", "fp16"])
    if op == "glu":
        return dict(op=op, m=m, n=n, dtype=dtype, q="int8" if n % 2 else rng.choice(["int8", "int4"]),
                    act=rng.choice(["silu", "gelu_tanh"]), smooth=rng.random() < 0.5)
    return dict(op=op, m=m, n=n, dtype=dtype, q="int8" if n % 2 else rng.choice(["int8", "int4", "none"]),
                gate=rng.choice(["none", "channel", "sequence", "token"]), beta=rng.random() < 0.5,
                smooth=rng.random() < 0.5)


def _sequences(m):
    """Sequences of equal length in a batch of m tokens: 8, or the largest of 4, 2, 1 that divides it."""
    return next(s for s in (8, 4, 2, 1) if m % s == 0)


def prepare(case, seed):
    """Inputs on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case)
    m, n = case["m"], case["n"]
    if case["op"] == "matmul":
        k, t = case["k"], _T[case["out"]]
        # codes of a bell shape whose tails reach +-127, as rows scaled by their maximum have
        s["x"] = (normal(m, k) * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = (normal(n, k) * 36).round_().clamp_(-127, 127).to(torch.int8)
        s["sx"] = uniform(0.01, 0.05, m)
        s["sw"] = uniform(0.0002, 0.001, n)
        s["bias"] = normal(n).to(t) if case["bias"] else None
        return s
    t = _T[case["dtype"]]
    s["smooth"] = uniform(0.5, 2.0, n).to(t) if case["smooth"] else None
    if case["op"] == "glu":
        s["x"] = (normal(m, 2 * n) * 1.5).to(t)
        return s
    wide = torch.ones(n, device="cuda")
    wide[torch.randperm(n, generator=g, device="cuda")[: max(1, n // 100)]] = 20.0  # outlier channels
    s["h"] = (normal(m, n) * 0.7).to(t)
    s["x"] = (normal(m, n) * wide).to(t)
    s["gamma_post"] = uniform(0.5, 1.5, n).to(t)
    s["gamma"] = uniform(0.5, 1.5, n).to(t)
    s["beta"] = (normal(n) * 0.1).to(t) if case["beta"] else None
    rows = {"none": 0, "channel": 1, "sequence": _sequences(m), "token": m}[case["gate"]]
    s["gate"] = uniform(-0.5, 1.5, rows, n).to(t) if rows else None
    s["alpha"] = 0.25
    return s


def work(case):
    """Bytes and operations of one pass that no implementation avoids."""
    m, n = case["m"], case["n"]
    if case["op"] == "matmul":
        k, e = case["k"], 4 if case["out"] == "fp32" else 2
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * e + (n * e if case["bias"] else 0),
                "flops": 2 * m * n * k}
    code = {"int8": 1.0, "int4": 0.5, "none": 2.0}[case["q"]]
    scale = 0 if case["q"] == "none" else 4 * m
    if case["op"] == "glu":
        return {"bytes": m * n * (4 + code) + scale + (2 * n if case["smooth"] else 0), "flops": 12 * m * n}
    rows = {"none": 0, "channel": 1, "sequence": _sequences(m), "token": m}[case["gate"]]
    vectors = 2 + bool(case["beta"]) + bool(case["smooth"]) + rows
    return {"bytes": m * n * (6 + code) + scale + 2 * n * vectors, "flops": 16 * m * n}


# ------------------------------------------------------------------ plain forms

def _to16(v, t):
    """64 bits to 16 in one rounding: through 32 bits rounded to odd, so that no border is met twice."""
    f = v.float()
    bits = f.view(torch.int32) - (f.double().abs() > v.abs()).int()
    return (bits | (f.double() != v).int()).view(torch.float32).to(t)


def _quantize(v, q, t):
    """Rows of v (64 bits): the values that their codes stand for, and their scales."""
    scale = (v.abs().amax(-1, keepdim=True) / _Q[q]).float()
    codes = (v / torch.where(scale == 0, torch.ones_like(scale), scale)).round().clamp(-_Q[q], _Q[q])
    return (codes.float() * scale).to(t), scale.squeeze(-1)


def _plain(s):
    if s["op"] == "matmul":
        y = s["x"].double() @ s["w"].double().T
        y = y * s["sx"].double()[:, None] * s["sw"].double()
        if s["bias"] is not None:
            y = y + s["bias"].double()
        return y.to(_T[s["out"]])
    t, n = _T[s["dtype"]], s["n"]
    if s["op"] == "glu":
        a, u = s["x"][:, :n].double(), s["x"][:, n:].double()
        z = a if s["act"] == "silu" else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)
        v = a / (1 + torch.exp(-z)) * u
        if s["smooth"] is not None:
            v = v * s["smooth"].double()
        return _quantize(v, s["q"], t)
    h = s["h"].double()
    p = h / (h * h).mean(-1, keepdim=True).add(_EPS).sqrt() * s["gamma_post"].double()
    if s["gate"] is not None:
        p = (p.view(s["gate"].shape[0], -1, n) * s["gate"].double()[:, None]).view_as(p)
    x = _to16(s["x"].double() + s["alpha"] * p, t)
    v = x.double()
    v = v / (v * v).mean(-1, keepdim=True).add(_EPS).sqrt() * s["gamma"].double()
    if s["beta"] is not None:
        v = v + s["beta"].double()
    if s["smooth"] is not None:
        v = v * s["smooth"].double()
    if s["q"] == "none":
        return v.to(t), x
    return (*_quantize(v, s["q"], t), x)


# ------------------------------------------------------------------ the library's operators

def _values(y, scale, q, t):
    """What codes stand for: codes * scale (INT4: two codes a byte, the even column in the low nibble)."""
    if q == "int4":
        b = y.view(torch.int8)
        y = torch.stack(((b << 4) >> 4, b >> 4), -1).flatten(-2)
    return torch.mul(y, scale[:, None], out=torch.empty(y.shape, dtype=t, device=y.device))


def _own(s):
    import int4_quant_b200 as lib

    if s["op"] == "matmul":
        return lib.quant_matmul(s["x"], s["sx"], s["w"], s["sw"], s["bias"], out_dtype=_T[s["out"]])
    t = _T[s["dtype"]]
    if s["op"] == "glu":
        y, scale = lib.glu_dynamic_quant(s["x"], s["smooth"], activation=s["act"], qdtype=s["q"])
        return _values(y, scale, s["q"], t), scale
    y, scale, x = lib.post_norm_add_rms_norm_dynamic_quant(
        s["h"], s["x"], s["gamma_post"], s["gamma"], s["beta"], s["gate"], s["smooth"],
        residual_scale=s["alpha"], eps=_EPS, qdtype=None if s["q"] == "none" else s["q"])
    if s["q"] == "none":
        return y, x
    return _values(y, scale, s["q"], t), scale, x


def run(state):
    """One pass through the case's operator."""
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64-bit definitions

def _round16(v, t):
    """v rounded to the 16-bit type t: the type's cast, put right where a neighbour is nearer."""
    r = v.to(t)
    bits = r.view(torch.int16)
    best, err = r.double(), (r.double() - v).abs()
    for step in (-1, 1):
        c = (bits + step).view(t).double()
        nearer = (c - v).abs() < err
        best, err = torch.where(nearer, c, best), torch.where(nearer, (c - v).abs(), err)
    return best


def exact(case, seed):
    """The definition in 64 bits: norms by vector norms, the sigmoid by tanh, the product in pieces
    whose sums are whole numbers."""
    s = prepare(case, seed)
    m, n = case["m"], case["n"]
    d = lambda v: v.to(torch.float64)  # noqa: E731
    if case["op"] == "matmul":
        acc = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        for i in range(0, case["k"], 2048):
            acc += torch.einsum("mk,nk->mn", d(s["x"][:, i:i + 2048]), d(s["w"][:, i:i + 2048])).round()
        y = acc * torch.outer(d(s["sx"]), d(s["sw"]))
        return y if s["bias"] is None else y + d(s["bias"])

    def quantized(v):
        top = torch.maximum(v.max(-1).values, -v.min(-1).values)
        scale = (top / _Q[case["q"]]).float()
        step = d(scale)[:, None].clamp_min(torch.finfo(torch.float64).tiny)
        low = torch.floor(v / step)
        over = v - (low + 0.5) * step  # above, below or on the half-way point between two codes
        up = (over > 0) | ((over == 0) & (low.remainder(2) != 0))
        return (low + up) * d(scale)[:, None], d(scale)

    ones = torch.ones(n, dtype=torch.float64, device="cuda")
    smooth = ones if s["smooth"] is None else d(s["smooth"])
    if case["op"] == "glu":
        a, u = d(s["x"]).chunk(2, -1)
        z = a if case["act"] == "silu" else math.sqrt(8 / math.pi) * a * (1 + 0.044715 * a ** 2)
        return quantized(0.5 * a * (1 + torch.tanh(0.5 * z)) * u * smooth)

    def over_rms(v):
        return v * torch.rsqrt(torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / n + _EPS)

    gate = ones[None] if s["gate"] is None else d(s["gate"])
    gate = gate.repeat_interleave(m // gate.shape[0], 0)
    x = _round16(torch.addcmul(d(s["x"]), over_rms(d(s["h"])) * d(s["gamma_post"]), gate, value=s["alpha"]),
                 _T[case["dtype"]])
    v = (over_rms(x) * d(s["gamma"]) + (0 if s["beta"] is None else d(s["beta"]))) * smooth
    return (v, x) if case["q"] == "none" else (*quantized(v), x)

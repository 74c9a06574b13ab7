"""The fused norms and the gated activation, with their quantization, on a GPU
against plain 64-bit implementations (float64 torch on the CPU)."""
import pytest
import torch

import int4_quant_b200 as lib
from int4_quant_b200 import _abi as A
from int4_quant_b200 import build as B
from tests import _block_ref as R

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    A.lib()
    torch.cuda.set_device(0)


def shifted(t, offset):
    """A CUDA copy of t that starts `offset` elements into a larger buffer."""
    if t is None or offset == 0:
        return None if t is None else t.cuda()
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    buf[offset:].copy_(t.reshape(-1))
    return buf[offset:].view(t.shape)


def norms_case(rows, n, dtype="bf16", seed=0, gate_rows=0, beta=False, smooth=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = TDT[dtype]
    c = dict(h=(r(rows, n) * 0.7).to(t), x=(r(rows, n) * 1.5).to(t),
             gamma_post=(r(n) * 0.2 + 1).to(t), gamma=(r(n) * 0.2 + 1).to(t),
             beta=(r(n) * 0.1).to(t) if beta else None,
             smooth=(r(n).abs() + 0.5).to(t) if smooth else None,
             gate=(r(gate_rows, n) * 0.5 + 0.5).to(t) if gate_rows else None)
    return c


def run_norms(c, qdtype, alpha=0.25, eps=1e-6, offset=0, **kw):
    d = {k: shifted(v, offset) for k, v in c.items()}
    return lib.post_norm_add_rms_norm_dynamic_quant(
        d["h"], d["x"], d["gamma_post"], d["gamma"], d["beta"], d["gate"], d["smooth"],
        residual_scale=alpha, eps=eps, qdtype=qdtype, **kw)


def check_norms(c, got, qdtype, alpha=0.25, eps=1e-6, label=""):
    y, scale, x_out = got
    R.check_x(x_out, R.norms_x(c["h"], c["x"], c["gamma_post"], c["gate"], alpha, eps), label)
    v = R.norms_in(x_out.cpu(), c["gamma"], c["beta"], c["smooth"], eps)
    if qdtype is None:
        assert scale is None
        # one rounding to 16 bits (half a step) of a binary32 value a few 2^-24 off
        e = torch.finfo(y.dtype).eps / 2 * (1 + 2.0 ** -6)
        big = v.abs().amax(-1, keepdim=True)
        assert ((y.cpu().double() - v).abs() <= e * v.abs() + 2.0 ** -22 * big + 2.0 ** -24).all(), label
    else:
        R.check_codes(y, scale, v, qdtype, label)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("qdtype", ["int8", "int4", "int4_int32", None])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 64), (37, 264), (5, 4096), (2, 16384)])
def test_norms(rows, n, qdtype, dtype):
    c = norms_case(rows, n, dtype, seed=rows + n, gate_rows=1, smooth=True)
    check_norms(c, run_norms(c, qdtype), qdtype)


@pytest.mark.parametrize("rows,n", [(1, 1), (4, 2), (3, 7), (9, 1001), (2, 8190), (3, 16385)])
@pytest.mark.parametrize("qdtype", ["int8", None])
def test_norms_odd_lengths(rows, n, qdtype):
    c = norms_case(rows, n, seed=n, gate_rows=rows, beta=True, smooth=True)
    check_norms(c, run_norms(c, qdtype), qdtype)


@pytest.mark.parametrize("n", [16392, 32768, 131072, 40002])
@pytest.mark.parametrize("qdtype", ["int8", "int4", None])
def test_norms_long_rows(n, qdtype):
    c = norms_case(2, n, "fp16", seed=n, gate_rows=2, beta=True, smooth=True)
    check_norms(c, run_norms(c, qdtype), qdtype)


@pytest.mark.parametrize("gate_rows", [0, 1, 3, 12])
@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("smooth", [False, True])
def test_norms_optional_inputs(gate_rows, beta, smooth):
    c = norms_case(12, 520, seed=3, gate_rows=gate_rows, beta=beta, smooth=smooth)
    check_norms(c, run_norms(c, "int8"), "int8")


@pytest.mark.parametrize("offset", [1, 4])
def test_norms_misaligned(offset):
    c = norms_case(7, 512, seed=offset, gate_rows=1, beta=True)
    check_norms(c, run_norms(c, "int4", offset=offset), "int4")


@pytest.mark.parametrize("rows,n", [(2000, 1024), (1500, 4096), (600, 7168), (700, 1001)])
def test_norms_many_rows(rows, n):
    c = norms_case(rows, n, seed=rows, gate_rows=rows, smooth=True)
    check_norms(c, run_norms(c, "int8"), "int8")


@pytest.mark.parametrize("qdtype", ["int8", "int4", None])
@pytest.mark.parametrize("rows,n", [(300, 5002), (170, 258), (40, 9990)])
@pytest.mark.parametrize("offset", [0, 1])
def test_rows_of_pairs(rows, n, qdtype, offset):
    # even lengths that 16-byte loads do not divide, starting on and off 4-byte boundaries
    c = norms_case(rows, n, "fp16", seed=n, gate_rows=1, beta=True)
    check_norms(c, run_norms(c, qdtype, offset=offset), qdtype)
    if qdtype:
        x, s = glu_case(rows, n, seed=n, smooth=True)
        check_glu(x, s, "silu", qdtype, offset=offset)


@pytest.mark.parametrize("n", [520, 20000])
def test_norms_in_place(n):
    c = norms_case(6, n, seed=5, gate_rows=1)
    x = c["x"].cuda()
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    got = lib.post_norm_add_rms_norm_dynamic_quant(d["h"], x, d["gamma_post"], d["gamma"], None,
                                                   d["gate"], residual_scale=0.25, out={"x_out": x})
    assert got[2] is x
    check_norms(c, got, "int8")


@pytest.mark.parametrize("n", [520, 20000])
def test_norms_without_x_out(n):
    c = norms_case(6, n, seed=6, gate_rows=1)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    y = torch.empty(6, n, dtype=torch.int8, device="cuda")
    s = torch.empty(6, device="cuda")
    st = A.arnq_post_norm_add_rms_norm_dynamic_quant(
        d["h"], d["x"], d["gamma_post"], d["gate"], 1, 0.25, d["gamma"], None, None, 6, n,
        A.ARNQ_BF16, 1e-6, 1e-6, A.ARNQ_INT8, y, s, None, torch.cuda.current_stream())
    assert st == A.ARNQ_OK
    y2, s2, _ = run_norms(c, "int8")
    assert torch.equal(y, y2) and torch.equal(s, s2)


@pytest.mark.parametrize("qdtype", ["int8", "int4"])
@pytest.mark.parametrize("n", [256, 20000])
def test_norms_special_rows(qdtype, n):
    # zero rows, one with h alone zero, huge and tiny magnitudes, NaN, infinities
    c = norms_case(9, n, seed=8, gate_rows=1, smooth=True)
    c["h"][0] = 0
    c["x"][0] = 0
    c["h"][1] = 0
    c["h"][2] *= 1e30
    c["x"][3] *= 1e35
    c["h"][4] *= 1e-30
    c["x"][4] *= 1e-30
    c["x"][5, 3] = float("nan")
    c["x"][6, 4] = float("inf")
    c["h"][7] *= 1e-30
    c["x"][7] = 0
    for eps in (1e-6, 0.0):
        got = run_norms(c, qdtype, eps=eps)
        y, scale, x_out = [t.cpu() for t in got]
        keep = torch.tensor([0, 1, 2, 3, 4, 7, 8])
        sub = {k: (v[keep] if k in ("h", "x") else v) for k, v in c.items()}
        check_norms(sub, (y[keep], scale[keep], x_out[keep]), qdtype, eps=eps, label=str(eps))
        assert torch.isnan(scale[5]) and not torch.isfinite(scale[6])
        assert not R.codes_of(y[5:7], qdtype).any()


@pytest.mark.parametrize("n", [256, 250, 251, 20000])
def test_norms_special_rows_without_codes(n):
    c = norms_case(6, n, seed=18, gate_rows=1, smooth=True, beta=True)
    c["h"][0] = 0
    c["x"][0] = 0
    c["h"][1] *= 1e30
    c["x"][2] *= 1e35
    c["x"][3] *= 1e-30
    c["h"][3] *= 1e-30
    c["x"][4, 3] = float("nan")
    c["x"][5, 4] = float("inf")
    y, _, x_out = [t.cpu() if t is not None else None for t in run_norms(c, None, eps=0.0)]
    sub = {k: (v[:4] if k in ("h", "x") else v) for k, v in c.items()}
    check_norms(sub, (y[:4], None, x_out[:4]), None, eps=0.0)
    assert torch.isnan(y[4]).all() and torch.isnan(y[5, 4])


@pytest.mark.parametrize("qdtype", ["int8", "int4", None])
@pytest.mark.parametrize("n", [256, 250, 20000])
def test_norms_parameter_products_beyond_binary32(qdtype, n):
    # gamma_post * gate and gamma * smooth overflow a binary32 product where h, x' are zero
    c = norms_case(4, n, seed=19, gate_rows=1, smooth=True)
    c["gamma_post"][7], c["gate"][0, 7] = 1e30, 1e30
    c["gamma"][9], c["smooth"][9] = 3e25, 1e30
    c["h"][:, 7] = 0
    c["h"][:, 9] = 0
    c["x"][:, 9] = 0
    check_norms(c, run_norms(c, qdtype), qdtype)


@pytest.mark.parametrize("qdtype", ["int8", "int4"])
@pytest.mark.parametrize("n", [1024, 520, 1002, 20000])
def test_padding_rows(qdtype, n):
    # rows of zeros (of either sign) among others, in every position of a CTA's turn
    c = norms_case(700, n, seed=20, gate_rows=1, smooth=True)
    pad = torch.arange(700) % 3 != 1
    c["h"][pad] = 0
    c["x"][pad] = -0.0
    y, scale, x_out = got = run_norms(c, qdtype)
    check_norms(c, got, qdtype)
    assert not scale.cpu()[pad].any() and not R.codes_of(y, qdtype)[pad].any()
    x, s = glu_case(700, n, seed=21)
    x[pad] = 0
    check_glu(x, s, "silu", qdtype)
    x[pad, n:] = 1.0  # an up projection alone
    check_glu(x, s, "gelu_tanh", qdtype)


@pytest.mark.parametrize("alpha", [0.0, 1.0, -0.5, 1e-38, 1e30])
def test_norms_residual_scale(alpha):
    c = norms_case(4, 264, seed=9, gate_rows=4)
    check_norms(c, run_norms(c, "int8", alpha=alpha), "int8", alpha=alpha)


def test_norms_ties():
    # constant magnitudes: every quotient is +-Q or 0, every sum of squares exact
    c = norms_case(2, 64, seed=1)
    c["h"][:] = 0
    c["x"][:] = 1.5
    c["x"][0, ::2] = -1.5
    c["gamma"][:] = 1
    c["gamma"][5] = 0.5  # a quotient of 63.5: to even, 64 (the scale's rounding decides)
    check_norms(c, run_norms(c, "int8"), "int8")


# ------------------------------------------------------------------ gated activation

def glu_case(rows, n, dtype="bf16", seed=0, smooth=False):
    g = torch.Generator().manual_seed(seed)
    t = TDT[dtype]
    x = (torch.randn(rows, 2 * n, generator=g) * 2).to(t)
    s = (torch.randn(n, generator=g).abs() + 0.5).to(t) if smooth else None
    return x, s


def check_glu(x, s, act, qdtype, offset=0, label=""):
    y, scale = lib.glu_dynamic_quant(shifted(x, offset), shifted(s, offset), activation=act,
                                     qdtype=qdtype)
    R.check_codes(y, scale, R.glu_in(x, s, act), qdtype, label)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("qdtype", ["int8", "int4", "int4_int32"])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 64), (5, 4096), (2, 16384), (2, 20000)])
def test_glu(rows, n, qdtype, act, dtype):
    x, s = glu_case(rows, n, dtype, seed=rows + n, smooth=True)
    check_glu(x, s, act, qdtype)


@pytest.mark.parametrize("rows,n", [(1, 1), (4, 3), (9, 1001), (3, 16385), (2, 131071), (700, 1001)])
def test_glu_odd_lengths(rows, n):
    x, s = glu_case(rows, n, "fp16", seed=n)
    check_glu(x, s, "gelu_tanh", "int8")


@pytest.mark.parametrize("rows,n", [(2000, 1024), (900, 5120), (300, 14336)])
def test_glu_many_rows(rows, n):
    x, s = glu_case(rows, n, seed=n, smooth=True)
    check_glu(x, s, "silu", "int8")


@pytest.mark.parametrize("offset", [1, 4])
def test_glu_misaligned(offset):
    x, s = glu_case(7, 512, seed=offset, smooth=True)
    check_glu(x, s, "silu", "int4", offset=offset)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("qdtype", ["int8", "int4"])
@pytest.mark.parametrize("n", [256, 20000])
def test_glu_special_rows(qdtype, act, n):
    x, s = glu_case(8, n, seed=8)
    x[0] = 0
    x[1, :n] = 0
    x[2, :n] = -x[2, :n].abs() * 40 - 50   # gates whose sigmoid leaves binary32's range
    x[3, n:] *= 1e37
    x[4, :n] = -200.0                       # every value tiny
    x[5] *= 1e-25
    check_glu(x[:6], s, act, qdtype)
    x[6, 1] = float("nan")
    x[7, n + 2] = float("inf")
    y, scale = [t.cpu() for t in lib.glu_dynamic_quant(x.cuda(), activation=act, qdtype=qdtype)]
    assert torch.isnan(scale[6]) and not torch.isfinite(scale[7])
    assert not R.codes_of(y[6:], qdtype).any()


def test_rows_are_deterministic_and_replay():
    # the same bits on every call, on another stream and from a captured graph
    c = norms_case(64, 4096, seed=2, gate_rows=8, smooth=True)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    x, s = (t.cuda() for t in glu_case(64, 4096, seed=4, smooth=True))

    def both(stream=None):
        a = lib.post_norm_add_rms_norm_dynamic_quant(
            d["h"], d["x"], d["gamma_post"], d["gamma"], None, d["gate"], d["smooth"],
            residual_scale=0.25, stream=stream)
        return [*a, *lib.glu_dynamic_quant(x, s, stream=stream)]

    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    torch.cuda.synchronize()
    for a, b in zip(ref, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)

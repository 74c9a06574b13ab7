"""Rows at the edges of what the binary32 paths of the fused norms and the gated
activation may decide, on a GPU against plain 64-bit implementations.

The library decides in fp64 what binary32 cannot, the reference computes in fp64
throughout: the two differ by some 1e-14 of a quotient, a code next to that near
a half-way point has a chance of 1e-12, and so codes and scales have to be equal
here, without exception."""
import math

import pytest
import torch

import int4_quant_b200 as lib
from int4_quant_b200 import _abi as A
from int4_quant_b200 import build as B
from tests import _block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    A.lib()
    torch.cuda.set_device(0)


def same_codes(y, scale, v, qdtype):
    want, s = R.quantize(v, qdtype)
    got = scale.cpu()
    assert ((got == s) | (got.isnan() & s.isnan())).all()
    off = R.codes_of(y, qdtype) != want
    assert not off.any(), int(off.sum())


def glu_arg(g, act):
    return g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)


@pytest.mark.parametrize("qdtype", ["int8", "int4"])
@pytest.mark.parametrize("act,lowest", [("gelu_tanh", -9.5), ("gelu_tanh", -6.0), ("silu", -78.0)])
def test_glu_maximum_at_a_low_gate(act, lowest, qdtype):
    # the row's largest value has a gate far below zero, where the exponential's argument
    # costs binary32 many units in the last place; the others spread over the code range
    rows, n, t = 2048, 4096, torch.bfloat16
    g = torch.Generator().manual_seed(1)
    gate = torch.randn(rows, n, generator=g).to(t)
    low = torch.empty(rows).uniform_(lowest, -2.0, generator=g).to(t)
    at, r = torch.randint(0, n, (rows,), generator=g), torch.arange(rows)
    gate[r, at] = low
    top = low.double().abs() / (1 + torch.exp(-glu_arg(low.double(), act))) * 1e18
    a = gate.double()
    size = (a / (1 + torch.exp(-glu_arg(a, act)))).abs().clamp_min(1e-30)
    up = ((torch.rand(rows, n, generator=g).double() * 2 - 1) * 0.99 * top[:, None] / size).to(t)
    up[r, at] = 1e18
    x = torch.cat([gate, up], 1)
    y, scale = lib.glu_dynamic_quant(x.cuda(), activation=act, qdtype=qdtype)
    same_codes(y, scale, R.glu_in(x, None, act), qdtype)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("qdtype", ["int8", "int4"])
@pytest.mark.parametrize("n", [1024, 1002, 20000])
def test_glu_products_below_the_normal_range(n, qdtype, act):
    # up * smooth falls below 2^-126 (bf16 alone reaches that), a large gate lifts the value
    # far above it again
    t = torch.bfloat16
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    gate = ((r(64, n) + 0.1) * 1e30).to(t)
    up = ((r(64, n) - 0.5) * 2e-20).to(t)
    smooth = ((r(n) + 0.1) * 3e-23).to(t)
    x = torch.cat([gate, up], 1)
    y, scale = lib.glu_dynamic_quant(x.cuda(), smooth.cuda(), activation=act, qdtype=qdtype)
    same_codes(y, scale, R.glu_in(x, smooth, act), qdtype)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("size", [1e-38, 3e-39, 1e-40])
def test_glu_gates_below_the_normal_range(size, act):
    g = torch.Generator().manual_seed(3)
    gate = ((torch.rand(64, 1024, generator=g) - 0.5) * 2 * size).to(torch.bfloat16)
    up = ((torch.rand(64, 1024, generator=g) + 0.1) * 1e37).to(torch.bfloat16)
    x = torch.cat([gate, up], 1)
    y, scale = lib.glu_dynamic_quant(x.cuda(), activation=act)
    same_codes(y, scale, R.glu_in(x, None, act), "int8")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("n", [256, 251, 20000])
def test_glu_smooth_not_finite_beside_zeros(n, bad, act):
    # 0 times an infinity or a NaN is NaN: a zero gate, a zero up value, both, neither
    g = torch.Generator().manual_seed(4)
    x = torch.randn(5, 2 * n, generator=g).to(torch.bfloat16)
    smooth = torch.ones(n, dtype=torch.bfloat16)
    smooth[5] = bad
    x[0, 5] = 0
    x[1, n + 5] = -0.0
    x[2, 5] = x[2, n + 5] = 0
    x[3] = 0
    y, scale = lib.glu_dynamic_quant(x.cuda(), smooth.cuda(), activation=act)
    same_codes(y, scale, R.glu_in(x, smooth, act), "int8")
    assert torch.isnan(scale[:4]).all() and not torch.isfinite(scale[4])
    assert not R.codes_of(y, "int8").any()


def norms(h, x, gamma_post, gamma, gate=None, beta=None, smooth=None, qdtype="int8", alpha=1.0, eps=1e-6,
          eps_post=None):
    """Runs the fused norms; (y, scale, x_out), x_out checked bit by bit and y
    against the 64-bit form of what follows x_out."""
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, scale, x_out = got = lib.post_norm_add_rms_norm_dynamic_quant(
        c(h), c(x), c(gamma_post), c(gamma), c(beta), c(gate), c(smooth), residual_scale=alpha, eps=eps,
        eps_post=eps_post, qdtype=qdtype)
    want = R.norms_x(h, x, gamma_post, gate, alpha, eps if eps_post is None else eps_post)
    a = x_out.cpu()
    off = ~((a == want) | (a.isnan() & want.isnan()))
    assert not off.any(), int(off.sum())
    v = R.norms_in(a, gamma, beta, smooth, eps)
    if qdtype is not None:
        same_codes(y, scale, v, qdtype)
    return got, v


@pytest.mark.parametrize("n", [256, 250, 251, 1000, 20000])
@pytest.mark.parametrize("qdtype", ["int8", None])
def test_norms_zeros_beside_a_factor_beyond_binary32(n, qdtype):
    # h of 1e-39 without eps: residual_scale / Rms(h) overflows binary32, and zeros times it
    # must not; also behind the row's end
    t = torch.bfloat16
    g = torch.Generator().manual_seed(5)
    h = (torch.randn(6, n, generator=g) * 1e-39).to(t)
    h[:, 3] = 0
    h[1, 8:40] = 0
    h[2, :] = 0
    h[2, 5] = 1e-38
    x = torch.randn(6, n, generator=g).to(t)
    x[4] = 0
    ones = torch.ones(n, dtype=t)
    norms(h, x, ones, ones, qdtype=qdtype, eps_post=0.0)
    norms(h, x, ones, ones, gate=ones[None], qdtype=qdtype, alpha=-3.0, eps=0.0, eps_post=0.0)


@pytest.mark.parametrize("n", [512, 510, 511, 20000])
def test_norms_gate_products_below_the_normal_range(n):
    # gamma_post * gate below 2^-126 (bf16 alone reaches that) beside a large h and residual_scale
    t = torch.bfloat16
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.rand(s, generator=g).double() + 1  # noqa: E731
    h = (torch.randn(4, n, generator=g).double() * 2.0 ** 50).to(t)
    gamma_post, gate = (r(n) * 2.0 ** -70).to(t), (r(1, n) * 2.0 ** -75).to(t)
    x = (torch.randn(4, n, generator=g).double() * 2.0 ** -55).to(t)
    norms(h, x, gamma_post, torch.ones(n, dtype=t), gate=gate, alpha=2.0 ** 90, eps=0.0)


@pytest.mark.parametrize("qdtype", ["int8", "int4", None])
@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("n", [512, 510, 20000])
def test_norms_values_below_the_normal_range_lifted_again(n, beta, qdtype):
    # x' / Rms below 2^-126 beside a large gamma * smooth
    t = torch.bfloat16
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(s, generator=g).double()  # noqa: E731
    x, gamma, smooth = r(4, n) * 2.0 ** 50, torch.full((n,), 2.0 ** -70).double(), torch.ones(n).double()
    x[:, 1::2] = r(4, n // 2) * 2.0 ** -90
    gamma[1::2] = 2.0 ** 60
    smooth[1::2] = 2.0 ** 62
    b = (r(n) * 2.0 ** -20).to(t) if beta else None
    if beta:
        smooth[1::2], gamma[1::2] = 1.0, 2.0 ** 122
    (y, _, _), v = norms(torch.zeros(4, n, dtype=t), x.to(t), torch.ones(n, dtype=t), gamma.to(t), beta=b,
                         smooth=smooth.to(t), qdtype=qdtype, eps=0.0)
    if qdtype is None:
        # binary32: the factor, two products and the sum round once each (2^-24), then once to bf16
        size = v.abs() + (0 if b is None else 2 * b.double().abs() * smooth.to(t).double())
        assert ((y.cpu().double() - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -21 * size).all()


@pytest.mark.parametrize("n", [8, 96, 250, 256])
@pytest.mark.parametrize("in_place", [False, True])
def test_norms_small_rows_summed_again(n, in_place):
    # one warp a row; x' so small or large that its sum of squares is taken again from x_out
    t = torch.bfloat16
    g = torch.Generator().manual_seed(8)
    h = torch.zeros(400, n, dtype=t)
    x = (torch.randn(400, n, generator=g).double() * 10.0 ** torch.randint(-36, 20, (400, 1), generator=g)).to(t)
    one = torch.ones(n, dtype=t)
    d = x.cuda()
    y, scale, x_out = lib.post_norm_add_rms_norm_dynamic_quant(
        h.cuda(), d, one.cuda(), one.cuda(), eps=0.0, out={"x_out": d} if in_place else None)
    assert torch.equal(x_out.cpu(), x)
    same_codes(y, scale, R.norms_in(x, one, None, None, 0.0), "int8")

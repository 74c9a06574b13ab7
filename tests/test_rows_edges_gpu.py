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

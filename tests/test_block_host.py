"""Host-side refusals of the operators around the quantized product (no GPU):
every check runs before any CUDA call, on fake device addresses."""
import math

import pytest
import torch

import int4_quant_b200 as lib
from int4_quant_b200 import _abi as A
from int4_quant_b200 import build as B


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    A.lib()


P = {k: 0x7F0000000000 + i * 0x100000 for i, k in enumerate(
    ["h", "x", "gp", "gate", "g", "b", "s", "y", "sc", "xo", "w", "sw", "bias", "ws"])}


def norms(**kw):
    a = dict(h=P["h"], x=P["x"], gamma_post=P["gp"], gate=None, gate_rows=0, residual_scale=1.0,
             gamma=P["g"], beta=None, smooth=None, rows=0, n=64, dt=A.ARNQ_BF16, eps_post=1e-6,
             eps=1e-6, qdt=A.ARNQ_INT8, y=P["y"], scale=P["sc"], x_out=P["xo"], stream=None)
    a["rows"] = 12
    a.update(kw)
    return A.arnq_post_norm_add_rms_norm_dynamic_quant(**a)


@pytest.mark.parametrize("kw,expect", [
    (dict(h=None), A.ARNQ_ERR_NULL_PTR),
    (dict(x=None), A.ARNQ_ERR_NULL_PTR),
    (dict(gamma_post=None), A.ARNQ_ERR_NULL_PTR),
    (dict(gamma=None), A.ARNQ_ERR_NULL_PTR),
    (dict(y=None), A.ARNQ_ERR_NULL_PTR),
    (dict(scale=None), A.ARNQ_ERR_NULL_PTR),
    (dict(rows=0), A.ARNQ_ERR_EMPTY),
    (dict(n=0), A.ARNQ_ERR_EMPTY),
    (dict(rows=-1), A.ARNQ_ERR_SHAPE),
    (dict(rows=2 ** 31), A.ARNQ_ERR_SHAPE),
    (dict(n=A.ARNQ_MAX_N + 8), A.ARNQ_ERR_SHAPE),
    (dict(n=63, qdt=A.ARNQ_INT4), A.ARNQ_ERR_SHAPE),
    (dict(n=60, qdt=A.ARNQ_INT4_INT32), A.ARNQ_ERR_SHAPE),
    (dict(dt=A.ARNQ_FP32), A.ARNQ_ERR_DTYPE),
    (dict(qdt=3), A.ARNQ_ERR_DTYPE),
    (dict(eps=-1e-6), A.ARNQ_ERR_EPS),
    (dict(eps_post=math.nan), A.ARNQ_ERR_EPS),
    (dict(residual_scale=math.inf), A.ARNQ_ERR_ARG),
    (dict(gate=P["gate"], gate_rows=0), A.ARNQ_ERR_ARG),
    (dict(gate_rows=1), A.ARNQ_ERR_ARG),
    (dict(gate=P["gate"], gate_rows=5), A.ARNQ_ERR_ARG),
    (dict(gate=P["gate"], gate_rows=-1), A.ARNQ_ERR_ARG),
    (dict(gate=P["gate"], gate_rows=24), A.ARNQ_ERR_ARG),
    (dict(gamma_post=P["gp"] + 1), A.ARNQ_ERR_ALIGN),
    (dict(scale=P["sc"] + 2), A.ARNQ_ERR_ALIGN),
    (dict(qdt=A.ARNQ_INT4_INT32, y=P["y"] + 2), A.ARNQ_ERR_ALIGN),
    (dict(qdt=A.ARNQ_NO_CODES, y=P["y"] + 1), A.ARNQ_ERR_ALIGN),
    (dict(x_out=P["xo"] + 1), A.ARNQ_ERR_ALIGN),
])
def test_norms_refusals(kw, expect):
    assert norms(**kw) == expect


def test_no_codes_is_refused_elsewhere():
    assert A.arnq_glu_dynamic_quant(P["x"], None, 4, 64, 0, 0, A.ARNQ_NO_CODES, P["y"], P["sc"],
                                    None) == A.ARNQ_ERR_DTYPE
    assert A.arnq_workspace_size(4, 64, 0, A.ARNQ_NO_CODES, -1, 0, 0)[0] == A.ARNQ_ERR_DTYPE


def glu(**kw):
    a = dict(x=P["x"], smooth=None, rows=8, n=64, dt=A.ARNQ_BF16, act=A.ARNQ_SILU, qdt=A.ARNQ_INT8,
             y=P["y"], scale=P["sc"], stream=None)
    a.update(kw)
    return A.arnq_glu_dynamic_quant(**a)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), A.ARNQ_ERR_NULL_PTR),
    (dict(y=None), A.ARNQ_ERR_NULL_PTR),
    (dict(scale=None), A.ARNQ_ERR_NULL_PTR),
    (dict(rows=0), A.ARNQ_ERR_EMPTY),
    (dict(n=0), A.ARNQ_ERR_EMPTY),
    (dict(n=-8), A.ARNQ_ERR_SHAPE),
    (dict(n=A.ARNQ_MAX_N + 1), A.ARNQ_ERR_SHAPE),
    (dict(n=7, qdt=A.ARNQ_INT4), A.ARNQ_ERR_SHAPE),
    (dict(dt=2), A.ARNQ_ERR_DTYPE),
    (dict(act=2), A.ARNQ_ERR_ARG),
    (dict(act=-1), A.ARNQ_ERR_ARG),
    (dict(x=P["x"] + 1), A.ARNQ_ERR_ALIGN),
    (dict(smooth=P["s"] + 1), A.ARNQ_ERR_ALIGN),
    (dict(scale=P["sc"] + 1), A.ARNQ_ERR_ALIGN),
])
def test_glu_refusals(kw, expect):
    assert glu(**kw) == expect


def matmul(**kw):
    a = dict(x=P["x"], scale_x=P["sc"], w=P["w"], scale_w=P["sw"], bias=None, m=8, n=64, k=32,
             out_dt=A.ARNQ_BF16, y=P["y"], workspace=P["ws"], workspace_bytes=256, stream=None)
    a.update(kw)
    return A.arnq_quant_matmul(**a)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), A.ARNQ_ERR_NULL_PTR),
    (dict(scale_x=None), A.ARNQ_ERR_NULL_PTR),
    (dict(w=None), A.ARNQ_ERR_NULL_PTR),
    (dict(scale_w=None), A.ARNQ_ERR_NULL_PTR),
    (dict(y=None), A.ARNQ_ERR_NULL_PTR),
    (dict(m=0), A.ARNQ_ERR_EMPTY),
    (dict(n=0), A.ARNQ_ERR_EMPTY),
    (dict(k=0), A.ARNQ_ERR_EMPTY),
    (dict(m=-1), A.ARNQ_ERR_SHAPE),
    (dict(m=2 ** 31), A.ARNQ_ERR_SHAPE),
    (dict(n=A.ARNQ_MAX_N + 1), A.ARNQ_ERR_SHAPE),
    (dict(k=A.ARNQ_MAX_K + 1), A.ARNQ_ERR_SHAPE),
    (dict(out_dt=3), A.ARNQ_ERR_DTYPE),
    (dict(y=P["y"] + 1), A.ARNQ_ERR_ALIGN),
    (dict(out_dt=A.ARNQ_FP32, y=P["y"] + 2), A.ARNQ_ERR_ALIGN),
    (dict(bias=P["bias"] + 1), A.ARNQ_ERR_ALIGN),
    (dict(scale_x=P["sc"] + 2), A.ARNQ_ERR_ALIGN),
    (dict(scale_w=P["sw"] + 2), A.ARNQ_ERR_ALIGN),
    (dict(workspace=None), A.ARNQ_ERR_WORKSPACE),
    (dict(workspace_bytes=255), A.ARNQ_ERR_WORKSPACE),
    (dict(workspace=P["ws"] + 4), A.ARNQ_ERR_ALIGN),
])
def test_matmul_refusals(kw, expect):
    assert matmul(**kw) == expect


@pytest.mark.parametrize("kw,k,expect", [
    (dict(kernel=3), 256, A.ARNQ_ERR_PLAN),
    (dict(kernel=-1), 256, A.ARNQ_ERR_PLAN),
    (dict(kernel=A.ARNQ_MATMUL_PAIR), 250, A.ARNQ_ERR_PLAN),
    (dict(tokens=24), 256, A.ARNQ_ERR_PLAN),
    (dict(tokens=272), 256, A.ARNQ_ERR_PLAN),
    (dict(split=3), 256, A.ARNQ_ERR_PLAN),
    (dict(split=16), 4096, A.ARNQ_ERR_PLAN),
    (dict(split=4), 256, A.ARNQ_ERR_PLAN),
    (dict(wait_limit_us=-1), 256, A.ARNQ_ERR_PLAN),
    (dict(test_hold_bytes=65537), 256, A.ARNQ_ERR_PLAN),
    (dict(test_hold_bytes=16), 250, A.ARNQ_ERR_PLAN),
])
def test_matmul_plan_refusals(kw, k, expect):
    p = A.arnq_matmul_plan()
    for name, v in kw.items():
        setattr(p, name, v)
    assert A.arnq_quant_matmul_planned(P["x"], P["sc"], P["w"], P["sw"], None, 8, 64, k, A.ARNQ_BF16,
                                       P["y"], P["ws"], 256, None, p) == expect


def test_torch_calls_refuse_cpu_tensors():
    codes = torch.zeros(4, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        lib.quant_matmul(codes, torch.zeros(4), codes, torch.zeros(4))
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    v = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.post_norm_add_rms_norm_dynamic_quant(x, x, v, v)
    with pytest.raises(ValueError):
        lib.glu_dynamic_quant(x)

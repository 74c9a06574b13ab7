"""Plain 64-bit implementations of the operators around the quantized product
(torch, float64), and the comparisons the tests make with them."""
import math

import numpy as np
import torch

from tests._util import codes

Q = {"int8": 127.0, "int4": 7.0, "int4_int32": 7.0}


def to16(v, t):
    """float64 -> 16 bits, one rounding to nearest even: the two neighbours of
    the cast compared with v, the cast itself kept unless one is nearer (its
    own error is below one unit in the last place, and a value half-way
    between two neighbours passes through binary32 unchanged)."""
    r = v.to(t)
    bits = r.view(torch.int16)
    best, err = r, (r.double() - v).abs()
    for step in (-1, 1):
        c = (bits + step).view(t)
        e = (c.double() - v).abs()
        best, err = torch.where(e < err, c, best), torch.where(e < err, e, err)
    return best


def over_rms(v, eps):
    rms = (v * v).mean(-1, keepdim=True).add(eps).sqrt()
    return torch.where(rms == 0, torch.zeros_like(v), v / rms)


def norms_x(h, x, gamma_post, gate, alpha, eps):
    p = over_rms(h.double(), eps) * gamma_post.double()
    if gate is not None:
        g = gate.double().reshape(-1, h.shape[-1])
        p = p * g.repeat_interleave(h.shape[0] // g.shape[0], 0)
    return to16(x.double() + float(np.float32(alpha)) * p, x.dtype)


def norms_in(x_out, gamma, beta, smooth, eps):
    v = over_rms(x_out.double(), eps) * gamma.double()
    if beta is not None:
        v = v + beta.double()
    return v if smooth is None else v * smooth.double()


def glu_in(x, smooth, act):
    n = x.shape[-1] // 2
    g, u = x[:, :n].double(), x[:, n:].double()
    z = g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
    v = g / (1 + torch.exp(-z)) * u
    return v if smooth is None else v * smooth.double()


def quantize(v, qdtype):
    """(codes as int64, binary32 scales) of rows of float64 values."""
    q = Q[qdtype]
    scale = (v.abs().amax(-1) / q).float()
    s = scale.double()[:, None]
    ok = (s > 0) & torch.isfinite(s)
    c = torch.where(ok, v / torch.where(ok, s, torch.ones_like(s)), torch.zeros_like(v))
    return c.round().clamp(-q, q).long(), scale


def codes_of(y, qdtype):
    return torch.from_numpy(codes(y.cpu().numpy(), qdtype).astype(np.int64))


def check_codes(y, scale, v, qdtype, label=""):
    """Scales within one binary32 step and codes equal but for 1e-5 of them off
    by one (in small cases: equal).  The kernel decides both in fp64, as the
    reference does; what differs between the two is some 2^-50."""
    want, s = quantize(v, qdtype)
    got = codes_of(y, qdtype)
    a, b = scale.cpu().double(), s.double()
    assert torch.equal(torch.isnan(a), torch.isnan(b)), label
    fine = torch.isfinite(b)
    assert torch.equal(a[~fine & ~torch.isnan(b)], b[~fine & ~torch.isnan(b)]), label
    rel = (a[fine] - b[fine]).abs() / b[fine].clamp_min(1e-300)
    assert rel.numel() == 0 or rel.max() <= 2.0 ** -23, (label, rel.max())
    d = (got - want).abs()
    assert d.max() <= 1, (label, int(d.max()))
    assert int((d != 0).sum()) <= int(1e-5 * d.numel()), (label, int((d != 0).sum()))


def check_x(x_out, ref, label=""):
    """x_out equal to the once-rounded 64-bit sum but for 1e-5 of the elements,
    those one 16-bit step off (in small cases: equal); both are decided in fp64."""
    a, b = x_out.cpu(), ref.cpu()
    same = (a.view(torch.int16) == b.view(torch.int16)) | (a == b) | (torch.isnan(a) & torch.isnan(b))
    off = (~same).sum()
    assert int(off) <= int(1e-5 * a.numel()), (label, int(off))
    if off:
        step = torch.finfo(a.dtype).eps * b.double().abs()[~same].clamp_min(torch.finfo(a.dtype).tiny)
        assert ((a.double() - b.double()).abs()[~same] <= 2 * step).all(), label

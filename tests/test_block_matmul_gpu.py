"""The INT8 product with token and channel scales on a GPU, against the sum in
64 bits (exact: the products' sums stay below 2^53)."""
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


def case(m, n, k, bias=None, seed=0, full=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lim = 128 if full else 127
    x = torch.randint(-lim, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-lim, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(m, generator=g, device="cuda") * 0.05 + 0.01
    sw = torch.rand(n, generator=g, device="cuda") * 0.001 + 0.0002
    b = None if bias is None else torch.randn(n, generator=g, device="cuda").to(bias)
    return x, sx, w, sw, b


def check(x, sx, w, sw, b, y, label=""):
    """Binary32: the sum's conversion, two products and the addition round once
    each (2^-24 of what they round), the output once more by half a step."""
    acc = x.double() @ w.double().T
    prod = acc * sx.double()[:, None] * sw.double()
    ref = prod if b is None else prod + b.double()
    half = torch.finfo(y.dtype).eps / 2
    bound = prod.abs() * 3 * 2.0 ** -24 * 1.001 + ref.abs() * 2.0 ** -24 * 1.001
    if y.dtype != torch.float32:
        bound = bound + (ref.abs() + bound) * half + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    err = (y.double() - ref).abs()
    bad = err > bound
    assert not bad.any(), (label, int(bad.sum()), bad.nonzero()[:4].tolist(), float(err.max()))


def run(m, n, k, out=torch.bfloat16, bias=False, seed=0, **kw):
    c = case(m, n, k, out if bias else None, seed, **kw)
    y = lib.quant_matmul(c[0], c[1], c[2], c[3], c[4], out_dtype=out)
    check(*c, y, (m, n, k))


@pytest.mark.parametrize("m,n,k", [(16, 128, 128), (1, 128, 128), (1, 8, 16), (16, 128, 512),
                                   (7, 256, 1024), (32, 384, 4096), (256, 128, 256),
                                   (200, 1000, 1040), (257, 520, 2064)])
def test_small(m, n, k):
    run(m, n, k, seed=m + n + k)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k", [(5, 260, 4096), (130, 514, 768), (600, 777, 528)])
def test_types_and_bias(m, n, k, out, bias):
    run(m, n, k, out, bias, seed=m)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 5, 7), (17, 129, 127), (129, 1023, 1001),
                                   (2, 64, 4099), (300, 130, 333)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_odd_sizes(m, n, k, out):
    run(m, n, k, out, True, seed=n)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (4, 1024, 16384), (16, 16384, 1024),
                                   (64, 5120, 5120), (512, 4096, 1024), (1111, 2048, 2048),
                                   (4096, 4096, 512)])
def test_ordinary_sizes(m, n, k):
    run(m, n, k, seed=k)


@pytest.mark.parametrize("k", [131071, 131056])
def test_longest_sums(k):
    # every code -128: the largest sum, 2^31 - 2^14 or below
    x = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((130, k), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    sx = torch.ones(3, device="cuda")
    sw = torch.ones(130, device="cuda")
    check(x, sx, w, sw, None, lib.quant_matmul(x, sx, w, sw, out_dtype=torch.float32))


def test_full_code_range():
    run(33, 256, 1024, torch.float32, seed=1, full=True)


@pytest.mark.parametrize("offset", [1, 4, 8])
def test_misaligned_codes(offset):
    x, sx, w, sw, _ = case(9, 130, 512, seed=offset)
    bx = torch.empty(x.numel() + offset, dtype=torch.int8, device="cuda")
    bw = torch.empty(w.numel() + offset, dtype=torch.int8, device="cuda")
    bx[offset:].copy_(x.reshape(-1))
    bw[offset:].copy_(w.reshape(-1))
    x2, w2 = bx[offset:].view(x.shape), bw[offset:].view(w.shape)
    y = lib.quant_matmul(x2, sx, w2, sw)
    check(x, sx, w, sw, None, y)
    assert torch.equal(y, lib.quant_matmul(x, sx, w, sw))


def test_output_beside_others():
    # an output that starts off a vector boundary, and canaries around it
    x, sx, w, sw, _ = case(50, 200, 256, seed=3)
    buf = torch.full((50 * 200 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[33:33 + 50 * 200].view(50, 200)
    lib.quant_matmul(x, sx, w, sw, out=y)
    check(x, sx, w, sw, None, y)
    assert (buf[:33] == 7).all() and (buf[33 + 10000:] == 7).all()


def test_scales_propagate():
    x, sx, w, sw, _ = case(4, 128, 128, seed=5)
    sx[0], sx[1], sx[2] = 0.0, float("nan"), float("inf")
    y = lib.quant_matmul(x, sx, w, sw, out_dtype=torch.float32)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    check(x[3:], sx[3:], w, sw, None, y[3:])


def test_leading_dimensions_and_empty():
    x, sx, w, sw, _ = case(12, 128, 64, seed=6)
    y = lib.quant_matmul(x.view(3, 4, 64), sx.view(3, 4), w, sw)
    assert y.shape == (3, 4, 128)
    check(x, sx, w, sw, None, y.view(12, 128))
    with pytest.raises(lib.ArnqError):
        lib.quant_matmul(x[:0], sx[:0], w, sw)
    with pytest.raises(ValueError):
        lib.quant_matmul(x, sx, w[:, :32], sw)
    with pytest.raises(ValueError):
        lib.quant_matmul(x.t(), sx, w, sw)


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (300, 512, 1024), (2048, 2048, 512), (9, 100, 99)])
def test_deterministic_streams_and_graph(m, n, k):
    x, sx, w, sw, _ = case(m, n, k, seed=7)
    ref = lib.quant_matmul(x, sx, w, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = lib.quant_matmul(x, sx, w, sw, stream=side)
    b = lib.quant_matmul(x, sx, w, sw)
    torch.cuda.synchronize()
    assert torch.equal(ref, a) and torch.equal(ref, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.quant_matmul(x, sx, w, sw)
    y.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, y)


def test_block_of_operators():
    """A gated MLP with INT8 weights between its norms, as a model runs it, each
    step against its 64-bit form on the step's own inputs."""
    n, inner, rows = 512, 1024, 40
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t = torch.bfloat16
    gamma = [(r(n) * 0.1 + 1).to(t) for _ in range(3)]
    x1, x2 = r(rows, n).to(t), r(rows, n).to(t)
    w1 = torch.randint(-127, 128, (2 * inner, n), generator=g, device="cuda", dtype=torch.int8)
    w2 = torch.randint(-127, 128, (n, inner), generator=g, device="cuda", dtype=torch.int8)
    sw1, sw2 = torch.full((2 * inner,), 0.001, device="cuda"), torch.full((n,), 0.001, device="cuda")
    gate = r(4, n).to(t)

    def block():
        a, sa, _, _, x = lib.add_rms_norm_dynamic_quant(x1, x2, gamma[0])
        gu = lib.quant_matmul(a, sa, w1, sw1)
        b, sb = lib.glu_dynamic_quant(gu)
        h = lib.quant_matmul(b, sb, w2, sw2)
        y, sy, xo = lib.post_norm_add_rms_norm_dynamic_quant(h, x, gamma[1], gamma[2], gate=gate,
                                                             residual_scale=0.5)
        return a, sa, x, gu, b, sb, h, y, sy, xo

    a, sa, x, gu, b, sb, h, y, sy, xo = got = block()
    check(a, sa, w1, sw1, None, gu)
    R.check_codes(b, sb, R.glu_in(gu.cpu(), None, "silu"), "int8")
    check(b, sb, w2, sw2, None, h)
    c = lambda v: v.cpu()  # noqa: E731
    R.check_x(xo, R.norms_x(c(h), c(x), c(gamma[1]), c(gate), 0.5, 1e-6))
    R.check_codes(y, sy, R.norms_in(c(xo), c(gamma[2]), None, None, 1e-6), "int8")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = block()
    for v in again:
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, again):
        assert torch.equal(p, q)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(513, 256, 128), (700, 300, 640), (1024, 1000, 4096), (2048, 777, 1040),
                                   (5000, 264, 144), (1500, 4104, 2048), (3000, 8, 16), (520, 16384, 256)])
def test_many_tokens(m, n, k, out):
    run(m, n, k, out, True, seed=m + n)


def test_many_tokens_output_off_alignment():
    x, sx, w, sw, _ = case(800, 512, 256, seed=4)
    buf = torch.full((800 * 512 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[33:33 + 800 * 512].view(800, 512)
    lib.quant_matmul(x, sx, w, sw, out=y)
    check(x, sx, w, sw, None, y)
    assert (buf[:33] == 7).all() and (buf[33 + 800 * 512:] == 7).all()


def test_many_tokens_leaves_neighbours_alone():
    # ragged rows and channels of an aligned output inside a larger buffer
    x, sx, w, sw, _ = case(777, 264, 256, seed=8)
    buf = torch.full((1000, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.quant_matmul(x, sx, w, sw, out=buf[:777])
    check(x, sx, w, sw, None, buf[:777])
    assert (buf[777:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(8192, 7168, 256), (4500, 2560, 384), (2816, 6000, 128), (9000, 4352, 1040),
                                   (40000, 520, 512)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_more_tiles_than_pairs(m, n, k, out):
    # several tiles for each pair of CTAs: two at a time, singles behind them, odd rows of tiles
    run(m, n, k, out, out == torch.float32, seed=m)


def planned(c, ws=None, **kw):
    x, sx, w, sw, b = c
    p = A.arnq_matmul_plan()
    for name, v in kw.items():
        setattr(p, name, v)
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda") if ws is None else ws
    st = A.arnq_quant_matmul_planned(x, sx, w, sw, b, x.shape[0], w.shape[0], x.shape[1], A.ARNQ_FP32, y,
                                     ws, 256, torch.cuda.current_stream(), p)
    assert st == A.ARNQ_OK, A.arnq_status_string(st)
    torch.cuda.synchronize()
    return y, lib.workspace_status(ws)


@pytest.mark.parametrize("m,n,k", [(1, 128, 1024), (100, 300, 1040), (300, 520, 2064), (513, 776, 1024)])
def test_plans_give_the_same_bits(m, n, k):
    c = case(m, n, k, torch.float32, seed=m)
    ref, status = planned(c)
    check(*c, ref)
    assert status[0] == 0
    for kw in (dict(kernel=2), dict(kernel=1), dict(kernel=1, split=1), dict(kernel=1, split=2, tokens=16),
               dict(kernel=1, split=4, tokens=64), dict(kernel=1, split=8, tokens=256)):
        y, status = planned(c, **kw)
        assert torch.equal(ref, y) and status[0] == 0, kw


def test_two_streams_at_once():
    # both kernels side by side, again and again: SMs, TMEM and shared memory shared between them
    a, b = case(1200, 1024, 1024, seed=1), case(16, 2048, 2048, seed=2)
    ra, rb = lib.quant_matmul(*a[:4]), lib.quant_matmul(*b[:4])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ya = [lib.quant_matmul(*a[:4], stream=s1) if i % 2 else lib.quant_matmul(*b[:4], stream=s1) for i in range(40)]
    yb = [lib.quant_matmul(*b[:4], stream=s2.cuda_stream) if i % 2 else
          lib.quant_matmul(*a[:4], stream=s2.cuda_stream) for i in range(40)]
    torch.cuda.synchronize()
    for i in range(40):
        assert torch.equal(ya[i], ra if i % 2 else rb) and torch.equal(yb[i], rb if i % 2 else ra)


@pytest.mark.parametrize("kw", [dict(kernel=1, split=1), dict(kernel=1, split=4), dict(kernel=2)])
def test_a_wait_that_runs_out_is_reported(kw):
    c = case(300, 512, 4096, seed=3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    _, status = planned(c, ws, wait_limit_us=2000, test_hold_bytes=64, **kw)
    assert status == (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
    # the context and the kernels work on
    y, status = planned(c, **kw)
    check(*c, y)
    assert status[0] == 0

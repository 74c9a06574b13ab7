"""The torch calls of the operators around the quantized product: streams,
outputs, status, refusals that need CUDA tensors."""
import pytest
import torch

import int4_quant_b200 as lib
from int4_quant_b200 import _abi as A
from int4_quant_b200 import build as B
from tests.test_block_matmul_gpu import case, planned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    A.lib()
    torch.cuda.set_device(0)


def test_stream_handles():
    # the handle a call launches on: of a stream, of its integer handle, of the default stream's, 0
    side = torch.cuda.Stream()
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    lib.glu_dynamic_quant(x)
    launched = lambda s: lib._on_stream(lambda h: (h, torch.cuda.current_stream().cuda_stream), 0, s)  # noqa: E731
    for s in (side, side.cuda_stream):
        assert launched(s) == (side.cuda_stream,) * 2
    default = torch.cuda.default_stream()
    assert default.cuda_stream == 0
    with torch.cuda.stream(side):
        assert launched(default) == launched(0) == (0, 0)
        assert launched(None) == (side.cuda_stream,) * 2


@pytest.mark.parametrize("op", ["matmul", "norms", "glu"])
def test_the_default_streams_handle_keeps_its_order(op):
    # behind work on the default stream that makes the inputs, called from another stream
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        torch.cuda.synchronize()
        b = a
        for _ in range(6):
            b = torch.relu(b @ a) * 0.01
        bits = (b[:64, :256] > 0)
        if op == "matmul":
            x = bits.to(torch.int8)
            w, s = torch.ones(16, 256, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
            call = lambda st: lib.quant_matmul(x, s, w, s[:16], stream=st)  # noqa: E731
        else:
            x, one = bits.to(torch.bfloat16) + 1, torch.ones(256, dtype=torch.bfloat16, device="cuda")
            call = (lambda st: lib.glu_dynamic_quant(x, stream=st)[0]) if op == "glu" else \
                (lambda st: lib.post_norm_add_rms_norm_dynamic_quant(x, x, one, one, stream=st)[0])  # noqa: E731
        with torch.cuda.stream(side):
            y = call(0)
        torch.cuda.synchronize()
        assert torch.equal(y, call(None))


def test_a_gate_of_no_rows_is_refused():
    # its address is NULL, which stands for no gate
    x, one = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        lib.post_norm_add_rms_norm_dynamic_quant(x, x, one, one, gate=x[:0])
    with pytest.raises(lib.ArnqError):
        lib.post_norm_add_rms_norm_dynamic_quant(x, x, one, one, gate=x[:3])


def product(m=16, n=64, k=64):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    return r(m, k), torch.ones(m, device="cuda"), r(n, k), torch.ones(n, device="cuda")


def record(stream, code=A.ARNQ_ERR_DEVICE_TIMEOUT, row=-1):
    """Writes a status where a kernel of that stream would."""
    slab, _ = lib._status_slabs[0]
    block = slab[lib._status_blocks[0][stream.cuda_stream]]
    block[:16].copy_(torch.tensor([code, 0, row & 0xFFFFFFFF, row >> 32 & 0xFFFFFFFF]).to(torch.uint32)
                     .view(torch.uint8))
    torch.cuda.synchronize()


@pytest.fixture
def no_blocks(monkeypatch):
    monkeypatch.setattr(lib, "_status_slabs", {})
    monkeypatch.setattr(lib, "_status_blocks", {})


def test_status_of_streams(no_blocks):
    c, here = product(), torch.cuda.current_stream()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    assert lib.quant_matmul_status() == (0, 0)
    for s in (None, s1, s2):
        lib.quant_matmul(*c, stream=s)
    assert lib.quant_matmul_status() == lib.quant_matmul_status(0) == (0, 0)
    record(s1)
    late = (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
    assert lib.quant_matmul_status() == lib.quant_matmul_status("cuda:0") == late
    assert lib.quant_matmul_status(stream=s1) == lib.quant_matmul_status(stream=s1.cuda_stream) == late
    for s in (here, s2, 0, torch.cuda.Stream()):
        assert lib.quant_matmul_status(stream=s) == (0, 0)
    lib.quant_matmul(*c, stream=s1)  # a later call leaves it
    assert lib.quant_matmul_status(stream=s2, clear=True) == (0, 0)
    assert lib.quant_matmul_status(stream=s1, clear=True) == late
    assert lib.quant_matmul_status(clear=True) == (0, 0)
    record(s2)
    assert lib.quant_matmul_status(clear=True) == late
    assert lib.quant_matmul_status() == (0, 0)


def test_a_captured_first_call_is_refused(no_blocks):
    c = product()
    ref = (c[0].double() @ c[2].double().T).to(torch.bfloat16)
    with pytest.raises(RuntimeError, match="once before"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.zeros(4, device="cuda")
            lib.quant_matmul(*c)
    torch.cuda.synchronize()
    lib.quant_matmul_status()  # once outside
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.quant_matmul(*c)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and lib.quant_matmul_status() == (0, 0)


def test_a_replay_leaves_the_status(no_blocks):
    # a stream's first call is one that is captured: a recorded status outlives the replays
    c = product()
    lib.quant_matmul(*c)
    graphs, streams, ys = [], [], []
    for _ in range(2):  # two graphs that share torch's capture stream, and its block
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            streams.append(torch.cuda.current_stream())
            ys.append(lib.quant_matmul(*c))
    record(streams[0])
    for g in graphs:
        g.replay()
    assert lib.quant_matmul_status(stream=streams[0], clear=True) == (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
    for g in graphs:
        g.replay()
    assert lib.quant_matmul_status() == (0, 0)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], lib.quant_matmul(*c))


def test_blocks_are_handed_on(no_blocks, monkeypatch):
    # the number of blocks is bounded, however many streams there were
    monkeypatch.setattr(lib, "_STATUS_BLOCKS", 3)
    at = [lib._status_block(0, 1000 + i) for i in range(5)]
    assert len(set(at[:3])) == 3 and at[3:] == at[:2]
    assert at[1] == lib._status_block(0, 1004) and at[2] == lib._status_block(0, 1002)
    assert len(lib._status_blocks[0]) == 3
    base, size = lib._status_slabs[0][1], 3 * A.ARNQ_WORKSPACE_BYTES
    assert all(base <= a < base + size for a in at)


def test_a_wait_that_ran_out_reaches_the_caller(no_blocks):
    c = (*case(64, 256, 1024, seed=2)[:4], None)
    lib.quant_matmul(*c)
    here = torch.cuda.current_stream()
    block = lib._status_slabs[0][0][lib._status_blocks[0][here.cuda_stream]]
    planned(c, block, kernel=1, wait_limit_us=2000, test_hold_bytes=64)
    assert lib.quant_matmul_status(stream=here) == (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
    assert lib.quant_matmul_status(clear=True) == (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
    assert lib.quant_matmul_status() == (0, 0)


def all_calls():
    c = product()
    x, one = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    return [lib.quant_matmul(*c), *lib.glu_dynamic_quant(x),
            *lib.post_norm_add_rms_norm_dynamic_quant(x, x, one, one, qdtype="int4")]


def test_modes_see_the_outputs():
    from torch.overrides import TorchFunctionMode
    from torch.utils._python_dispatch import TorchDispatchMode

    class Dispatched(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(func(*args, **(kwargs or {})))
            return seen[-1]

    class Called(TorchFunctionMode):
        def __torch_function__(self, func, types, args=(), kwargs=None):
            seen.append(func(*args, **(kwargs or {})))
            return seen[-1]

    ref = all_calls()
    for mode in (Dispatched, Called):
        seen = []
        with mode():
            got = all_calls()
        made = {id(t) for t in seen}
        assert all(id(t) in made for t in got), mode
        for a, b in zip(ref, got):
            assert torch.equal(a, b)


def test_without_torchs_private_shortcuts(monkeypatch):
    ref = all_calls()
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_len_torch_dispatch_stack"):
        monkeypatch.delattr(torch._C, name)
    T = lib._Torch()
    monkeypatch.undo()
    monkeypatch.setattr(lib, "_torch_cache", T)
    side = torch.cuda.Stream()
    assert T.current_device() == 0 and T.raw_stream(0) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert T.raw_stream(0) == side.cuda_stream
    for a, b in zip(ref, all_calls()):
        assert torch.equal(a, b)


def test_status_of_a_device_and_a_stream(no_blocks):
    s = torch.cuda.Stream()
    lib.quant_matmul(*product(), stream=s)
    for device in (None, 0, "cuda", "cuda:0", torch.device("cuda", 0)):
        assert lib.quant_matmul_status(device, stream=s) == (0, 0)

    class Elsewhere:  # (a stream of a second device)
        device, cuda_stream = torch.device("cuda", 1), s.cuda_stream

    with pytest.raises(ValueError):
        lib.quant_matmul_status(0, stream=Elsewhere)

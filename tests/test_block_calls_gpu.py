"""The torch calls of the operators around the quantized product: streams,
outputs, status, refusals that need CUDA tensors."""
import pytest
import torch

import int4_quant_b200 as lib
from int4_quant_b200 import _abi as A
from int4_quant_b200 import build as B

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

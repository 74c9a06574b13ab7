"""Products whose waits run out: reported, over in time, and harmless to what
runs next.  (The held-back bytes are only expected, never copied: every copy and
MMA that such a call starts ends.)"""
import time

import pytest
import torch

import int4_quant_b200 as lib
from int4_quant_b200 import _abi as A
from int4_quant_b200 import build as B
from tests.test_block_matmul_gpu import case, check, planned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.build()
    A.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("tokens,split", [(16, 1), (16, 8), (48, 2), (144, 4), (256, 1), (256, 8)])
def test_epilogue_and_mma_give_up_together(tokens, split):
    # their limits run out at the same moment: the epilogue's warps agree on what they saw
    c = case(300, 512, 2048, seed=tokens + split)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for limit in (300, 301, 350, 400):
        ws.zero_()
        begin = time.monotonic()
        _, status = planned(c, ws, kernel=1, tokens=tokens, split=split, wait_limit_us=limit,
                            test_hold_bytes=64)
        assert status == (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
        assert time.monotonic() - begin < 5
    y, status = planned(c, kernel=1, tokens=tokens, split=split)
    check(*c, y)
    assert status[0] == 0


@pytest.mark.parametrize("k", [128, 512, 4096])
@pytest.mark.parametrize("kw", [dict(kernel=1, tokens=16, split=1), dict(kernel=1, tokens=256, split=1),
                                dict(kernel=2)])
def test_products_right_behind_one_that_gave_up(kw, k):
    # the copies are all started before the limit runs out (k = 128, 512) or not (4096);
    # nothing of the call is still at work when the next ones take its place
    c = case(600, 1024, k, seed=k)
    x, sx, w, sw, _ = c
    ref = lib.quant_matmul(x, sx, w, sw)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    held = A.arnq_matmul_plan(wait_limit_us=500, test_hold_bytes=64, **kw)
    y = torch.empty(600, 1024, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    after = []
    for _ in range(3):
        st = A.arnq_quant_matmul_planned(x, sx, w, sw, None, 600, 1024, k, A.ARNQ_FP32, y, ws, 256,
                                         torch.cuda.current_stream(), held)
        assert st == A.ARNQ_OK
        after += [lib.quant_matmul(x, sx, w, sw) for _ in range(4)]
    torch.cuda.synchronize()
    assert lib.workspace_status(ws) == (A.ARNQ_ERR_DEVICE_TIMEOUT, -1)
    for v in after:
        assert torch.equal(v, ref)


@pytest.mark.parametrize("m", [256, 512, 768, 300, 1100])
@pytest.mark.parametrize("n", [256 * 73, 256 * 74, 256 * 75])
@pytest.mark.parametrize("k", [128, 1024])
def test_signals_between_the_pairs_ctas_at_their_end(m, n, k):
    # one to five tiles a pair, the next kernel's barriers right behind them in the same memory
    c, d = case(m, n, k, seed=1), case(16, 512, 512, seed=2)
    rc, status = planned(c, kernel=2)
    check(*c, rc)
    rd = lib.quant_matmul(*d[:4])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x, sx, w, sw, _ = c
    plan, ys, others = A.arnq_matmul_plan(kernel=2), [], []
    for _ in range(6):
        ys.append(torch.empty(m, n, dtype=torch.float32, device="cuda"))
        st = A.arnq_quant_matmul_planned(x, sx, w, sw, None, m, n, k, A.ARNQ_FP32, ys[-1], ws, 256,
                                         torch.cuda.current_stream(), plan)
        assert st == A.ARNQ_OK
        others.append(lib.quant_matmul(*d[:4]))
    torch.cuda.synchronize()
    assert status[0] == 0 and lib.workspace_status(ws)[0] == 0
    for y, o in zip(ys, others):
        assert torch.equal(y, rc) and torch.equal(o, rd)

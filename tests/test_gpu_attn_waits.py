"""The attention kernels' waits are bounded: one that runs out ends the call with a status, and the next call is right."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, attention_ref, strided_rows
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("stage", [1, 2, 3])
@pytest.mark.parametrize("G,n,D,e4m3", [(3, 1, 128, False), (8, 4, 256, True), (8, 40, 128, False), (8, 40, 64, True),
                                        (16, 2, 64, True), (8, 9, 256, False)])
def test_a_wait_that_runs_out(G, n, D, e4m3, stage):
    # tiles enough a run that its ring wraps; last pages half full of NaN, and a page that is not there
    P = Paged([60000, 50001, 40100], [n, n, n], 1, D, 64, e4m3, seed=D, lead=2, tail=3)
    q = strided_rows(P.T, G, D, 0, torch.Generator().manual_seed(G)).contiguous()
    pages, bt = P.device()
    ws, qd = moe.AttnWorkspace(G, 1, D), q.cuda()
    o = torch.full((P.T, G, D), 9.0, dtype=torch.bfloat16, device="cuda")
    before = [p.view(torch.uint8 if e4m3 else torch.int16).clone() for p in (P.dk, P.dv)]
    ws.set_wait_test(stage)
    gone = bt.page_table.clone()
    gone[1, 50000 // 64] = -1
    moe.moe_paged_attention(pages, moe.KvBatch(bt.q_start, bt.kv_len, gone, P.T, n), qd, o, ws, D ** -0.5)
    assert moe.moe_attn_sync_status(ws) in (moe.MOE_ETIMEOUT, moe.MOE_ERANGE)  # the first of the two counts
    moe.moe_paged_attention(pages, bt, qd, o, ws, D ** -0.5)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_ETIMEOUT
    assert (o[:2] == 9).all() and (o[-3:] == 9).all()  # token rows of no request
    assert all(torch.equal(a, p.view(a.dtype)) for a, p in zip(before, (P.dk, P.dv)))
    ws.set_wait_test(0)
    moe.moe_paged_attention(pages, bt, qd, o, ws, D ** -0.5)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    ref, tol = attention_ref(P, q, G, D ** -0.5, 0)
    mine = slice(2, P.T - 3)
    assert ((o[mine].cpu().double() - ref[mine]).abs() <= tol[mine]).all()

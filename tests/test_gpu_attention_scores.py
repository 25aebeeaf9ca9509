"""Scores at the ends of fp32's range in moe_paged_attention."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, attention_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("size", [2.0 ** 34, 2.0 ** 112])
@pytest.mark.parametrize("where", [5, 130, 480])
@pytest.mark.parametrize("G,n", [(4, 1), (8, 4), (8, 20)])
def test_one_score_above_others_far_below(G, n, where, size):
    """Scores of -size and -2 size: the one key with the former takes all of the weight."""
    P = Paged([700], [n], 1, 128, 32, seed=n)
    P.k.fill_(-2.0)
    P.k[int(P.table[0, where // 32]), 0, where % 32] = -1.0
    q = torch.full((n, G, 128), 2.0 ** 60, dtype=torch.bfloat16)
    pages, bt = P.device()
    ws, o = moe.AttnWorkspace(G, 1, 128), torch.zeros(n, G, 128, dtype=torch.bfloat16, device="cuda")
    moe.moe_paged_attention(pages, bt, q.cuda(), o, ws, size * 2.0 ** -67)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    want = P.rows("v", 0, 0)[where]
    assert (o.cpu().double() == want).all()


@pytest.mark.parametrize("n", [3, 40])
def test_rows_that_see_nothing_are_zeros_still(n):
    P = Paged([2], [n], 1, 64, 16)
    q = torch.randn(n, 4, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    pages, bt = P.device()
    ws, o = moe.AttnWorkspace(4, 1, 64), torch.full((n, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_paged_attention(pages, bt, q.cuda(), o, ws, 0.125)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    o = o.cpu().double()
    assert (o[:n - 2] == 0).all()
    ref, tol = attention_ref(P, q, 4, 0.125, 0)
    assert ((o - ref).abs() <= tol)[n - 2:].all()

"""Scores at the ends of fp32's range in moe_paged_attention."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, U_BF16, U_F32, attention_ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("size", [s * 2.0 ** e for s in (1, -1) for e in (-30, 12, 15, 17, 18, 19, 21, 24, 26, 28)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,L,window", [(4, 1, 300, 0), (4, 1, 9000, 0), (8, 4, 700, 0), (8, 3, 700, 150), (8, 20, 900, 0),
                                          (8, 20, 900, 200)])
def test_equal_scores_of_any_size(G, n, L, window, D, e4m3, size):
    """Every score of a call is the same, of any size up to 2^29: plain means of the values."""
    P = Paged([L], [n], 1, D, 32, e4m3, seed=D)
    P.k.fill_(-1.375)
    kk = float(P.rows("k", 0, 0)[0, 0])
    assert (P.rows("k", 0, 0) == kk).all() and kk < 0
    # D products of q and k: exact in fp32, as every size is a power of two times 11 (E4M3 scales: one rounding, the same for all)
    q = torch.full((n, G, D), 2.0 ** 60, dtype=torch.bfloat16)
    scale = -size * 2.0 ** -60 / D / (2.0 if e4m3 else 1.0)
    pages, bt = P.device()
    ws, o = moe.AttnWorkspace(G, 1, D), torch.zeros(n, G, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_paged_attention(pages, bt, q.cuda(), o, ws, scale, window)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    v = P.rows("v", 0, 0)
    for i in range(n):
        at = L - n + i
        seen = v[max(0, at - window + 1) if window else 0:at + 1]
        mean, mag = seen.mean(0), seen.abs().mean(0)
        # one weight for all, rounded to bf16; fp32 sums of as many terms, the division, one rounding
        tol = 2 * U_BF16 * mean.abs() * (1 + 2.0 ** -8) + 4 * len(seen) * U_F32 * mag
        assert ((o[i].cpu().double() - mean).abs() <= tol).all(), i


@pytest.mark.parametrize("size", [2.0 ** 34, 2.0 ** 112])
@pytest.mark.parametrize("where", [5, 130, 480])
@pytest.mark.parametrize("G,n", [(4, 1), (8, 4), (8, 20)])
def test_one_score_above_others_far_below(G, n, where, size):
    """Scores of -size and -2 size: the one key with the former takes all of the weight.  (Products that fp32 holds
    exactly, so that no size is too large.)"""
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

"""What must not reach a row of moe_paged_attention: rows of other requests, and what a tile of rows holds beside them."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, attention_ref, strided_rows
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def attend(P, q, G, window=0):
    pages, bt = P.device()
    ws, o = moe.AttnWorkspace(G * P.Hkv, P.Hkv, P.D), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    moe.moe_paged_attention(pages, bt, q.cuda(), o, ws, P.D ** -0.5, window)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    return o.cpu()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(1, 1), (3, 1), (5, 2), (7, 1), (8, 3), (20, 1), (8, 20)])
def test_rows_of_other_requests(G, n, D, e4m3):
    """A neighbour's scores, however peaked, change no bit of a request's rows.  (Keys enough for several tiles a run.)"""
    P = Paged([40000, 39000, 38000], [n] * 3, 1, D, 32, e4m3, seed=G, lead=1, tail=2)
    q = strided_rows(P.T, G, D, 0, torch.Generator().manual_seed(D + G)).contiguous()
    first = attend(P, q, G)
    rows = slice(1 + n, 1 + 2 * n)  # the second request's
    for other in (slice(1, 1 + n), slice(1 + 2 * n, P.T)):
        for times in (60.0, 1e30):
            p = q.clone()
            p[other] *= times
            assert torch.equal(attend(P, p, G)[rows], first[rows]), (other, times)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [3, 5, 6, 7, 9])
def test_what_other_calls_left_in_shared_memory(G, D):
    """Rows of a tile that are nobody's hold what the call before had there."""
    last = Paged([60000, 50000], [1, 1], 1, D, 64, seed=G)
    long = Paged([60000], [1], 2, D, 64, seed=G + 1)
    q = strided_rows(2, G, D, 0, torch.Generator().manual_seed(G)).contiguous()
    full = torch.randn(1, 32, D, generator=torch.Generator().manual_seed(D)).to(torch.bfloat16)
    (lp, lb), (fp, fb) = last.device(), long.device()
    lw, fw = moe.AttnWorkspace(G, 1, D), moe.AttnWorkspace(32, 2, D)
    qd, fo, outs = q.cuda(), torch.empty(1, 32, D, dtype=torch.bfloat16, device="cuda"), []
    for times in (0.0, 60.0, 1e30):
        fd, o = (full * times).cuda(), torch.zeros_like(qd)
        torch.cuda.synchronize()
        moe.moe_paged_attention(fp, fb, fd, fo, fw, D ** -0.5)  # 16 rows a tile, on every SM
        moe.moe_paged_attention(lp, lb, qd, o, lw, D ** -0.5)   # nothing between the two
        assert moe.moe_attn_sync_status(lw) == moe.MOE_OK
        outs.append(o.cpu())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    ref, tol = attention_ref(last, q, G, D ** -0.5, 0)
    assert ((outs[0].double() - ref).abs() <= tol).all()

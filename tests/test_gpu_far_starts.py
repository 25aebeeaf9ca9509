"""Starts of requests far below the call's rows, where the difference of two leaves 32 bits: reported, and nothing astray."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, strided_rows
from tests.gpu_util import require_gpu
from tests.test_gpu_kv_move import pools

pytestmark = pytest.mark.gpu
FAR = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 7, -2 ** 30, -1]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(far):
    """Requests of rows 0..3 and of none that are: the second one's end is far below its beginning."""
    return i32([0, 4, far])


@pytest.mark.parametrize("far", FAR)
def test_masks(far):
    batch = moe.KvBatch(starts(far), i32([0] * 2), i32([[0]] * 2), 12, 4)
    t, err = moe.Tree(batch, i32([-1, 0, 1, 0] + [-1] * 8)), i32([0])
    for x in (t.depth, t.above, t.below):
        x.fill_(77)
    moe.moe_tree_prepare(batch, t, err=err)
    assert err.item() == moe.MOE_ERANGE and t.depth.tolist() == [0, 1, 2, 1] + [77] * 8
    assert t.above[:4, 0].tolist() == [1, 3, 7, 9]
    assert (t.above[4:] == 77).all() and (t.below[4:] == 77).all()


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("drawn", [True, False])
def test_verification(far, drawn):
    batch = moe.KvBatch(starts(far), i32([0] * 2), i32([[0]] * 2), 12, 4)
    row = torch.full((12, 10), 0.1, device="cuda")
    half = torch.full((12,), 0.5, device="cuda")
    d = moe.verify_desc(row, i32([0] * 12), i32([-1] + [0] * 11), half, half[:2].contiguous(), draft=row if drawn else None)
    path, count, token, err = i32([[5] * 3] * 2), i32([5, 5]), i32([5, 5]), i32([0])
    moe.moe_verify_drafts(batch, d, path, count, token, err=err)
    assert err.item() == moe.MOE_ERANGE and count.tolist()[1] == 0 and token.tolist()[1] == -1
    assert path.tolist()[1] == [-1] * 3 and count.tolist()[0] >= 1


@pytest.mark.parametrize("far", FAR)
def test_compaction(far):
    raw, layers = pools(2, 4, 1, 16, 64)
    batch = moe.KvBatch(starts(far), i32([20, 20]), i32([[0, 1], [2, 3]]), 12, 4)
    want = raw.clone()
    want[:, :, 1, :, 1] = raw[:, :, 1, :, 2]  # place 18 to 17
    lens, err = i32([0, 0]), i32([0])
    moe.moe_kv_compact(layers, batch, i32([[0, 2], [0, 2]]), i32([2, 2]), lens, err=err)
    assert err.item() == moe.MOE_ERANGE and lens.tolist() == [18, 20]
    assert torch.equal(raw, want)


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("D,G,n", [(64, 2, 4), (64, 8, 40), (256, 8, 4), (256, 8, 20)])
def test_attention(far, D, G, n):
    P = Paged([100, 90, 80], [n] * 3, 1, D, 16)
    pages, bt = P.device()
    q = strided_rows(P.T, G, D, 0, torch.Generator().manual_seed(0)).contiguous().cuda()
    ws, o = moe.AttnWorkspace(G, 1, D), torch.full((P.T, G, D), 9.0, dtype=torch.bfloat16, device="cuda")
    bad = moe.KvBatch(i32([0, n, far, 3 * n]), bt.kv_len, bt.page_table, P.T, n)
    t = moe.Tree(bt, i32(([-1] + [0] * (n - 1)) * 3))
    moe.moe_tree_prepare(bt, t)
    for call in (lambda b: moe.moe_paged_attention(pages, b, q, o, ws, 0.125), lambda b: moe.moe_tree_attention(pages, b, t, q, o, ws, 0.125)):
        call(bad)
        assert moe.moe_attn_sync_status(ws) == moe.MOE_ERANGE and (o == 9).all()
    call(bt)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK and (o != 9).any(2).all()

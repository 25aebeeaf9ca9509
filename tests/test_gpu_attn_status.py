"""moe_attn_sync_status waits for its stream and no other, and resets the word there."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, strided_rows
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def test_status_of_a_stream_beside_a_busy_default_stream():
    P = Paged([64, 30], [1, 1], 1, 64, 16, table_extra=0)
    P.table[0, 1] = -1  # MOE_ERANGE
    q = strided_rows(2, 2, 64, 0, torch.Generator().manual_seed(0)).contiguous().cuda()
    pages, bt = P.device()
    good = moe.KvBatch(bt.q_start, bt.kv_len, bt.page_table.clamp(min=0), P.T, 1)
    ws, o = moe.AttnWorkspace(2, 1, 64), torch.empty_like(q)
    side, busy = torch.cuda.Stream(), torch.cuda.Event()
    big = torch.ones(1 << 30, dtype=torch.int8, device="cuda")
    big.add_(1)
    moe.moe_paged_attention(pages, good, q, o, ws, 0.125)  # first-call set-up
    torch.cuda.synchronize()
    for _ in range(600):  # about a quarter of a second on the default stream
        big.add_(1)
    busy.record()
    with torch.cuda.stream(side):
        for _ in range(5):
            moe.moe_paged_attention(pages, bt, q, o, ws, 0.125)
            assert moe.moe_attn_sync_status(ws) == moe.MOE_ERANGE
            moe.moe_paged_attention(pages, good, q, o, ws, 0.125)
            assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    assert not busy.query()  # the default stream is still at work: neither the copy nor the reset went through it
    torch.cuda.synchronize()


@pytest.mark.parametrize("G,n", [(2, 4), (8, 40)])
def test_request_starts_that_decrease_are_reported(G, n):
    """Nothing is computed: the schedule's count holds rows of requests that follow one another."""
    P = Paged([100, 90, 80], [n, n, n], 1, 64, 16)
    pages, bt = P.device()
    q = strided_rows(P.T, G, 64, 0, torch.Generator().manual_seed(0)).contiguous().cuda()
    ws, o = moe.AttnWorkspace(G, 1, 64), torch.full((P.T, G, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 2 * n, n, 3 * n], dtype=torch.int32).cuda()
    moe.moe_paged_attention(pages, moe.KvBatch(start, bt.kv_len, bt.page_table, P.T, n), q, o, ws, 0.125)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_ERANGE
    assert (o == 9).all()
    moe.moe_paged_attention(pages, bt, q, o, ws, 0.125)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    assert (o != 9).any(2).all()

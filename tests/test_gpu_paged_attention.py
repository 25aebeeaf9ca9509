"""moe_paged_attention against softmax attention in 64 bits."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, attention_ref, strided_rows
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def on_device(x):
    return torch.as_strided((x._base if x._base is not None else x).cuda(), x.shape, x.stride(), x.storage_offset())


def run(P, q, Hq, scale, window, pad=0, ws=None, status=moe.MOE_OK):
    pages, bt = P.device()
    ws = ws or moe.AttnWorkspace(Hq, P.Hkv, P.D)
    base = torch.full((P.T, Hq * P.D + pad), 9.0, dtype=torch.bfloat16, device="cuda")
    o = base[:, :Hq * P.D].unflatten(1, (Hq, P.D))
    moe.moe_paged_attention(pages, bt, on_device(q), o, ws, scale, window)
    assert moe.moe_attn_sync_status(ws) == status
    assert (base[:, Hq * P.D:] == 9).all()
    return o


def check(P, Hq, window=0, q_std=1.0, pad=0, seed=3, scale=None):
    q = strided_rows(P.T, Hq, P.D, pad, torch.Generator().manual_seed(seed), q_std)
    scale = P.D ** -0.5 if scale is None else scale
    o = run(P, q, Hq, scale, window, pad).cpu().double()
    ref, tol = attention_ref(P, q, Hq, scale, window)
    none = ref.isnan()
    assert (o[none] == 9).all()  # token rows of no request
    bad = ((o - ref).abs() > tol) & ~none
    assert not (bad | (o.isnan() & ~none)).any(), (int(bad.sum()), float((o - ref).abs()[~none].max()))


CASES = [
    # lens, new, Hq, Hkv, D, page, window, e4m3, layout
    ([1], [1], 1, 1, 64, 16, 0, False, "hnd"),
    ([127], [1], 8, 1, 128, 16, 0, False, "hnd"),
    ([128], [1], 8, 2, 128, 128, 0, False, "nhd"),
    ([129], [4], 16, 2, 256, 64, 0, False, "hnd"),
    ([717], [4], 16, 2, 256, 64, 0, True, "kv"),
    ([5, 0, 260, 1, 128], [5, 0, 2, 1, 16], 4, 4, 64, 32, 0, False, "kv"),
    ([3, 400, 255, 256, 257], [1] * 5, 12, 4, 128, 16, 0, True, "nhd"),
    ([700, 40], [16, 16], 16, 1, 64, 8, 0, False, "hnd"),
    ([530], [130], 8, 1, 128, 64, 0, False, "hnd"),
    ([300, 290], [37, 211], 6, 2, 256, 1, 0, True, "hnd"),
    ([2000], [1], 64, 1, 64, 64, 0, False, "nhd"),
    ([1000, 90, 33], [1, 1, 1], 24, 8, 64, 32, 100, False, "hnd"),
    ([1000, 700], [9, 200], 4, 1, 128, 16, 50, False, "kv"),
    ([640], [3], 8, 2, 256, 64, 1, True, "hnd"),
    ([200, 300], [2, 2], 10, 2, 128, 32, 128, False, "hnd"),
    ([9000], [1], 4, 1, 128, 64, 0, False, "hnd"),
    ([9001], [4], 8, 1, 256, 64, 0, True, "hnd"),
    ([9000], [1], 12, 1, 256, 64, 0, False, "hnd"),
    ([30000], [1], 10, 1, 256, 64, 0, True, "kv"),
    ([30011], [2], 12, 2, 64, 64, 0, False, "nhd"),
    ([300, 131], [1, 3], 8, 2, 64, 2, 0, True, "hnd"),
    ([300, 131], [50, 9], 16, 2, 64, 2, 0, True, "hnd"),
    ([300, 131], [1, 4], 8, 2, 64, 8, 90, True, "nhd"),
    ([257, 140], [2, 1], 8, 2, 128, 1, 0, True, "kv"),
    ([257, 140], [70, 1], 8, 1, 128, 1, 33, True, "hnd"),
    ([7, 130, 12, 300, 1, 64, 90, 2] * 20, [1, 4, 2, 1, 1, 3, 1, 2] * 20, 8, 2, 64, 16, 0, False, "hnd"),
]


@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,page,window,e4m3,layout", CASES)
def test_attention(lens, ns, Hq, Hkv, D, page, window, e4m3, layout):
    check(Paged(lens, ns, Hkv, D, page, e4m3, layout, lead=1, tail=2), Hq, window, pad=8)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(1, 1), (3, 5), (8, 2), (5, 7), (16, 4), (16, 9), (33, 1), (7, 40)])
def test_every_tile_shape(G, n, D, e4m3):
    check(Paged([n + 400, n + 3], [n, n], 2, D, 16, e4m3, seed=G), 2 * G)


@pytest.mark.parametrize("e4m3", [False, True])
def test_peaked_scores(e4m3):
    """Large scores: most weights vanish, the running maximum moves often."""
    check(Paged([1500, 300], [4, 2], 2, 128, 32, e4m3, seed=8, k_std=3.0), 16, q_std=8.0)


@pytest.mark.parametrize("G,n", [(4, 1), (8, 7)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_of_any_size_against_e4m3_keys(D, G, n):
    """Rows from 2^-125 up to 2^12 and zeros, columns 20 powers of two apart; infinities and NaN stay in their rows."""
    g = torch.Generator().manual_seed(D + G)
    P = Paged([700, 333], [n, n], 2, D, 32, True, seed=D)
    q = strided_rows(P.T, 2 * G, D, 8, g)
    q *= (2.0 ** -torch.randint(0, 21, (P.T, 1, D), generator=g)).to(torch.bfloat16)
    size = torch.tensor([0, 12, -30, -64, -112, -125, -3, 8])
    q *= (2.0 ** size[torch.randint(0, 8, (P.T, 2 * G, 1), generator=g)].double()).float().to(torch.bfloat16)
    q[0, 0] = 0
    q[0, 1, 5] = float("inf")
    q[1, 2, 7] = float("nan")
    scale = D ** -0.5
    o = run(P, q, 2 * G, scale, 0, 8).cpu().double()
    ref, tol = attention_ref(P, q, 2 * G, scale, 0)
    assert o[0, 1].isnan().all() and o[1, 2].isnan().all()
    fine = torch.ones(P.T, 2 * G, dtype=torch.bool)
    fine[0, 1] = fine[1, 2] = False
    # a column is off by 2^-22 of its row's largest at most; its score then by that of sum |k|, and a
    # weight by twice the largest such; rows below 2^-103 score less than 2^-90 and count as zeros
    for b in range(2):
        for h in range(2):
            k, v = P.rows("k", b, h).abs().sum(1).max(), P.rows("v", b, h).abs().amax(0)
            rows, heads = slice(b * n, (b + 1) * n), slice(h * G, (h + 1) * G)
            most = q[rows, heads].double().abs().amax(-1, keepdim=True)
            tol[rows, heads] += 2 * 2.0 ** -22 * most * k * scale * v
    assert ((o - ref).abs() <= tol)[fine].all()


def test_scores_that_rise_along_the_cache():
    P = Paged([1200], [1], 1, 64, 16)
    for j in range(1200):  # key j scores about j / 16
        P.k[int(P.table[0, j // 16]), 0, j % 16] = j / 16
    q = torch.full((1, 2, 64), 1 / 64, dtype=torch.bfloat16)
    o = run(P, q, 2, 1.0, 0).cpu().double()
    ref, tol = attention_ref(P, q, 2, 1.0, 0)
    assert ((o - ref).abs() <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,n", [(4, 1), (8, 4), (8, 7)])
@pytest.mark.parametrize("D", [64, 256])
def test_many_units_of_many_tiles_beside_junk(D, G, n, e4m3):
    """Every run passes several ends of requests, whose last pages hold NaN, with its rings full."""
    g = torch.Generator().manual_seed(D + n)
    lens = [int(x) for x in torch.exp(torch.rand(24, generator=g) * 3.5 + 5.3)]  # 200 .. 6600
    ns = [int(x) for x in torch.randint(1, n + 1, (24,), generator=g)]
    P = Paged(lens, ns, 2, D, 64, e4m3, seed=n)
    q = strided_rows(P.T, 2 * G, D, 0, g)
    ref, tol = attention_ref(P, q, 2 * G, D ** -0.5, 0)
    pages, bt = P.device()
    ws, qd = moe.AttnWorkspace(2 * G, 2, D), q.cuda()
    for _ in range(5):
        o = torch.empty_like(qd)
        moe.moe_paged_attention(pages, bt, qd, o, ws, D ** -0.5)
        assert ((o.cpu().double() - ref).abs() <= tol).all()
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("n", [3, 50])
def test_any_scale(scale, n):
    check(Paged([300], [n], 1, 128, 16), 8, scale=scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 20, 64])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("e4m3", [False, True])
def test_chunks(D, G, window, e4m3):
    """Row tiles of two 128s: whole and ragged ones, one of the two empty, several units and splits."""
    per = 128 // G
    ns = [2 * per, per + 1, per, 4 * per + 3, 1]
    lens = [n + e for n, e in zip(ns, [700, 0, 129, 1300, 255])]
    check(Paged(lens, ns, 2, D, 32, e4m3, lead=3, seed=G), 2 * G, window)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunks_with_peaked_scores(e4m3):
    check(Paged([900, 600], [90, 300], 2, 128, 32, e4m3, seed=8, k_std=3.0), 16, q_std=8.0)


@pytest.mark.parametrize("value,e4m3", [(float("nan"), False), (float("inf"), False), (float("nan"), True)])
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("D", [64, 128])
def test_what_a_chunk_s_token_does_not_see_does_not_reach_it(value, window, D, e4m3):
    P = Paged([300], [100], 1, D, 16, e4m3)  # positions 200 .. 299, 8 heads: rows of both tiles
    for at in (250, 299, 130):
        P.v[int(P.table[0, at // 16]), 0, at % 16, at % D] = value
    q = strided_rows(P.T, 8, D, 0, torch.Generator().manual_seed(0))
    o = run(P, q, 8, 0.1, window).cpu().double()
    ref, tol = attention_ref(P, q, 8, 0.1, window)
    near = (o - ref).abs() <= tol
    for at in (250, 299, 130):
        rows = [i for i in range(100) if at <= 200 + i and not (window and at <= 200 + i - window)]
        others = [i for i in range(100) if i not in rows]
        assert near[others][..., at % D].all()
        if rows:
            assert not o[rows][..., at % D].isfinite().any()
    clean = torch.ones(D, dtype=torch.bool)
    clean[[at % D for at in (250, 299, 130)]] = False
    assert near[..., clean].all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunks_give_the_same_bits_every_time(e4m3):
    P = Paged([4000, 500], [333, 200], 2, 128, 64, e4m3)
    pages, bt = P.device()
    q = strided_rows(P.T, 16, 128, 0, torch.Generator().manual_seed(0)).cuda()
    ws, first, o = moe.AttnWorkspace(16, 2, 128), torch.empty_like(q), torch.empty_like(q)
    moe.moe_paged_attention(pages, bt, q, first, ws, 0.1)
    for _ in range(10):
        moe.moe_paged_attention(pages, bt, q, o, ws, 0.1)
        assert torch.equal(o, first)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_sharp_first_key_and_a_long_flat_rest(e4m3):
    """One key takes most of the weight and thousands share what is left."""
    P = Paged([8000], [1], 1, 64, 64, e4m3, seed=2, k_std=0.05)
    P.k[int(P.table[0, 0]), 0, 0] = torch.full((64,), 1.25).to(P.k.dtype)
    q = torch.ones(1, 4, 64, dtype=torch.bfloat16)
    scale = 0.12  # key 0 scores about 9.6
    o = run(P, q, 4, scale, 0).cpu().double()
    ref, tol = attention_ref(P, q, 4, scale, 0)
    assert ((o - ref).abs() <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_new_tokens_beyond_the_cache_see_nothing(e4m3):
    """kv_len smaller than the new tokens: the first of them are at negative positions."""
    P = Paged([2, 0, 5], [5, 3, 5], 1, 64, 16, e4m3)
    q = strided_rows(P.T, 4, 64, 0, torch.Generator().manual_seed(0))
    o = run(P, q, 4, 0.125, 0).cpu().double()
    ref, tol = attention_ref(P, q, 4, 0.125, 0)
    empty = [0, 1, 2, 5, 6, 7]
    assert (o[empty] == 0).all()
    rest = [3, 4] + list(range(8, 13))
    assert ((o - ref).abs() <= tol)[rest].all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 30])
def test_what_a_token_does_not_see_does_not_reach_it(value, window):
    """A later token's key and value, and a value that has left the window, are not finite."""
    P = Paged([150], [6], 1, 128, 16)
    page, at = int(P.table[0, 147 // 16]), 147 % 16  # the position of the fourth new token
    P.k[page, 0, at], P.v[page, 0, at, 5] = value, value
    if window:
        P.v[int(P.table[0, 116 // 16]), 0, 116 % 16, 7] = value  # in the window of 144 and 145 only
    q = strided_rows(P.T, 8, 128, 0, torch.Generator().manual_seed(0))
    o = run(P, q, 8, 0.1, window).cpu().double()
    ref, tol = attention_ref(P, q, 8, 0.1, window)
    clean = [2] if window else [0, 1, 2]
    assert ((o - ref).abs() <= tol)[clean].all()
    if window:
        other = [d for d in range(128) if d != 7]
        assert ((o - ref).abs() <= tol)[:2][..., other].all()
        assert not o[:2, :, 7].isfinite().any()
    assert o[3:, :, 5].isnan().all()


def test_pages_before_the_window_may_be_gone():
    P = Paged([1000], [2], 2, 64, 16)
    q = strided_rows(2, 4, 64, 0, torch.Generator().manual_seed(0))
    ref, tol = attention_ref(P, q, 4, 0.125, 100)
    P.table[0, :(998 - 99) // 16] = -1  # the first visible position is 998 - 99
    o = run(P, q, 4, 0.125, 100).cpu().double()
    assert ((o - ref).abs() <= tol).all()


@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_a_bad_page_reads_as_zeros_and_is_reported(bad):
    P = Paged([300, 200], [1, 1], 1, 64, 16)
    q = strided_rows(2, 2, 64, 0, torch.Generator().manual_seed(0))
    for j in range(32, 48):
        P.k[int(P.table[0, 2]), 0, j - 32] = 0
        P.v[int(P.table[0, 2]), 0, j - 32] = 0
    ref, tol = attention_ref(P, q, 2, 0.125, 0)
    P.table[0, 2] = bad
    o = run(P, q, 2, 0.125, 0, status=moe.MOE_ERANGE).cpu().double()
    assert ((o - ref).abs() <= tol).all()


def test_a_length_beyond_the_table_is_cut_and_reported():
    P = Paged([64, 30], [1, 1], 1, 64, 16, table_extra=0)
    q = strided_rows(2, 2, 64, 0, torch.Generator().manual_seed(0))
    ref, tol = attention_ref(P, q, 2, 0.125, 0)
    P.lens[0] = 1 << 30
    o = run(P, q, 2, 0.125, 0, status=moe.MOE_ERANGE).cpu().double()
    assert ((o - ref).abs() <= tol).all()


def test_offsets_past_32_bits():
    """Pages more than 2^32 bytes into the pool."""
    D, page, npages = 256, 64, 160000  # 5.2 GB a pool
    k = torch.zeros(npages, 1, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    P = Paged([200], [1], 1, D, page, table_extra=0)
    far = torch.tensor([npages - 1, 3, npages - 2, 140001])
    for i in range(4):
        k[far[i]], v[far[i]] = P.k[int(P.table[0, i])].cuda(), P.v[int(P.table[0, i])].cuda()
    q = strided_rows(1, 4, D, 0, torch.Generator().manual_seed(0))
    ref, tol = attention_ref(P, q, 4, 0.06, 0)
    ws, o = moe.AttnWorkspace(4, 1, D), torch.empty(1, 4, D, dtype=torch.bfloat16, device="cuda")
    bt = moe.KvBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([200], dtype=torch.int32).cuda(),
                     far.int().view(1, 4).cuda(), 1, 1)
    moe.moe_paged_attention(moe.KvPages(k, v), bt, q.cuda(), o, ws, 0.06)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    assert ((o.cpu().double() - ref).abs() <= tol).all()


def test_the_same_bits_every_time_on_any_stream_and_in_a_graph():
    P = Paged([3000, 17, 900], [1, 4, 2], 2, 128, 32)
    pages, bt = P.device()
    q = strided_rows(P.T, 16, 128, 0, torch.Generator().manual_seed(0)).cuda()
    ws = moe.AttnWorkspace(16, 2, 128)
    first = torch.empty_like(q)
    moe.moe_paged_attention(pages, bt, q, first, ws, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = torch.empty_like(q)
    with torch.cuda.stream(s):
        for _ in range(20):
            moe.moe_paged_attention(pages, bt, q, o, ws, 0.1)
        s.synchronize()
        assert torch.equal(o, first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            moe.moe_paged_attention(pages, bt, q, o, ws, 0.1)
        o.zero_()
        graph.replay()
        s.synchronize()
        assert torch.equal(o, first)
        # a replay reads the lengths of its time
        bt.kv_len.copy_(torch.tensor([2999, 16, 899], dtype=torch.int32))
        graph.replay()
        s.synchronize()
    P.lens = [2999, 16, 899]
    ref, tol = attention_ref(P, q.cpu(), 16, 0.1, 0)
    assert ((o.cpu().double() - ref).abs() <= tol).all()
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK


def test_max_n_does_not_change_the_result():
    P = Paged([200, 300], [1, 6], 1, 128, 16)
    pages, bt = P.device()
    q = strided_rows(P.T, 8, 128, 0, torch.Generator().manual_seed(0))
    ref, tol = attention_ref(P, q, 8, 0.1, 0)
    ws = moe.AttnWorkspace(8, 1, 128)
    for max_n in (0, 1, 6, 64, 100000):
        bt.c.max_n = max_n
        o = torch.zeros(P.T, 8, 128, dtype=torch.bfloat16, device="cuda")
        moe.moe_paged_attention(pages, bt, q.cuda(), o, ws, 0.1)
        assert ((o.cpu().double() - ref).abs() <= tol).all()


def test_refusals_with_a_workspace():
    P = Paged([20], [1], 2, 64, 16)
    pages, bt = P.device()
    ws = moe.AttnWorkspace(4, 2, 64)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1.0, window=-1)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_paged_attention(pages, bt, q, torch.empty_like(q), ws, **kw)
        assert e.value.code == moe.MOE_EINVAL
    for other in (moe.AttnWorkspace(4, 1, 64), moe.AttnWorkspace(4, 2, 128)):
        with pytest.raises((moe.MoeError, ValueError)):
            moe.moe_paged_attention(pages, bt, q, torch.empty_like(q), other, 1.0)


def test_sizes_past_the_schedule_s_count_are_refused():
    k = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(1, 1024, 1, 64).contiguous()
    q = torch.zeros(64, 1024, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 1 << 24, dtype=torch.int32, device="cuda")
    ws = moe.AttnWorkspace(1024, 1024, 64)
    bt = moe.KvBatch(torch.tensor([0, 64], dtype=torch.int32).cuda(), torch.tensor([64], dtype=torch.int32).cuda(), table,
                     64, 64)
    pages = moe.KvPages(k, k)
    moe.moe_paged_attention(pages, bt, q, torch.empty_like(q), ws, 1.0)  # 2^24 tokens: within the count
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    c = pages.c
    c.page, c.head_stride, c.tok_stride = 1 << 15, 64, 64 * 1024  # 2^39 tokens a table: refused before any launch
    with pytest.raises(moe.MoeError) as e:
        moe.moe_paged_attention(pages, bt, q, torch.empty_like(q), ws, 1.0)
    assert e.value.code == moe.MOE_EINVAL


@pytest.mark.parametrize("n", [2, 80])
def test_a_window_that_holds_everything(n):
    P = Paged([300], [n], 1, 64, 16)
    q = strided_rows(n, 8, 64, 0, torch.Generator().manual_seed(0))
    assert torch.equal(run(P, q, 8, 0.1, 0), run(P, q, 8, 0.1, (1 << 31) - 1))
    assert torch.equal(run(P, q, 8, 0.1, 0), run(P, q, 8, 0.1, 300))

"""Attention of drafted trees over a paged cache against a 64-bit softmax over each node's own keys."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import Paged, strided_rows
from tests.gpu_util import require_gpu
from tests.tree_util import random_parents, rows_of, sees, tree_attention_ref, tree_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def attend(P, parents, G, window=0, scale=None, q=None, pad=0, seed=0, spoil=None):
    """(o, ref, bound, error): o on the CPU, rows of no request as they were (7)."""
    Hq = G * P.Hkv
    g = torch.Generator().manual_seed(seed + 5)
    q = strided_rows(P.T, Hq, P.D, pad, g) if q is None else q
    scale = P.D ** -0.5 if scale is None else scale
    pages, batch = P.device()
    ws = moe.AttnWorkspace(Hq, P.Hkv, P.D)
    tree = tree_of(P, batch, parents)
    o = torch.full((P.T, Hq, P.D), 7.0, dtype=torch.bfloat16, device="cuda")
    qd = torch.empty(P.T, Hq * P.D + pad, dtype=torch.bfloat16, device="cuda")[:, :Hq * P.D].unflatten(1, (Hq, P.D))
    qd.copy_(q)
    moe.moe_tree_attention(pages, batch, tree, qd, o, ws, scale=scale, window=window)
    err = moe.moe_attn_sync_status(ws)
    ref, tol = tree_attention_ref(P, q, Hq, scale, window, parents)
    return o.cpu().double(), ref, tol, err


def check(o, ref, tol):
    mine = ~torch.isnan(ref[:, 0, 0])
    bad = (o[mine] - ref[mine]).abs() / tol[mine]
    assert torch.isfinite(o[mine]).all()
    assert bad.max() <= 1.0 if bad.numel() else True, float(bad.max())
    assert (o[~mine] == 7.0).all()


CASES = [
    # D, Hkv, G, page, lens, ns, spread, window
    (128, 2, 4, 16, [40], [4], 2, 0),                      # 16 rows, inside one tile
    (128, 2, 4, 16, [300, 133], [8, 5], 3, 0),             # 32 rows, the tree over a tile's end
    (128, 1, 8, 32, [1000, 7], [8, 7], 4, 0),              # 64 rows; a request that is its tree alone
    (128, 2, 8, 64, [700, 40, 129], [40, 33, 1], 6, 0),    # the two 128-row tiles
    (128, 1, 3, 16, [500], [100], 9, 0),                   # heads that do not fill a tile
    (64, 3, 5, 16, [257, 90], [3, 2], 2, 0),
    (64, 2, 2, 128, [1000], [200], 12, 0),
    (64, 1, 1, 32, [600, 256], [256, 256], 20, 0),         # 256 nodes, one of them without a prefix
    (64, 1, 64, 16, [200], [6], 2, 0),                     # a token a tile
    (256, 2, 8, 64, [717], [8], 4, 0),
    (256, 1, 2, 16, [300, 64], [64, 64], 8, 0),
    (256, 1, 16, 32, [130], [1], 1, 0),                    # one node
    (128, 2, 4, 16, [900, 500], [8, 16], 1, 0),            # chains
    (128, 2, 4, 16, [900, 500, 60], [8, 16, 12], 3, 200),  # windows
    (128, 1, 8, 16, [900, 300], [64, 40], 5, 100),
    (128, 1, 8, 16, [400, 300], [64, 40], 2, 5),           # windows smaller than the tree is deep
    (64, 2, 3, 32, [2000, 100], [12, 12], 2, 3),
    (256, 1, 4, 64, [600], [50], 2, 4),
    (128, 2, 2, 16, [300, 20], [10, 10], 3, 1),            # each node itself alone
    (128, 1, 4, 1, [70], [9], 3, 0),                       # pages of one token
    (64, 1, 8, 2, [150], [30], 4, 0),
    (256, 1, 3, 16, [500, 200], [100, 40], 9, 0),          # one 128-row tile of 42 tokens
    (256, 2, 64, 32, [300, 7], [3, 7], 2, 0),              # two tokens a tile
    (256, 1, 8, 64, [1000, 256, 129], [256, 256, 9], 20, 0),
    (256, 2, 8, 16, [900, 300, 40], [40, 33, 20], 5, 100),
    (256, 1, 8, 1, [140], [20], 1, 0),                     # pages of one token
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,Hkv,G,page,lens,ns,spread,window", CASES)
def test_trees(D, Hkv, G, page, lens, ns, spread, window, e4m3):
    if e4m3 and D * page < 128:
        pytest.skip("a page of 8-bit keys fills a line")
    P = Paged(lens, ns, Hkv, D, page, e4m3=e4m3, seed=len(lens) + D)
    parents = [random_parents(n, spread, n) for n in ns]
    o, ref, tol, err = attend(P, parents, G, window)
    assert err == 0
    check(o, ref, tol)


@pytest.mark.parametrize("layout", ["nhd", "kv"])
def test_layouts_strides_and_rows_of_nobody(layout):
    P = Paged([300, 5, 0, 77], [6, 5, 0, 9], 2, 128, 16, layout=layout, lead=3, tail=4, seed=2)
    parents = [random_parents(n, 3, n) if n else [] for n in P.ns]
    o, ref, tol, err = attend(P, parents, 4, pad=64)
    assert err == 0
    check(o, ref, tol)


@pytest.mark.parametrize("D,G,n", [(128, 2, 6), (128, 8, 40), (64, 8, 30), (256, 4, 10), (256, 8, 40)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_what_a_node_does_not_see_may_be_anything(D, G, n, e4m3):
    """Siblings' keys and values that are NaN or infinite reach only their own descendants."""
    P = Paged([200 + n, n], [n, n], 1, D, 16, e4m3=e4m3, seed=n)
    parents = [random_parents(n, 3, 4)] * 2
    clean = attend(P, parents, G)
    check(*clean[:3])
    for bad in (n // 2, n - 1):
        for b in range(2):
            place = P.lens[b] - n + bad
            for pool in (P.k, P.v):
                raw = pool.view(torch.uint8) if e4m3 else pool
                raw[int(P.table[b, place // 16]), :, place % 16] = 0x7F if e4m3 else float("nan")
    o, _, _, err = attend(P, parents, G)
    assert err == 0
    touched = np.concatenate([sees(parents[0])[:, [n // 2, n - 1]].any(1)] * 2)
    keep = torch.from_numpy(~touched)
    assert (o[keep] == clean[0][keep]).all()
    assert torch.isnan(o[~keep]).all()


@pytest.mark.parametrize("D,G,n", [(128, 2, 6), (128, 8, 40), (64, 2, 7), (256, 8, 40)])
def test_infinite_values_reach_the_nodes_that_see_them(D, G, n):
    P = Paged([150 + n], [n], 1, D, 16, seed=3)
    parents = random_parents(n, 2, 1)
    place = P.lens[0] - n + 2
    P.v[int(P.table[0, place // 16]), 0, place % 16, 5] = float("inf")
    o, _, _, err = attend(P, [parents], G)
    assert err == 0
    below = torch.from_numpy(sees(parents)[:, 2].copy())
    assert torch.isinf(o[below][:, :, 5]).all() and torch.isfinite(o[~below]).all()
    assert torch.isfinite(o[:, :, :5]).all() and torch.isfinite(o[:, :, 6:]).all()


def test_more_tokens_than_the_cache_counts():
    """kv_len below the number of nodes: those before the cache's first place do not exist and see nothing."""
    P = Paged([3, 50], [6, 6], 2, 128, 16, seed=1)
    parents = [[-1, 0, 0, 1, 3, 3], random_parents(6, 2, 0)]
    o, ref, tol, err = attend(P, parents, 4)
    assert err == 0
    check(o, ref, tol)
    assert (o[:3] == 0).all()


def test_forests_see_the_prefix():
    P = Paged([140], [7], 1, 64, 16, seed=4)
    o, ref, tol, err = attend(P, [[-1, -1, 0, 1, -1, 4, 2]], 4)
    assert err == 0
    check(o, ref, tol)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("n,G,D", [(6, 4, 128), (40, 8, 128), (40, 8, 256)])
def test_scales(scale, n, G, D):
    P = Paged([200], [n], 1, D, 16, seed=6)
    o, ref, tol, err = attend(P, [random_parents(n, 4, 2)], G, scale=scale)
    assert err == 0
    check(o, ref, tol)


def test_a_chain_is_paged_attention():
    """Two kernels of one operator: both within the bound, so within two of it of one another."""
    P = Paged([500, 90], [8, 8], 2, 128, 16, seed=8)
    g = torch.Generator().manual_seed(1)
    q = strided_rows(P.T, 8, 128, 0, g)
    o, ref, tol, err = attend(P, [list(range(-1, 7))] * 2, 4, q=q)
    pages, batch = P.device()
    ws = moe.AttnWorkspace(8, 2, 128)
    o2 = torch.empty(P.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    moe.moe_paged_attention(pages, batch, q.cuda(), o2, ws, scale=128 ** -0.5)
    assert ((o - o2.cpu().double()).abs() <= 2 * tol).all()


def test_long_contexts_and_many_requests():
    r = np.random.RandomState(0)
    ns = r.randint(1, 17, 40).tolist()
    P = Paged([int(x) + n for x, n in zip(r.randint(0, 700, 40), ns)], ns, 2, 64, 16, seed=5)
    o, ref, tol, err = attend(P, [random_parents(n, 4, n) for n in ns], 4)
    assert err == 0
    check(o, ref, tol)
    for D in (64, 256):
        P = Paged([9000], [12], 1, D, 64, seed=5)
        o, ref, tol, err = attend(P, [random_parents(12, 4, 0)], 8)
        assert err == 0
        check(o, ref, tol)
    P = Paged([70000, 30000], [30, 9], 1, 256, 64, seed=5)  # rings and schedules that go round
    o, ref, tol, err = attend(P, [random_parents(30, 4, 0), random_parents(9, 2, 0)], 8)
    assert err == 0
    check(o, ref, tol)


def test_masks_of_nothing_read_nothing_astray():
    """A tree that was never prepared has empty masks: a node sees the prefix alone, and nothing is read out of range."""
    P = Paged([100, 40], [5, 30], 1, 128, 16, seed=9)
    pages, batch = P.device()
    ws = moe.AttnWorkspace(4, 1, 128)
    t = moe.Tree(batch, torch.from_numpy(rows_of(P, [[-1] * 5, [-1] * 30])).cuda())
    q = strided_rows(P.T, 4, 128, 0, torch.Generator().manual_seed(0))
    o = torch.empty(P.T, 4, 128, dtype=torch.bfloat16, device="cuda")
    moe.moe_tree_attention(pages, batch, t, q.cuda(), o, ws, scale=0.1)
    assert moe.moe_attn_sync_status(ws) == 0 and torch.isfinite(o).all()


def test_bad_pages_are_reported():
    P = Paged([200], [6], 1, 128, 16, seed=9)
    P.table[0, 3] = P.k.shape[0] + 5
    pages, batch = P.device()
    ws = moe.AttnWorkspace(4, 1, 128)
    t = tree_of(P, batch, [random_parents(6, 2, 0)])
    q = strided_rows(P.T, 4, 128, 0, torch.Generator().manual_seed(0))
    o = torch.empty(P.T, 4, 128, dtype=torch.bfloat16, device="cuda")
    moe.moe_tree_attention(pages, batch, t, q.cuda(), o, ws, scale=0.1)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_ERANGE and torch.isfinite(o).all()


@pytest.mark.parametrize("n,G", [(6, 4), (60, 8)])
def test_a_captured_call_follows_its_tensors(n, G):
    """Captured once with its tree, replayed on other trees and lengths: what a serving loop does."""
    P = Paged([200 + n], [n], 1, 128, 16, seed=1)
    first, second = random_parents(n, 3, 1), random_parents(n, 2, 2)
    g = torch.Generator().manual_seed(2)
    q = strided_rows(P.T, G, 128, 0, g)
    pages, batch = P.device()
    ws = moe.AttnWorkspace(G, 1, 128)
    t = moe.Tree(batch, torch.tensor(first, dtype=torch.int32, device="cuda"))
    qd, o = q.cuda(), torch.empty(P.T, G, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_tree_prepare(batch, t)
        moe.moe_tree_attention(pages, batch, t, qd, o, ws, scale=0.1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            moe.moe_tree_prepare(batch, t)
            moe.moe_tree_attention(pages, batch, t, qd, o, ws, scale=0.1)
    torch.cuda.synchronize()
    for parents, length in ((second, 200 + n), (first, 150 + n), (second, 130 + n)):
        t.parent.copy_(torch.tensor(parents, dtype=torch.int32))
        batch.kv_len.fill_(length)
        P.lens = [length]
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = tree_attention_ref(P, q, G, 0.1, 0, [parents])
        check(o.cpu().double(), ref, tol)
    assert moe.moe_attn_sync_status(ws) == 0


@pytest.mark.parametrize("stage", [1, 2, 3])
@pytest.mark.parametrize("D,G,n,e4m3", [(128, 4, 4, False), (256, 4, 16, True), (128, 8, 40, False), (64, 8, 40, True),
                                        (256, 8, 40, False), (256, 8, 40, True)])
def test_waits_that_run_out_are_reported(stage, D, G, n, e4m3):
    # a slot is waited for from a run's fourth to eighth tile on: 1172 tiles are in at most 304 runs
    P = Paged([60000, 50001, 40100], [n] * 3, 1, D, 64, e4m3=e4m3, seed=1)
    parents = [random_parents(n, 3, b) for b in range(3)]
    q = strided_rows(P.T, G, D, 0, torch.Generator().manual_seed(2))
    pages, batch = P.device()
    ws = moe.AttnWorkspace(G, 1, D)
    t = tree_of(P, batch, parents)
    qd, o = q.cuda(), torch.full((P.T, G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws.set_wait_test(stage)
    moe.moe_tree_attention(pages, batch, t, qd, o, ws, scale=0.1)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_ETIMEOUT
    ws.set_wait_test(0)
    moe.moe_tree_attention(pages, batch, t, qd, o, ws, scale=0.1)
    assert moe.moe_attn_sync_status(ws) == 0
    ref, tol = tree_attention_ref(P, q, G, 0.1, 0, parents)
    check(o.cpu().double(), ref, tol)


@pytest.mark.parametrize("D,G,n", [(128, 4, 6), (128, 8, 40), (256, 8, 20), (64, 8, 40)])
def test_lengths_past_the_table(D, G, n):
    """Keys end where the table does; the nodes past it see those, and the call says so."""
    P = Paged([100], [n], 1, D, 16, seed=2, table_extra=0)
    parents = random_parents(n, 3, 0)
    q = strided_rows(P.T, G, D, 0, torch.Generator().manual_seed(3))
    pages, batch = P.device()
    ws = moe.AttnWorkspace(G, 1, D)
    t = tree_of(P, batch, [parents])
    o = torch.empty(P.T, G, D, dtype=torch.bfloat16, device="cuda")
    cap = P.width * 16
    for pool in (P.dk, P.dv):
        pool.nan_to_num_(0.25)
    batch.kv_len.fill_(cap + n + 3)
    moe.moe_tree_attention(pages, batch, t, q.cuda(), o, ws, scale=0.1)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_ERANGE
    k, v = (torch.cat([x[int(i), 0].float() for i in P.table[0]]).double().cpu() for x in (P.dk, P.dv))
    w = torch.softmax(torch.einsum("tgd,jd->tgj", q.double(), k) * 0.1, -1)
    ref = torch.einsum("tgj,jd->tgd", w, v)
    mag = torch.einsum("tgj,jd->tgd", w, v.abs())
    ds = 2 * D * 2.0 ** -24 * (torch.einsum("tgd,jd->tgj", q.double().abs(), k.abs()) * 0.1).amax(-1, keepdim=True)
    tol = mag * (2.0 ** -8 + 2 * ds + 2.0 ** -21 + 2 * cap * 2.0 ** -24) + ref.abs() * 2.0 ** -8 * (1 + 2.0 ** -8)
    assert ((o.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("n,G,D", [(6, 4, 128), (40, 8, 128), (30, 8, 256)])
def test_the_same_call_gives_the_same_bits(n, G, D):
    """On any stream, beside another batch, in any run."""
    lens, ns = [700 + n, 300 + n, 2000 + n], [n] * 3
    P = Paged(lens, ns, 2, D, 16, seed=3)
    parents = [random_parents(n, 3, b) for b in range(3)]
    q = strided_rows(P.T, 2 * G, D, 0, torch.Generator().manual_seed(3)).cuda()
    pages, batch = P.device()
    t = tree_of(P, batch, parents)
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        ws = moe.AttnWorkspace(2 * G, 2, D)
        for _ in range(3):
            o = torch.empty(P.T, 2 * G, D, dtype=torch.bfloat16, device="cuda")
            moe.moe_tree_attention(pages, batch, t, q, o, ws, scale=0.1, stream=s)
            outs.append((o, ws))
    torch.cuda.synchronize()
    for o, _ in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0][0].view(torch.int16))


def test_calls_that_the_schedule_cannot_count_are_refused():
    """Nothing is launched: the addresses are never followed."""
    import ctypes as C
    from tests.test_attn_refusals import P16, batch, pages
    ws = moe.AttnWorkspace(2, 2, 128)
    t = moe.moe_tree(P16, P16, P16, P16, 1)
    p = pages()
    for b, ok in ((batch(T=1 << 22, B=1 << 12, table_stride=1 << 17), False), (batch(T=0, B=1 << 12, table_stride=1 << 17), True)):
        rc = moe.load().moe_tree_attention(C.byref(p), C.byref(b), C.byref(t), P16, 256, 2, P16, 256, 1.0, 0, ws.handle, None)
        assert rc == (moe.MOE_OK if ok else moe.MOE_EINVAL)
    for bad in (dict(words=0), dict(words=9), dict(above=None), dict(below=None), dict(depth=None)):
        t = moe.moe_tree(*[{**dict(parent=P16, depth=P16, above=P16, below=P16, words=1), **bad}[n] for n, _ in moe.moe_tree._fields_])
        b = batch()
        assert moe.load().moe_tree_attention(C.byref(p), C.byref(b), C.byref(t), P16, 256, 2, P16, 256, 1.0, 0, ws.handle,
                                             None) == moe.MOE_EINVAL

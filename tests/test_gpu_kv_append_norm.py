"""Norms of each head's queries and keys, rotation at a tree's positions and the write into pages, against 64 bits."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import E4M3_STEP, U_BF16, U_E4M3, U_F32, Paged, strided_rows
from tests.gpu_util import require_gpu
from tests.tree_util import depths, random_parents, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


EPS = 1e-6


def reference(x, w, pos, freq, interleaved, eps):
    """(y, size) in fp64: x [T, H, D] normalised by heads and turned; size: of what a turned column is made of.

    w None: not normalised."""
    x = x.double()
    if w is not None:
        x = w.double() * x / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    y, size = x.clone(), x.abs()
    pairs = len(freq)
    ang = torch.from_numpy(np.outer(pos, freq)).view(len(pos), 1, pairs)
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    if pairs:
        y[..., a] = x[..., a] * ang.cos() - x[..., b] * ang.sin()
        y[..., b] = x[..., b] * ang.cos() + x[..., a] * ang.sin()
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def fp32_bound(D, size, normed):
    """Of the value before its last rounding: the sum of D squares (D u of itself), its root and rsqrtf (half of that and
    2 units), three products, sincospif (2 units), the angle's conversion (pi u, as a fraction of half a turn below one),
    its 2^-33 turn (2^-30 rad), and two products and a sum."""
    return size * (((D + 2) / 2 + 4 + 3 if normed else 0) * U_F32 + (4 + 4 + 3) * U_F32 + 2.0 ** -30)


def run(P, Hq, rot, interleaved, w, parents, inplace=False, pad=0, seed=0, theta=1e4, scale_x=1.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (strided_rows(P.T, h, P.D, pad, g) for h in (Hq, P.Hkv, P.Hkv))
    q.mul_(scale_x)
    wq, wk = ((1 + 0.3 * torch.randn(P.D, generator=g)).to(torch.bfloat16) for _ in range(2))
    freq = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) if rot else np.zeros(0)
    pages, batch = P.device()
    before = [x.view(torch.uint8).cpu().clone() for x in (P.dk, P.dv)]
    rope = moe.Rope(rot, inv_freq=freq, interleaved=interleaved) if rot else None
    norm = {"both": lambda: moe.HeadNorm(wq.cuda(), wk.cuda(), EPS), "ones": lambda: moe.HeadNorm(None, None, EPS),
            "keys": lambda: moe.HeadNorm(None, wk.cuda(), EPS), "none": lambda: None}[w]()
    one = torch.ones(P.D, dtype=torch.bfloat16)
    wq, wk = {"both": (wq, wk), "ones": (one, one), "keys": (one, wk), "none": (None, None)}[w]
    tree = None
    if parents is not None:
        tree = moe.Tree(batch, torch.from_numpy(rows_of(P, parents)).cuda())
        moe.moe_tree_prepare(batch, tree)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    up = lambda x: torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)  # noqa: E731
    qd = up(q)
    qo = qd if inplace else torch.full((P.T, Hq, P.D), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_append_norm(pages, batch, rope, norm, qd, qo, up(k), up(v), tree=tree, err=err)
    assert err.item() == 0
    # rows and places
    rows, pos, ids, places = [], [], [], []
    for b in range(P.B):
        d = depths(parents[b]) if parents is not None else list(range(P.ns[b]))
        for i in range(P.ns[b]):
            p = P.lens[b] - P.ns[b] + i
            rows.append(int(P.start[b]) + i)
            pos.append(P.lens[b] - P.ns[b] + d[i])
            ids.append(int(P.table[b, p // P.page]))
            places.append(p % P.page)
    normed = w != "none"
    ref, size = reference(q[rows], wq, pos, freq, interleaved, EPS)
    got = qo.cpu().double()
    bound = fp32_bound(P.D, size, normed)
    off = (got[rows] - ref).abs() - (ref.abs() + bound) * U_BF16 - bound - 2.0 ** -133
    assert (off <= 0).all(), float(off.max())
    rest = np.setdiff1d(np.arange(P.T), rows)
    assert (got[rest] == (q[rest].double() if inplace else 7.0)).all()
    kref, ksize = reference(k[rows], wk, pos, freq, interleaved, EPS)
    for pool, x, size, scale, b0 in ((P.dk, kref, ksize, P.k_scale, before[0]), (P.dv, v[rows].double(), None, P.v_scale, before[1])):
        bound = fp32_bound(P.D, size, normed) if size is not None else torch.zeros_like(x)
        raw = pool.view(torch.uint8).cpu().clone()
        mine = pool.cpu()[ids, :, places].double() if not P.e4m3 else pool.cpu().float()[ids, :, places].double()
        if P.e4m3:
            s = scale.double().view(1, -1, 1)
            y, bound = x / s, bound / s + (x / s).abs() * U_F32
            off = (mine - y.clamp(-448, 448)).abs() - (y.abs() + bound) * U_E4M3 - bound - E4M3_STEP / 2
        else:
            off = (mine - x).abs() - (x.abs() + bound) * U_BF16 - bound - 2.0 ** -133
        assert (off <= 0).all(), float(off.max())
        # nothing else was written
        raw[ids, :, places] = 0
        b0[ids, :, places] = 0
        assert torch.equal(raw, b0)


TREES = [([40], [4], 2), ([300, 20, 0, 133], [9, 20, 0, 64], 3), ([257], [256], 7), ([65536 + 5], [3], 1)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 16, True), (128, 128, True), (128, 32, False),
                                               (256, 64, False), (256, 256, True), (128, 0, False)])
@pytest.mark.parametrize("lens,ns,spread", TREES[:3])
def test_trees(D, rot, interleaved, lens, ns, spread, e4m3):
    P = Paged(lens, ns, 2, D, 16, e4m3=e4m3, lead=1, tail=2, seed=D + len(ns))
    run(P, 6, rot, interleaved, "both", [random_parents(n, spread, n) if n else [] for n in ns])


@pytest.mark.parametrize("w", ["both", "ones", "keys", "none"])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (3, 3, 128), (32, 4, 128), (64, 1, 64), (20, 5, 256)])
def test_heads_and_weights(Hq, Hkv, D, w, tree):
    ns = [5, 1, 17]
    P = Paged([5, 70, 40], ns, Hkv, D, 32, seed=Hq)
    run(P, Hq, D // 2, False, w, [random_parents(n, 2, n) for n in ns] if tree else None, pad=64)


def test_in_place_and_far():
    P = Paged([5, 70], [5, 9], 2, 128, 16, layout="nhd", seed=1)
    run(P, 8, 128, False, "both", [random_parents(5, 2, 5), random_parents(9, 2, 9)], inplace=True)
    P = Paged([TREES[3][0][0]], [3], 1, 64, 64, seed=1)
    run(P, 2, 64, False, "both", [[-1, 0, 0]])


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_small_and_large_rows(scale):
    """Tiny rows are bounded by eps, large ones by their own size."""
    P = Paged([30], [6], 1, 128, 16, seed=2)
    run(P, 4, 64, False, "both", None, scale_x=scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,interleaved", [(64, False), (128, True), (256, False)])
def test_without_norm_and_tree_it_is_append(D, interleaved, e4m3):
    P = Paged([40, 9], [7, 9], 2, D, 16, e4m3=e4m3, seed=3)
    g = torch.Generator().manual_seed(1)
    q, k, v = (strided_rows(P.T, h, D, 0, g).cuda() for h in (4, 2, 2))
    rope = moe.Rope(D // 2, interleaved=interleaved)
    got = []
    for call in (moe.moe_kv_append, lambda p, b, r, *a: moe.moe_kv_append_norm(p, b, r, None, *a)):
        pages, batch = P.device()
        qo = torch.empty_like(q)
        call(pages, batch, rope, q, qo, k, v)
        got.append([x.view(torch.uint8).cpu().clone() for x in (qo, P.dk, P.dv)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_keys_alone_and_bad_pages():
    P = Paged([40], [6], 2, 128, 16, seed=3)
    P.table[0, 2] = 10 ** 6
    g = torch.Generator().manual_seed(1)
    k, v = (strided_rows(P.T, 2, 128, 0, g).cuda() for _ in range(2))
    pages, batch = P.device()
    before = [x.clone() for x in (P.dk, P.dv)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_kv_append_norm(pages, batch, None, moe.HeadNorm(eps=1e-5), None, None, k, v, err=err)
    assert err.item() == moe.MOE_ERANGE  # places 34 .. 39 lie in the page that is not there
    for a, b in zip(before, (P.dk, P.dv)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_weights_of_another_width_are_refused():
    P = Paged([40], [6], 2, 128, 16, seed=3)
    pages, batch = P.device()
    x = torch.zeros(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_kv_append_norm(pages, batch, None, moe.HeadNorm(torch.ones(64, dtype=torch.bfloat16, device="cuda")), x, x, x, x)

"""moe_kv_append against the rotation and the rounding in 64 bits."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import E4M3_STEP, Paged, U_BF16, U_E4M3, U_F32, strided_rows
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def turned(x, pos, f, rot, interleaved):
    """fp64 rotation of [T, H, D] rows, and the size of the pair each column belongs to."""
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    if rot:
        a = torch.tensor(pos, dtype=torch.float64).view(-1, 1, 1) * torch.from_numpy(f)
        i = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        u, w = x[..., i[0]], x[..., i[1]]
        y[..., i[0]], y[..., i[1]] = u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()
        size[..., i[0]] = size[..., i[1]] = u.abs() + w.abs()
    return y, size


CASES = [
    # lens, new, Hq, Hkv, D, rot, interleaved, page, e4m3, layout
    ([1], [1], 1, 1, 64, 64, False, 16, False, "hnd"),
    ([5], [4], 16, 2, 256, 64, False, 64, False, "hnd"),
    ([17, 16, 0, 33, 15], [3, 1, 0, 16, 15], 6, 3, 128, 128, True, 16, False, "nhd"),
    ([100, 7, 64], [1, 1, 1], 8, 1, 128, 96, False, 1, True, "hnd"),
    ([300, 129], [130, 129], 4, 4, 64, 16, True, 128, True, "kv"),
    ([77, 78], [2, 9], 0, 2, 256, 256, False, 32, False, "kv"),
    ([40], [33], 5, 1, 256, 240, True, 8, True, "nhd"),
    ([3] * 300, [1] * 300, 2, 1, 64, 32, False, 4, False, "hnd"),
    ([9, 8], [4, 4], 4, 2, 128, 0, False, 16, True, "hnd"),
]


@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,rot,il,page,e4m3,layout", CASES)
@pytest.mark.parametrize("far", [0, 1_000_003])
def test_append(lens, ns, Hq, Hkv, D, rot, il, page, e4m3, layout, far):
    if far:  # the same pages, met at positions about a million later
        far = far // page * page
    P = Paged(lens, ns, Hkv, D, page, e4m3, layout, seed=len(lens) + D, lead=2, tail=3)
    if far:
        if len(lens) > 10:
            pytest.skip("table of a million entries for 300 requests")
        P.table = np.concatenate([np.full((P.B, far // page), -1, np.int32), P.table], 1)
    g = torch.Generator().manual_seed(5)
    q = strided_rows(P.T, max(Hq, 1), D, 8, g)
    kv = strided_rows(P.T, 2 * Hkv, D, 24, g)
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot) if rot else None
    pages, _ = P.device()
    bt = moe.KvBatch(torch.from_numpy(P.start).cuda(),
                     torch.tensor([l + far if n else 0 for l, n in zip(lens, ns)], dtype=torch.int32).cuda(),
                     torch.from_numpy(P.table).cuda(), P.T, max(ns))
    rope = moe.Rope(rot, interleaved=il) if rot else None
    dev = lambda x: torch.as_strided(  # noqa: E731
        x._base.cuda() if x._base is not None else x.cuda(), x.shape, x.stride(), x.storage_offset())
    qd, kd, vd = (dev(x) for x in (q, k, v))
    qo = torch.full((P.T, max(Hq, 1), D), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_kv_append(pages, bt, rope, qd if Hq else None, qo if Hq else None, kd, vd, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    mine = slice(P.lead, P.lead + sum(ns))
    pos = [p + far for r in P.positions() for p in r]
    # fp32 rotation: a fraction of a turn off by 2^-24 of itself, sincospif within 2 ulp, two products and a sum
    rel = 16 * U_F32
    if Hq:
        ref, size = turned(q[mine], pos, f, rot, il)
        got = qo.cpu().double()
        assert ((got[mine] - ref).abs() <= U_BF16 * ref.abs() + (1 + U_BF16) * rel * size + 1e-38).all()
        assert (got[:P.lead] == 7).all() and (got[mine.stop:] == 7).all()
    for which, pool, before, scale, new in (("k", P.dk, P.k, P.k_scale, k), ("v", P.dv, P.v, P.v_scale, v)):
        ref, size = turned(new[mine], pos, f, rot if which == "k" else 0, il)
        raw = torch.uint8 if e4m3 else torch.int16
        got, old = pool.cpu(), before.clone()
        written = torch.zeros(old.shape[0], page, dtype=torch.bool)
        for r, (b, p) in enumerate([(b, p) for b, rr in enumerate(P.positions()) for p in rr]):
            at = int(P.table[b, (p + far) // page]), p % page
            written[at] = True
            x = got[at[0], :, at[1]].float().double()
            if e4m3:
                s = scale.double().view(-1, 1)
                want, tol = (ref[r] / s).clamp(-448, 448), size[r] / s * rel
                tol = tol + torch.maximum(U_E4M3 * want.abs() * (1 + 4 * U_F32), torch.full_like(want, E4M3_STEP / 2)) + 4 * U_F32 * want.abs()
            else:
                want, tol = ref[r], U_BF16 * ref[r].abs() + (1 + U_BF16) * rel * size[r] + 1e-38
            assert ((x - want).abs() <= tol).all(), (which, b, p)
        same = (got.view(raw) == old.view(raw)) | written.view(old.shape[0], 1, page, 1)
        assert same.all()


def test_values_saturate_and_nan_stays_in_e4m3():
    P = Paged([4], [4], 1, 64, 16, e4m3=True, junk=0.0)
    P.k_scale, P.v_scale = torch.ones(1), torch.full((1,), 2.0)
    pages, bt = P.device()
    x = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 448, 464.0, 0.0009765625] * 8)
    k = x.to(torch.bfloat16).view(1, 1, 64).expand(4, 1, 64).contiguous().cuda()
    moe.moe_kv_append(pages, bt, None, None, None, k, k)
    got = P.dk[int(P.table[0, 0]), 0, 0, :8].cpu().float()
    assert got[:4].tolist() == [448, -448, 448, -448] and got[4].isnan() and got[5:].tolist() == [448, 448, 0.0]
    got = P.dv[int(P.table[0, 0]), 0, 3, :8].cpu().float()
    assert got[:4].tolist() == [448, -448, 448, -448] and got[4].isnan() and got[5:].tolist() == [224, 224, 0.0]


def test_in_place_queries_and_custom_frequencies():
    P = Paged([700], [3], 1, 128, 64)
    pages, bt = P.device()
    g = torch.Generator().manual_seed(1)
    q, k = strided_rows(3, 4, 128, 0, g), strided_rows(3, 1, 128, 0, g)
    f = np.linspace(-2.0, 9.0, 64)  # any finite frequency, whole turns and negative ones too
    qd = q.cuda()
    moe.moe_kv_append(pages, bt, moe.Rope(128, inv_freq=f), qd, qd, k.cuda(), k.cuda())
    ref, size = turned(q, [697, 698, 699], f, 128, False)
    # the given f's 53 bits, at most 9 rad a step, 700 steps
    tol = U_BF16 * ref.abs() + (1 + U_BF16) * (16 * U_F32 + 700 * 9 * 2.0 ** -52) * size
    assert ((qd.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("what", ["page below", "page beyond", "position below", "position beyond"])
def test_bad_places_are_reported_and_nothing_is_stored(what):
    P = Paged([40, 40], [2, 2], 2, 64, 16, table_extra=0, junk=0.0)
    good = P.table.copy()
    if what == "page below":
        P.table[1, 2] = -1
    elif what == "page beyond":
        P.table[1, 2] = P.k.shape[0]
    elif what == "position below":
        P.lens[1] = 1  # two new tokens in a cache of one: the first is at -1
    else:
        P.lens[1] = 49  # 48 places in the table
    pages, bt = P.device()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = P.dk.clone()
    moe.moe_kv_append(pages, bt, None, None, None, k, k, err=err)
    assert int(err) == moe.MOE_ERANGE
    changed = (P.dk != before).any(-1).any(1)
    stored = {(int(good[0, 2]), 6), (int(good[0, 2]), 7)}
    if what == "position below":
        stored.add((int(good[1, 0]), 0))
    elif what == "position beyond":
        stored.add((int(good[1, 2]), 15))
    assert {(int(p), int(i)) for p, i in changed.nonzero()} == stored


def test_another_stream_and_a_graph():
    P = Paged([20, 9], [1, 1], 2, 64, 16)
    pages, bt = P.device()
    g = torch.Generator().manual_seed(3)
    q, k = strided_rows(2, 4, 64, 0, g).cuda(), strided_rows(2, 2, 64, 0, g).cuda()
    rope, qo = moe.Rope(64), torch.empty_like(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            moe.moe_kv_append(pages, bt, rope, q, qo, k, k)
        bt.kv_len.copy_(torch.tensor([19, 9], dtype=torch.int32))  # a replay reads the lengths of its time
        graph.replay()
    s.synchronize()
    one, kk = qo.clone(), P.dk.clone()
    moe.moe_kv_append(pages, bt, rope, q, qo, k, k)
    torch.cuda.synchronize()
    assert torch.equal(one, qo) and torch.equal(kk.view(torch.int16), P.dk.view(torch.int16))

"""What the calls of a drafted-tree step refuse, on the CPU: nothing is launched; and that the definition of
verification, as the tests compute it, keeps the target's distribution."""
import ctypes as C

import numpy as np
import pytest
import torch

from serving_router_top_gb300 import build, moe
from tests.test_attn_refusals import BAD_PAGES, P16, batch, pages
from tests.tree_util import random_parents, verify_ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load()


def tree(**kw):
    d = dict(parent=P16, depth=P16, above=P16, below=P16, words=2)
    d.update(kw)
    return moe.moe_tree(*[d[n] for n, _ in moe.moe_tree._fields_])


@pytest.mark.parametrize("kw", [dict(words=0), dict(words=9), dict(words=-1), dict(parent=None), dict(depth=None),
                                dict(above=None), dict(below=None)])
def test_trees_are_checked(lib, kw):
    b, t = batch(), tree(**kw)
    assert lib.moe_tree_prepare(C.byref(b), C.byref(t), None, None) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(B=-1), dict(T=-1), dict(q_start=None)])
def test_tree_batches_are_checked(lib, kw):
    b, t = batch(**kw), tree()
    assert lib.moe_tree_prepare(C.byref(b), C.byref(t), None, None) == moe.MOE_EINVAL
    assert lib.moe_tree_prepare(None, C.byref(t), None, None) == moe.MOE_EINVAL
    assert lib.moe_tree_prepare(C.byref(b), None, None, None) == moe.MOE_EINVAL


def append(lib, p=None, b=None, t=None, rope=None, norm=None, q=P16, qs=256, qo=P16, qos=256, Hq=2, k=P16, ks=256, v=P16,
           vs=256):
    p, b = p or pages(), b or batch()
    return lib.moe_kv_append_norm(C.byref(p), C.byref(b), t and C.byref(t), rope, norm and C.byref(norm), q, qs, qo, qos, Hq,
                                  k, ks, v, vs, None, None)


@pytest.mark.parametrize("w_q,w_k,eps", [(None, None, 0.0), (None, None, -1.0), (None, None, float("nan")),
                                         (None, None, float("inf")), (P16 + 8, None, 1e-6), (None, P16 + 2, 1e-6)])
def test_head_norms_are_checked(lib, w_q, w_k, eps):
    assert append(lib, norm=moe.moe_head_norm(w_q, w_k, eps)) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_append_norm_checks_pools(lib, kw):
    assert append(lib, p=pages(**kw)) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(q=None), dict(Hq=0), dict(qo=P16 + 8), dict(k=None), dict(v=P16 + 14), dict(qs=248),
                                dict(ks=128), dict(t=tree(depth=None))])
def test_append_norm_rows_are_checked(lib, kw):
    assert append(lib, **kw) == moe.MOE_EINVAL


def verify(lib, b=None, path=P16, stride=4, count=P16, token=P16, **kw):
    d = dict(target=P16, target_stride=100, draft=P16, draft_stride=100, token=P16, parent=P16, u=P16, u_last=P16, V=100)
    d.update(kw)
    b, d = b or batch(), moe.moe_verify_desc(*[d[n] for n, _ in moe.moe_verify_desc._fields_])
    return lib.moe_verify_drafts(C.byref(b), C.byref(d), path, stride, count, token, None, None)


@pytest.mark.parametrize("kw", [dict(target=None), dict(token_=None), dict(parent=None), dict(u=None), dict(u_last=None),
                                dict(V=0), dict(V=-1), dict(V=(1 << 24) + 1), dict(target_stride=99), dict(draft_stride=99),
                                dict(target=P16 + 2), dict(draft=P16 + 1), dict(path=None), dict(stride=0), dict(count=None),
                                dict(out=None)])
def test_verification_is_checked(lib, kw):
    kw = dict(kw)
    b, d = batch(), dict(target=P16, target_stride=100, draft=P16, draft_stride=100, token=P16, parent=P16, u=P16,
                         u_last=P16, V=100)
    out = dict(path=P16, stride=4, count=P16, out=P16)
    for k, v in kw.items():
        if k in out:
            out[k] = v
        else:
            d[k.rstrip("_")] = v
    desc = moe.moe_verify_desc(*[d[n] for n, _ in moe.moe_verify_desc._fields_])
    assert lib.moe_verify_drafts(C.byref(b), C.byref(desc), out["path"], out["stride"], out["count"], out["out"], None,
                                 None) == moe.MOE_EINVAL


def test_verification_of_nothing_is_ok(lib):
    assert verify(lib, b=batch(B=0)) == moe.MOE_OK
    assert verify(lib, b=batch(B=-1)) == moe.MOE_EINVAL


def compact(lib, layers, b=None, L=None, path=P16, stride=4, count=P16, out=P16 * 2):
    arr, b = (moe.moe_kv_pages * len(layers))(*layers), b or batch()
    return lib.moe_kv_compact(arr, len(layers) if L is None else L, C.byref(b), path, stride, count, out, None, None)


def copy(lib, layers, L=None, src=P16, dst=P16, n=1):
    arr = (moe.moe_kv_pages * len(layers))(*layers)
    return lib.moe_kv_copy_pages(arr, len(layers) if L is None else L, src, dst, None, n, None, None)


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_moves_check_pools(lib, kw):
    assert compact(lib, [pages(**kw)]) == moe.MOE_EINVAL
    assert copy(lib, [pages(**kw)]) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(e4m3=1), dict(Hkv=1), dict(D=64), dict(page=8), dict(npages=5), dict(page_stride=8192),
                                dict(head_stride=4096), dict(tok_stride=256), dict(k=None), dict(v=P16 + 8)])
def test_layers_are_alike(lib, kw):
    assert compact(lib, [pages(), pages(**kw)]) == moe.MOE_EINVAL
    assert copy(lib, [pages(), pages(), pages(**kw)]) == moe.MOE_EINVAL


def test_moves_are_checked(lib):
    for kw in (dict(L=0), dict(L=4097), dict(path=None), dict(count=None), dict(stride=0), dict(out=P16)):
        assert compact(lib, [pages()], **kw) == moe.MOE_EINVAL, kw  # batch's kv_len is P16
    for kw in (dict(L=0), dict(L=4097), dict(src=None), dict(dst=None), dict(n=-1), dict(n=(1 << 20) + 1)):
        assert copy(lib, [pages()], **kw) == moe.MOE_EINVAL, kw
    assert copy(lib, [pages()], n=0) == moe.MOE_OK
    assert compact(lib, [pages()], b=batch(B=0)) == moe.MOE_OK


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def cpu_batch(T=4, B=2):
    return moe.KvBatch(ints(B + 1), ints(B), ints(B, 3), T, 2)


def test_arguments_are_told_by_type_and_shape():
    b = cpu_batch()
    with pytest.raises(ValueError):
        moe.Tree(b, ints(5))
    with pytest.raises(ValueError):
        moe.Tree(b, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        moe.Tree(moe.KvBatch(ints(3), ints(2), ints(2, 3), 4, 257), ints(4))
    with pytest.raises(ValueError):
        moe.HeadNorm(torch.zeros(128), None)
    with pytest.raises(ValueError):
        moe.HeadNorm(torch.zeros(128, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16))
    p = torch.zeros(4, 9)
    for kw in (dict(target=p.double()), dict(target=p[:, ::2]), dict(draft=torch.zeros(4, 8)), dict(token=ints(3)),
               dict(token=torch.zeros(4)), dict(parent=ints(4, 1)), dict(u=torch.zeros(3)), dict(u=torch.zeros(4).double()),
               dict(u_last=torch.zeros(2, 1))):
        a = dict(target=p, token=ints(4), parent=ints(4), u=torch.zeros(4), u_last=torch.zeros(2), draft=None)
        a.update(kw)
        with pytest.raises(ValueError):
            moe.verify_desc(**a)
    d = moe.verify_desc(p, ints(4), ints(4), torch.zeros(4), torch.zeros(2))
    for path, count, token in ((ints(2), ints(2), ints(2)), (ints(3, 2), ints(2), ints(2)), (ints(2, 2), ints(3), ints(2)),
                               (ints(2, 2), ints(2), ints(1)), (ints(2, 2).long(), ints(2), ints(2))):
        with pytest.raises(ValueError):
            moe.moe_verify_drafts(b, d, path, count, token)
    with pytest.raises(ValueError):
        moe.moe_verify_drafts(cpu_batch(T=5), d, ints(2, 2), ints(2), ints(2))
    with pytest.raises(ValueError):
        moe.KvLayers([])


def test_tensors_elsewhere_are_refused():
    b = cpu_batch()
    t = moe.Tree(b, ints(4))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    kv = moe.KvPages(bf(2, 2, 16, 64), bf(2, 2, 16, 64))
    rows = bf(4, 2, 64)
    d = moe.verify_desc(torch.zeros(4, 9), ints(4), ints(4), torch.zeros(4), torch.zeros(2))
    layers = moe.KvLayers([kv])
    for call in (lambda: moe.moe_tree_prepare(b, t),
                 lambda: moe.moe_kv_append_norm(kv, b, None, None, rows, rows, rows, rows, tree=t),
                 lambda: moe.moe_verify_drafts(b, d, ints(2, 2), ints(2), ints(2)),
                 lambda: moe.moe_kv_compact(layers, b, ints(2, 2), ints(2)),
                 lambda: moe.moe_kv_copy_pages(layers, ints(1), ints(1))):
        with pytest.raises(ValueError, match="another device"):
            call()


@pytest.mark.parametrize("drawn", [True, False])
def test_the_definition_keeps_the_targets_distribution(drawn):
    """Over u, the first token after node 0 (a kept child's, or the next) has the target's probabilities: by counting on a
    grid of random numbers that is even for the picked form, and within five standard deviations of draws for the other."""
    r = np.random.RandomState(3)
    V, N = 5, 6000
    p, q = (np.float32(x / x.sum()) for x in (r.rand(V) + 0.05, r.rand(V) + 0.05))
    parents = [-1, 0, 0, 0]
    seen = np.zeros(V)
    for _ in range(N):
        tokens = [-1] + (list(r.choice(V, 3, p=np.float64(q) / np.float64(q).sum())) if drawn else [4, 1, 4])
        path, nxt = verify_ref(parents, tokens, np.float32(r.rand(4)), np.float32(r.rand()), [p] * 4,
                               [q] * 4 if drawn else None, 4)
        seen[tokens[path[1]] if len(path) > 1 else nxt] += 1
    sd = np.sqrt(N * p * (1 - p))
    assert (np.abs(seen - N * p) < 5 * sd).all(), (seen, N * p)


def test_parents_rise():
    assert random_parents(5, 1, 0) == [-1, 0, 1, 2, 3]

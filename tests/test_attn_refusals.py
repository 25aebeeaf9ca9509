"""What the calls of a layer's attention half refuse, on the CPU: nothing is launched."""
import ctypes as C

import numpy as np
import pytest
import torch

from serving_router_top_gb300 import build, moe

P16 = 1 << 20  # a 16-byte aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load()


def pages(**kw):
    d = dict(k=P16, v=P16, e4m3=0, Hkv=2, D=128, page=16, npages=4, page_stride=2 * 16 * 128, head_stride=16 * 128,
             tok_stride=128, k_scale=None, v_scale=None)
    d.update(kw)
    return moe.moe_kv_pages(*[d[n] for n, _ in moe.moe_kv_pages._fields_])


def batch(**kw):
    d = dict(q_start=P16, kv_len=P16, page_table=P16, B=2, T=3, max_n=2, table_stride=4)
    d.update(kw)
    return moe.moe_kv_batch(*[d[n] for n, _ in moe.moe_kv_batch._fields_])


BAD_PAGES = [dict(k=None), dict(v=None), dict(k=P16 + 8), dict(v=P16 + 2), dict(e4m3=2), dict(e4m3=-1), dict(Hkv=0),
             dict(Hkv=1025), dict(D=0), dict(D=96), dict(D=512), dict(page=0), dict(page=24), dict(page=1 << 17),
             dict(npages=0), dict(page_stride=127), dict(page_stride=-4096), dict(head_stride=64), dict(tok_stride=127),
             dict(tok_stride=132), dict(e4m3=1, tok_stride=136), dict(tok_stride=1 << 57),
             dict(e4m3=1, D=64, page=1)]
BAD_BATCH = [dict(B=-1), dict(T=-1), dict(max_n=-1), dict(table_stride=-1), dict(q_start=None), dict(kv_len=None),
             dict(page_table=None)]


def append(lib, p=None, b=None, rope=None, q=P16, qs=256, qo=P16, qos=256, Hq=2, k=P16, ks=256, v=P16, vs=256):
    p, b = p or pages(), b or batch()
    return lib.moe_kv_append(C.byref(p), C.byref(b), rope, q, qs, qo, qos, Hq, k, ks, v, vs, None, None)


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_pools_are_checked(lib, kw):
    assert append(lib, p=pages(**kw)) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", BAD_BATCH)
def test_requests_are_checked(lib, kw):
    assert append(lib, b=batch(**kw)) == moe.MOE_EINVAL


@pytest.mark.parametrize("kw", [dict(q=None), dict(Hq=0), dict(Hq=-1), dict(qo=None), dict(k=None), dict(v=None),
                                dict(q=P16 + 4), dict(qo=P16 + 8), dict(k=P16 + 2), dict(v=P16 + 14), dict(qs=248),
                                dict(qos=260), dict(ks=128), dict(vs=-256)])
def test_append_rows_are_checked(lib, kw):
    assert append(lib, **kw) == moe.MOE_EINVAL


def test_nothing_to_do_is_ok(lib):
    assert append(lib, b=batch(T=0)) == moe.MOE_OK
    assert append(lib, b=batch(B=0)) == moe.MOE_OK
    assert append(lib, b=batch(B=0, q_start=None, kv_len=None, page_table=None)) == moe.MOE_OK


@pytest.mark.parametrize("rot,theta,f", [(0, 1e4, None), (8, 1e4, None), (24, 1e4, None), (272, 1e4, None),
                                         (64, 0.0, None), (64, -1.0, None), (64, np.inf, None), (64, np.nan, None),
                                         (16, 1e4, [1.0] * 7 + [np.nan]), (16, 1e4, [1.0] * 7 + [np.inf])])
def test_rope_is_checked(lib, rot, theta, f):
    with pytest.raises(moe.MoeError):
        moe.Rope(rot, theta=theta, inv_freq=f)


def test_rope_wants_half_rot_frequencies(lib):
    with pytest.raises(ValueError):
        moe.Rope(16, inv_freq=[1.0] * 16)


@pytest.mark.parametrize("Hq,Hkv,D", [(0, 1, 128), (3, 2, 128), (2, 0, 128), (65, 1, 128), (2, 2, 96), (2, 2, 0),
                                      (4096, 2048, 64)])
def test_attention_workspace_is_checked(lib, Hq, Hkv, D):
    with pytest.raises(moe.MoeError) as e:
        moe.AttnWorkspace(Hq, Hkv, D)
    assert e.value.code == moe.MOE_EINVAL


def test_attention_without_a_workspace(lib):
    p, b = pages(), batch()
    assert lib.moe_paged_attention(C.byref(p), C.byref(b), P16, 256, 2, P16, 256, 1.0, 0, None, None) == moe.MOE_EINVAL
    assert lib.moe_paged_attention(None, C.byref(b), P16, 256, 2, P16, 256, 1.0, 0, None, None) == moe.MOE_EINVAL
    assert lib.moe_attn_sync_status(None, None) == moe.MOE_EINVAL
    assert lib.moe_attn_ws_get_view(None, None) == moe.MOE_EINVAL
    assert lib.moe_attn_ws_destroy(None) == moe.MOE_OK and lib.moe_rope_destroy(None) == moe.MOE_OK
    assert lib.moe_attn_ws_create(None, 2, 2, 128) == moe.MOE_EINVAL
    assert lib.moe_rope_create(None, 64, 0, 1e4, None) == moe.MOE_EINVAL


def norm(lib, x=P16, xs=64, xo=P16, xos=64, xn=P16, xns=64, T=2, H=64, **kw):
    d = dict(y=P16, y_stride=64, post_norm=1, w_post=P16, gate=P16, gate_stride=64, gate_sigmoid=0, res_scale=1.0,
             w_pre=P16, eps=1e-6)
    d.update(kw)
    c = moe.moe_block_norm_desc(*[d[n] for n, _ in moe.moe_block_norm_desc._fields_])
    return lib.moe_block_norm(C.byref(c), x, xs, xo, xos, xn, xns, T, H, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(T=-1), dict(H=0), dict(H=16385), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(y=None), dict(x=P16 + 2),
                                dict(xo=P16 + 1), dict(xn=P16 + 1), dict(y=P16 + 1), dict(gate=P16 + 1),
                                dict(w_post=P16 + 1), dict(w_pre=P16 + 1), dict(xs=63), dict(xos=0), dict(xns=32),
                                dict(y_stride=0), dict(gate_stride=63), dict(gate_stride=-64)])
def test_block_norm_is_checked(lib, kw):
    assert norm(lib, **kw) == moe.MOE_EINVAL


def test_block_norm_nothing_to_do(lib):
    assert norm(lib, T=0) == moe.MOE_OK
    assert norm(lib, xo=None, xn=None) == moe.MOE_OK
    assert lib.moe_block_norm(None, P16, 64, P16, 64, P16, 64, 2, 64, None) == moe.MOE_EINVAL


def test_binding_refuses_shapes_types_and_layouts(lib):
    bf = torch.bfloat16
    k = torch.zeros(3, 2, 16, 64, dtype=bf)
    for kk, vv in [(k, k[:2]), (k, k.half()), (k.float(), k.float()), (k[..., ::2], k[..., ::2]), (k[0], k[0])]:
        with pytest.raises(ValueError):
            moe.KvPages(kk, vv)
    with pytest.raises(ValueError):
        moe.KvPages(k, k, k_scale=torch.ones(3))
    with pytest.raises(ValueError):
        moe.KvPages(k, k, v_scale=torch.ones(2, dtype=torch.float64))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for a in [(i(2), i(2), i(2, 4)), (i(3), i(2), i(3, 4)), (i(3).long(), i(2), i(2, 4)), (i(3), i(2), i(8)),
              (i(6)[::2], i(2), i(2, 4)), (i(3), i(2), i(2, 8)[:, :4])]:
        with pytest.raises(ValueError):
            moe.KvBatch(*a, T=3, max_n=1)
    pg, bt = moe.KvPages(k, k), moe.KvBatch(i(3), i(2), i(2, 4), 3, 2)
    ok = torch.zeros(3, 2, 64, dtype=bf)
    for bad in [torch.zeros(2, 2, 64, dtype=bf), torch.zeros(3, 2, 128, dtype=bf), ok.float(),
                torch.zeros(3, 64, 2, dtype=bf).transpose(1, 2), torch.zeros(3, 4, 64, dtype=bf)[:, ::2]]:
        with pytest.raises(ValueError):
            moe.moe_kv_append(pg, bt, None, ok, ok, bad, ok)
    x, y = torch.zeros(3, 64), torch.zeros(3, 64, dtype=bf)
    for kw in [dict(y=y.float()), dict(y=y, gate=y[:2]), dict(y=y, gate=y[:, :32]), dict(y=y, post_norm=True, w_post=y),
               dict(y=y, w_pre=torch.zeros(32, dtype=bf))]:
        with pytest.raises(ValueError):
            moe.block_norm_desc(**kw)
    d = moe.block_norm_desc(y=y)
    for a in [(x[:2], x, y), (x, x[:, :32], y), (x, x, y[:2]), (x.double(), x, y), (x, x, x)]:
        with pytest.raises(ValueError):
            moe.moe_block_norm(d, *a, 3, 64)

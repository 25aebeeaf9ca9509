"""What the attention half's binding refuses before the library is called, on the CPU."""
import pytest
import torch

from serving_router_top_gb300 import moe

BF = torch.bfloat16


@pytest.fixture
def no_call(monkeypatch):
    """Any call of the library fails the test: the arguments have to be refused before it."""
    def load():
        raise AssertionError("the library was called")
    monkeypatch.setattr(moe, "load", load)
    monkeypatch.setattr(moe, "_stream", lambda stream: None)


def apart(t):
    """The same shape and type with columns two elements apart."""
    return torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]


def test_norm_columns_are_contiguous(no_call):
    x, y = torch.zeros(3, 64), torch.zeros(3, 64, dtype=BF)
    d = moe.block_norm_desc(y=y)
    for rows in [(apart(x), x, y), (x, apart(x), y), (x, x, apart(y)), (torch.zeros(64, 3).t(), x, y)]:
        with pytest.raises(ValueError, match="got"):
            moe.moe_block_norm(d, *rows, 3, 64)


HALF = torch.float16


def kv(pool=BF, T=3):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(3, 2, 16, 64, dtype=pool)
    return moe.KvPages(k, k.clone()), moe.KvBatch(i(3), i(2), i(2, 4), T, 2)


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("dtype", [HALF, torch.float32])
def test_append_takes_bf16_rows(no_call, at, dtype):
    pages, batch = kv()
    rows = [torch.zeros(3, 2, 64, dtype=BF) for _ in range(4)]
    rows[at] = rows[at].to(dtype)
    with pytest.raises(ValueError, match="got"):
        moe.moe_kv_append(pages, batch, None, *rows)


class Workspace:
    Hq, handle = 4, None


@pytest.mark.parametrize("at", range(2))
@pytest.mark.parametrize("dtype", [HALF, torch.float32])
def test_attention_takes_bf16_rows(no_call, at, dtype):
    pages, batch = kv()
    rows = [torch.zeros(3, 4, 64, dtype=BF) for _ in range(2)]
    rows[at] = rows[at].to(dtype)
    with pytest.raises(ValueError, match="got"):
        moe.moe_paged_attention(pages, batch, *rows, Workspace(), 1.0)


def test_norm_takes_fp32_and_bf16_rows(no_call):
    x, y, w = torch.zeros(3, 64), torch.zeros(3, 64, dtype=BF), torch.zeros(64, dtype=BF)
    for kw in [dict(y=y.half()), dict(y=y, gate=y.half()), dict(y=y, post_norm=True, w_post=w.half()),
               dict(y=y, w_pre=w.half())]:
        with pytest.raises(ValueError):
            moe.block_norm_desc(**kw)
    bits = [t.view(b) for t, b in ((y, torch.int16), (y, torch.uint16), (w, torch.int16))]
    d = moe.block_norm_desc(y=bits[0], gate=bits[1], post_norm=True, w_post=w, w_pre=bits[2])
    for rows in [(x.int(), x, y), (x, x.int(), y), (x, x, y.half())]:
        with pytest.raises(ValueError, match="got"):
            moe.moe_block_norm(d, *rows, 3, 64)


def test_tensors_of_the_host_are_refused(no_call):
    pages, batch = kv()
    q = torch.zeros(3, 4, 64, dtype=BF)
    k = torch.zeros(3, 2, 64, dtype=BF)
    x, y = torch.zeros(3, 64), torch.zeros(3, 64, dtype=BF)
    for call in (lambda: moe.moe_kv_append(pages, batch, None, q, q, k, k),
                 lambda: moe.moe_kv_append(pages, batch, None, None, None, k, k),
                 lambda: moe.moe_paged_attention(pages, batch, q, q, Workspace(), 1.0),
                 lambda: moe.moe_block_norm(moe.block_norm_desc(y=y), x, x, y, 3, 64)):
        with pytest.raises(ValueError, match="another device"):
            call()


def test_wait_test_stages():
    from serving_router_top_gb300 import build
    build.build()
    assert moe.load().moe_attn_ws_set_wait_test(None, 0) == moe.MOE_EINVAL

"""Outputs of a verification and of a compaction that lie on their inputs, on the CPU: nothing is launched."""
import ctypes as C

import pytest

from serving_router_top_gb300 import build, moe
from tests.test_attn_refusals import P16, batch, pages


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load()


@pytest.mark.parametrize("out,count,B", [(0, 0, 2), (4, 0, 2), (-4, 0, 2), (0, 4096, 2), (4, 4096, 2), (-4, 4096, 2),
                                         (1020, 0, 256), (-1020, 4096, 256)])
def test_lengths_do_not_lie_on_what_is_read(lib, out, count, B):
    """kv_len_out over count, or over the batch's kv_len (P16): other CTAs, and the launches of later layers, read them."""
    p, b, at = pages(), batch(B=B), P16 * 4
    b.kv_len, path = P16 * 2, P16 * 8
    near = at + count if count == 0 else b.kv_len
    arr = (moe.moe_kv_pages * 1)(p)
    assert lib.moe_kv_compact(arr, 1, C.byref(b), path, 4, at, near + out, None, None) == moe.MOE_EINVAL


def test_lengths_do_not_lie_on_the_paths(lib):
    p, b = pages(), batch(B=2)
    b.kv_len = P16 * 2
    arr = (moe.moe_kv_pages * 1)(p)
    for off in (0, 28, -4):
        assert lib.moe_kv_compact(arr, 1, C.byref(b), P16 * 8, 4, P16 * 4, P16 * 8 + off, None, None) == moe.MOE_EINVAL


def verify(lib, **kw):
    """Two requests of three rows, every array 4096 bytes from the next."""
    at = {n: P16 + 4096 * i for i, n in enumerate(("q_start", "token", "parent", "u", "u_last", "path", "count", "out"))}
    at.update(kw)
    b = batch(B=2, T=3)
    b.q_start = at["q_start"]
    d = moe.moe_verify_desc(P16 * 2, 100, None, 0, at["token"], at["parent"], at["u"], at["u_last"], 100)
    return lib.moe_verify_drafts(C.byref(b), C.byref(d), at["path"], 4, at["count"], at["out"], None, None)


@pytest.mark.parametrize("out,words", [("path", 8), ("count", 2), ("out", 2)])
@pytest.mark.parametrize("other,held", [("q_start", 3), ("token", 3), ("parent", 3), ("u", 3), ("u_last", 2), ("path", 8), ("count", 2), ("out", 2)])
def test_what_is_kept_does_not_lie_on_what_is_read(lib, out, words, other, held):
    """The next tokens over the drafted ones, say: one request's is written while another's are read."""
    if out == other:
        return
    for off in (0, 4 * (held - 1), -4 * (words - 1)):
        assert verify(lib, **{other: P16 * 3, out: P16 * 3 + off}) == moe.MOE_EINVAL

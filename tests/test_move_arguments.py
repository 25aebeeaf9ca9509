"""Outputs of a compaction that lie on its inputs, on the CPU: nothing is launched."""
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

"""Nodes whose masks are empty (never prepared, or past the masks' words) see the keys before the tree and no other."""
import numpy as np
import pytest
import torch

import tests.tree_util as tree_util
from serving_router_top_gb300 import moe
from tests.attn_util import Paged, strided_rows
from tests.gpu_util import require_gpu
from tests.test_gpu_tree_attention import check
from tests.tree_util import depths, random_parents, rows_of, sees, tree_attention_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# one shape or more of each kernel and tile: D, G, nodes of two requests
SHAPES = [(64, 4, [5, 3]), (64, 8, [6, 4]), (64, 8, [40, 36]), (128, 4, [5, 3]), (128, 4, [5, 12]), (128, 8, [40, 36]),
          (256, 4, [4, 3]), (256, 8, [8, 6]), (256, 8, [40, 36])]


def compare(monkeypatch, P, G, t, batch, pages, masks, window):
    """Against the 64-bit softmax of rows that see `masks` and are as deep as they say."""
    q = strided_rows(P.T, G, P.D, 0, torch.Generator().manual_seed(0))
    ws, o = moe.AttnWorkspace(G, 1, P.D), torch.full((P.T, G, P.D), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_tree_attention(pages, batch, t, q.cuda(), o, ws, scale=0.1, window=window)
    assert moe.moe_attn_sync_status(ws) == 0
    monkeypatch.setattr(tree_util, "sees", lambda m: m[0])
    monkeypatch.setattr(tree_util, "depths", lambda m: m[1])
    ref, tol = tree_attention_ref(P, q, G, 0.1, window, masks)
    check(o.cpu().double(), ref, tol)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("D,G,ns", SHAPES)
def test_trees_that_were_never_prepared(monkeypatch, D, G, ns, window, e4m3):
    for base in ((100, 300), (0, 128)):
        P = Paged([b + n for b, n in zip(base, ns)], ns, 1, D, 16, e4m3=e4m3, seed=9, lead=1, tail=2)
        pages, batch = P.device()
        t = moe.Tree(batch, torch.from_numpy(rows_of(P, [[-1] * n for n in ns])).cuda())
        compare(monkeypatch, P, G, t, batch, pages, [(np.zeros((n, n), dtype=bool), [0] * n) for n in ns], window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("D,G", [(64, 8), (128, 2), (128, 8), (256, 1), (256, 8)])
def test_nodes_past_the_words_of_the_masks(monkeypatch, D, G, window, e4m3):
    """Masks of one word: nodes from the 32nd on are nobody's, and the call that prepares them says so."""
    ns = [40, 32, 35]
    P = Paged([140, 32, 400], ns, 1, D, 16, e4m3=e4m3, seed=4)
    pages, full = P.device()
    batch = moe.KvBatch(full.q_start, full.kv_len, full.page_table, P.T, 32)
    parents = [random_parents(n, 3, n) for n in ns]
    t, err = moe.Tree(batch, torch.from_numpy(rows_of(P, parents)).cuda()), torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_tree_prepare(batch, t, err=err)
    assert err.item() == moe.MOE_ERANGE and t.words == 1
    masks = []
    for p in parents:
        m, d = sees(p), depths(p)
        m[32:] = False
        masks.append((m, d[:32] + [0] * (len(p) - 32)))
    compare(monkeypatch, P, G, t, batch, pages, masks, window)

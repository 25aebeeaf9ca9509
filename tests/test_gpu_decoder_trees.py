"""The decoder with drafted trees, forks and norms of heads: every way down a tree is a request of its own."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import inputs as I
from serving_router_top_gb300 import moe
from serving_router_top_gb300.decoder import AttentionShape, Decoder
from tests.attn_util import U_BF16
from tests.gpu_util import require_gpu
from tests.tree_util import chains, random_parents

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def small(requests, s, layers=2):
    # every token takes every expert: no routing decision that a rounding could turn
    w = I.small_workload(T=4, H=256, I=128, E=4, k=4, I_shared=128, layers=layers, seed=5)
    return Decoder(w, s, requests=requests, max_len=96, maxT=128)


def near(got, ref):
    # as in the decoder's other tests: a few bf16 roundings of a row's size
    err = (got.float().cpu() - ref.float().cpu()).norm(dim=1) / ref.float().cpu().norm(dim=1)
    return float(err.max()) <= 16 * U_BF16


SHAPES = [AttentionShape(8, 2, 64, 64, page=16), AttentionShape(4, 4, 128, 32, page=8, window=20, qk_norm=True),
          AttentionShape(6, 1, 64, 16, page=32, e4m3=True, qk_norm=True), AttentionShape(8, 1, 256, 64, page=16, qk_norm=True)]


@pytest.mark.parametrize("s", SHAPES)
def test_ways_down_a_tree_are_chains(s):
    g = torch.Generator().manual_seed(0)
    prompt, parents = [20, 33], [random_parents(9, 3, 1), random_parents(6, 2, 2)]
    x = [torch.randn(n + len(p), 256, generator=g) for n, p in zip(prompt, parents)]
    d = small(2, s)
    d.forward(torch.cat([t[:n] for t, n in zip(x, prompt)]).cuda(), d.batch(prompt))
    bt, tree = d.tree_batch(parents)
    out = d.forward(torch.cat([t[n:] for t, n in zip(x, prompt)]).cuda(), bt, tree).clone()
    d.check()
    at = 0
    for r in range(2):
        for way in chains(parents[r])[-3:]:
            c = small(1, s)
            rows = torch.cat([x[r][:prompt[r]], x[r][prompt[r]:][way]]).cuda()
            ref = c.forward(rows, c.batch([len(rows)]))[prompt[r]:]
            assert near(out[at:at + len(parents[r])][way], ref)
        at += len(parents[r])


@pytest.mark.parametrize("s", SHAPES)
def test_what_is_kept_is_what_goes_on(s):
    """Trees, their verification with a target that is sure of a way, and the tokens after it, against a request that
    only had the kept ones."""
    g = torch.Generator().manual_seed(3)
    parents = [[-1, 0, 0, 1, 2, 4, 4, 6], [-1, 0, 1, 1], []]
    ways = [[0, 2, 4, 6], [0], []]
    prompt, after, V = [18, 30, 5], [3, 1, 2], 50
    x = [torch.randn(n + len(p) + a, 256, generator=g) for n, p, a in zip(prompt, parents, after)]
    d = small(3, s)
    d.forward(torch.cat([t[:n] for t, n in zip(x, prompt)]).cuda(), d.batch(prompt))
    bt, tree = d.tree_batch(parents)
    d.forward(torch.cat([t[n:n + len(p)] for t, n, p in zip(x, prompt, parents)]).cuda(), bt, tree)
    T = bt.c.T
    token = torch.arange(10, 10 + T, dtype=torch.int32)
    target = torch.zeros(T, V)
    at = 0
    for p, way in zip(parents, ways):
        for i in range(len(p)):
            nxt = [c for c in way if p[c] == i]
            target[at + i, int(token[at + nxt[0]]) if nxt else 49 - i] = 1.0
        at += len(p)
    desc = moe.verify_desc(target.cuda(), token.cuda(), tree.parent, torch.full((T,), 0.5).cuda(), torch.full((3,), 0.5).cuda())
    paths, nxt = d.accept(bt, desc)
    assert paths == ways and nxt == [49 - 6, 49, -1]
    assert d.lens == [22, 31, 5]
    out = d.forward(torch.cat([t[len(t) - a:] for t, a in zip(x, after)]).cuda(), d.batch(after))
    d.check()
    at = 0
    for r in range(3):
        c = small(1, s)
        rows = torch.cat([x[r][:prompt[r]], x[r][prompt[r]:][ways[r]], x[r][len(x[r]) - after[r]:]]).cuda()
        ref = c.forward(rows, c.batch([len(rows)]))[len(rows) - after[r]:]
        assert near(out[at:at + after[r]], ref)
        at += after[r]


@pytest.mark.parametrize("s", SHAPES[:2])
def test_forks_go_their_own_ways(s):
    g = torch.Generator().manual_seed(4)
    x, y, z = (torch.randn(n, 256, generator=g) for n in (37, 6, 6))
    d = small(2, s)
    d.forward(x.cuda(), d.batch([37, 0]))
    d.fork(0, 1)
    out = d.forward(torch.cat([y, z]).cuda(), d.batch([6, 6])).clone()
    d.check()
    for r, tail in enumerate((y, z)):
        c = small(1, s)
        ref = c.forward(torch.cat([x, tail]).cuda(), c.batch([43]))[37:]
        assert near(out[6 * r:6 * r + 6], ref)
    d.release(0)
    again = d.forward(y[:2].cuda(), d.batch([2, 0]))
    c = small(1, s)
    assert near(again, c.forward(y[:2].cuda(), c.batch([2]))) and d.lens == [2, 43]


def test_trees_that_are_none_are_refused():
    d = small(1, SHAPES[0])
    d.forward(torch.randn(8, 256).cuda(), d.batch([8]))
    for bad in ([[-1, 1]], [[0]], [[-1, -2]], [[-1] * 257]):
        with pytest.raises(ValueError):
            d.tree_batch(bad)
    assert d.lens == [8]
    with pytest.raises(ValueError):
        d.fork(0, 0)
    assert np.asarray(d.lens).tolist() == [8]

"""Forks, releases and other requests' tokens between a tree's forward pass and its verification."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.gpu_util import require_gpu
from tests.test_gpu_decoder_trees import SHAPES, near, small

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def alone(s, rows, last):
    """The last rows of a request of its own."""
    c = small(1, s)
    return c.forward(rows.cuda(), c.batch([len(rows)]))[len(rows) - last:]


@pytest.mark.parametrize("s", SHAPES[:2])
def test_others_go_on_while_a_tree_is_open(s):
    g = torch.Generator().manual_seed(7)
    rows = lambda n: torch.randn(n, 256, generator=g)  # noqa: E731
    a, b, c = rows(19), rows(33), rows(21)       # requests 0, 1 and 2; 3 is to be a fork of 1
    d = small(4, s)
    d.forward(torch.cat([a, b, c]).cuda(), d.batch([19, 33, 21, 0]))
    tree, other = rows(4), rows(2)
    bt, masks = d.tree_batch([[-1, 0, 0, 2], [], [-1, 0], []])
    d.forward(torch.cat([tree, other]).cuda(), bt, masks)
    d.fork(1, 3)
    d.release(2)
    more = rows(5)
    d.forward(more[:3].cuda(), d.batch([0, 3, 0, 0]))
    # the way 0, 2, 3 of request 0's tree
    target = torch.eye(8, device="cuda")[[5, 1, 6, 7, 0, 0]].contiguous()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    half = torch.full((6,), 0.5, device="cuda")
    desc = moe.verify_desc(target, i32([0, 3, 5, 6, 0, 0]), masks.parent, half, half[:4].contiguous())
    assert d.accept(bt, desc) == ([[0, 2, 3], [], [], []], [7, -1, -1, -1])
    assert d.lens == [22, 36, 0, 33]
    tail = rows(11)
    out = d.forward(torch.cat([tail[:3], more[3:], tail[3:7], tail[7:]]).cuda(), d.batch([3, 2, 4, 4]))
    d.check()
    ways = [torch.cat([a, tree[[0, 2, 3]], tail[:3]]), torch.cat([b, more]), tail[3:7], torch.cat([b, tail[7:]])]
    at = 0
    for way, last in zip(ways, (3, 2, 4, 4)):
        assert near(out[at:at + last], alone(s, way, last))
        at += last

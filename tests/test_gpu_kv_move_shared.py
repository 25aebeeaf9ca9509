"""Kept nodes in pools that layers share, and a layer whose keys are its values: each place moves once."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.gpu_util import require_gpu
from tests.test_gpu_kv_move import Step, pools

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# a place that is moved to is the next one's source, so a second move of a pool shows
PATH = [0, 2, 4, 6, 8, 9, 12, 18, 24, 36]


def step():
    return Step([300, 70, 48], [48] * 3, 16, [PATH, PATH, [0] + list(range(10, 48))])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("order", [[0, 0], [0, 1, 0, 1], [2, 0, 1, 1, 0, 2, 2], [0] * 100, [0, 1, 2] * 50, [0] + [1] * 299])
def test_layers_that_share_a_pool(order, e4m3):
    s = step()
    for _ in range(3):
        raw, layers = pools(3, s.npages, 8, 16, 128, e4m3)
        want, lens = s.expect(raw)
        untouched = [l for l in range(3) if l not in order]
        want[untouched] = raw[untouched]
        assert s.run(moe.KvLayers([layers.layers[l] for l in order])) == (lens, 0)
        assert torch.equal(raw, want)


def test_keys_that_are_values():
    s = step()
    for _ in range(3):
        raw, layers = pools(4, s.npages, 8, 16, 128)
        want, lens = s.expect(raw)
        want[:, 1] = raw[:, 1]
        assert s.run(moe.KvLayers([moe.KvPages(p.k, p.k) for p in layers.layers])) == (lens, 0)
        assert torch.equal(raw, want)

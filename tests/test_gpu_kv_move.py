"""Kept nodes moved to the front of their trees and pages copied, in every layer: byte for byte."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def pools(L, npages, Hkv, page, D, e4m3=False, layout="hnd", seed=0):
    """Bytes of L layers' keys and values and the tensors over them."""
    g = torch.Generator().manual_seed(seed)
    size = 1 if e4m3 else 2
    shape = {"hnd": (L, 2, npages, Hkv, page, D * size), "nhd": (L, 2, npages, page, Hkv, D * size),
             "kv": (L, npages, 2, Hkv, page, D * size)}[layout]
    raw = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
    typed = raw.view(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    view = lambda x: {"hnd": x, "nhd": x.transpose(3, 4), "kv": x.transpose(1, 2)}[layout]  # noqa: E731
    return view(raw), moe.KvLayers([moe.KvPages(x[0], x[1]) for x in view(typed)])


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Step:
    def __init__(self, lens, ns, page, paths, width=None, lead=0, seed=0, spare=2):
        r = np.random.RandomState(seed)
        self.lens, self.ns, self.page, self.paths = lens, ns, page, paths
        per = [-(-max(n, 0) // page) for n in lens]
        self.npages = sum(per) + spare
        order = r.permutation(self.npages)
        self.table = np.full((len(lens), max(per + [1]) + 1), -1)
        at = 0
        for b, m in enumerate(per):
            self.table[b, :m] = order[at:at + m]
            at += m
        start = np.concatenate([[lead], lead + np.cumsum(ns)])
        self.batch = moe.KvBatch(i32(start), i32(lens), i32(self.table), int(start[-1]), max(ns + [1]))
        width = width or max([len(p) for p in paths] + [1])
        self.path = np.full((len(lens), width), -1)
        for b, p in enumerate(paths):
            self.path[b, :len(p)] = p
        self.count = np.array([len(p) for p in paths])

    def expect(self, raw):
        raw = raw.clone()
        for b, p in enumerate(self.paths):
            base = self.lens[b] - self.ns[b]
            old = [raw[:, :, self.table[b, (base + i) // self.page], :, (base + i) % self.page].clone() for i in p]
            for d, x in enumerate(old):
                raw[:, :, self.table[b, (base + d) // self.page], :, (base + d) % self.page] = x
        return raw, [l - n + len(p) for l, n, p in zip(self.lens, self.ns, self.paths)]

    def run(self, layers, stream=None):
        out, err = torch.full((len(self.lens),), -5, dtype=torch.int32, device="cuda"), i32([0])
        moe.moe_kv_compact(layers, self.batch, i32(self.path), i32(self.count), out, err=err)
        return out.tolist(), err.item()


PATHS = [[0], [0, 1, 2], [0, 3, 4, 9], [0, 9], [0, 1, 5, 6, 7, 8, 9], list(range(10)), []]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("D,Hkv,page", [(64, 1, 16), (128, 3, 4), (256, 8, 64), (64, 40, 128), (256, 2, 1)])
def test_kept_nodes(D, Hkv, page, layout, e4m3):
    s = Step([10, 33, 100, 11, 70, 64, 10], [10] * 7, page, PATHS, width=12, lead=2)
    raw, layers = pools(3, s.npages, Hkv, page, D, e4m3, layout)
    want, lens = s.expect(raw)
    got, err = s.run(layers)
    assert err == 0 and got == lens
    assert torch.equal(raw, want)


@pytest.mark.parametrize("L", [1, 2, 127, 128, 129, 300])
def test_layers(L):
    s = Step([20, 7], [8, 6], 8, [[0, 2, 3, 7], [0, 5]])
    raw, layers = pools(L, s.npages, 1, 8, 64)
    want, lens = s.expect(raw)
    assert s.run(layers) == (lens, 0)
    assert torch.equal(raw, want)


def test_long_paths_and_no_nodes():
    """More kept nodes than one turn of the kernel, requests without nodes, and lengths alone."""
    r = np.random.RandomState(3)
    p = np.sort(r.permutation(np.arange(1, 700))[:560]).tolist()
    s = Step([900, 50, 700], [700, 0, 700], 16, [[0] + p, [], [0] + list(range(150, 699))])
    raw, layers = pools(2, s.npages, 2, 16, 64)
    want, lens = s.expect(raw)
    assert s.run(layers) == (lens, 0)
    assert torch.equal(raw, want)


@pytest.mark.parametrize("path,kept", [([0, 3, 3, 5], 2), ([0, 3, 2], 2), ([0, 10], 1), ([-1], 0), ([0, 2, -1], 2),
                                       ([2 ** 31 - 1], 0), ([1, 0], 1)])
def test_a_path_ends_before_an_index_that_does_not_rise(path, kept):
    s = Step([40, 30], [10, 10], 16, [path, [0, 4]])
    raw, layers = pools(2, s.npages, 2, 16, 64)
    s.paths[0] = path[:kept]
    want, lens = s.expect(raw)
    got, err = s.run(layers)
    assert err == moe.MOE_ERANGE and got == lens
    assert torch.equal(raw, want)


def test_counts_are_cut():
    s = Step([40, 30, 20], [10, 10, 10], 16, [[0, 4, 5], [0, 4], [0, 7]])
    raw, layers = pools(1, s.npages, 2, 16, 64)
    s.count[:] = [99, -3, 2]
    s.path[0, 2] = 5
    s.paths[1] = []
    want, lens = s.expect(raw)
    assert s.run(layers) == (lens, 0)
    assert torch.equal(raw, want)


def test_pages_that_are_not_there():
    s = Step([40, 30], [10, 10], 16, [[0, 4, 5], [0, 4]])
    raw, layers = pools(2, s.npages, 2, 16, 64)
    want, lens = s.expect(raw)
    for bad in (-1, s.npages, 2 ** 31 - 1):
        raw2, layers2 = pools(2, s.npages, 2, 16, 64)
        s.batch.page_table[0, 2] = bad   # places 32 .. 47: two of the three sources
        got, err = s.run(layers2)
        assert err == moe.MOE_ERANGE and got == lens
        only, _ = Step([40, 30], [10, 10], 16, [[0], [0, 4]]).expect(raw)
        assert torch.equal(raw2, only)


def test_verified_on_the_device():
    """The path and count that verification left on the device, in one captured sequence."""
    from tests.test_gpu_verify import Case
    c = Case([9, 6, 4], 500, False, spread=2, seed=3, near=0.1)
    s = Step([30, 6, 50], [9, 6, 4], 16, [[]] * 3)
    batch, desc = c.device()
    path, count, token, lens = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((3, 9), (3,), (3,), (3,)))
    raw, layers = pools(2, s.npages, 2, 16, 128)
    start = raw.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            moe.moe_verify_drafts(batch, desc, path, count, token)
            moe.moe_kv_compact(layers, s.batch, path, count, lens)
        graph.replay()
    torch.cuda.synchronize()
    want = c.expect(9)
    s.paths = [p[:n].tolist() for p, n in zip(want[0], want[1])]
    moved, now = s.expect(start)
    assert torch.equal(raw, moved) and lens.tolist() == now and count.tolist() == want[1]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("D,Hkv,page,L", [(64, 1, 2, 1), (128, 3, 16, 2), (256, 8, 64, 2), (128, 5, 128, 130), (64, 2, 256, 1)])
def test_pages_are_copied(D, Hkv, page, L, layout, e4m3):
    raw, layers = pools(L, 9, Hkv, page, D, e4m3, layout)
    want = raw.clone()
    src, dst, tokens = [1, 4, 1, 8], [0, 2, 7, 5], [page, page // 2, 0, page - 1]
    for a, b in zip(src, dst):
        want[:, :, b] = raw[:, :, a]
    moe.moe_kv_copy_pages(layers, i32(src), i32(dst))
    assert torch.equal(raw, want)
    raw, layers = pools(L, 9, Hkv, page, D, e4m3, layout, seed=1)
    want = raw.clone()
    for a, b, t in zip(src, dst, tokens):
        want[:, :, b, :, :t] = raw[:, :, a, :, :t]
    moe.moe_kv_copy_pages(layers, i32(src), i32(dst), tokens=i32(tokens))
    assert torch.equal(raw, want)


def test_copies_out_of_range():
    raw, layers = pools(2, 6, 2, 16, 64)
    want = raw.clone()
    want[:, :, 3] = raw[:, :, 2]
    want[:, :, 4, :, :16] = raw[:, :, 1, :, :16]
    err = i32([0])
    moe.moe_kv_copy_pages(layers, i32([2, 0, -1, 6, 1, 0]), i32([3, 6, 5, 5, 4, 5]), tokens=i32([16, 16, 16, 16, 99, -7]), err=err)
    assert err.item() == moe.MOE_ERANGE
    assert torch.equal(raw, want)


def test_many_pages():
    raw, layers = pools(1, 3000, 1, 2, 64)
    order = np.random.RandomState(0).permutation(3000)
    want = raw.clone()
    want[:, :, order[1500:]] = raw[:, :, order[:1500]]
    moe.moe_kv_copy_pages(layers, i32(order[:1500]), i32(order[1500:]))
    assert torch.equal(raw, want)


def test_pools_past_four_gigabytes():
    """Pages whose bytes lie past 2^32, copied and moved in."""
    page, D, npages = 64, 256, 140000  # 32 KB a page
    k, v = (torch.empty(npages, 1, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layers = moe.KvLayers([moe.KvPages(k, v)])
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 1, page, D, generator=g).to(torch.bfloat16).cuda()
    for pool in (k, v):
        pool[5], pool[npages - 2] = x[0], x[1]
    moe.moe_kv_copy_pages(layers, i32([5, npages - 2]), i32([npages - 1, 7]))
    for pool in (k, v):
        assert torch.equal(pool[npages - 1], x[0]) and torch.equal(pool[7], x[1])
    batch = moe.KvBatch(i32([0, 10]), i32([70]), i32([[npages - 1, npages - 2]]), 10, 10)
    lens = i32([0])
    moe.moe_kv_compact(layers, batch, i32([[0, 5, 8, -1]]), i32([3]), lens)
    for pool in (k, v):  # places 60, 65 and 68 to 60, 61 and 62
        want = x[0].clone()
        want[0, 61], want[0, 62] = x[1, 0, 1], x[1, 0, 4]
        assert torch.equal(pool[npages - 1], want)
    assert lens.tolist() == [63]


def test_lengths_in_32_bits():
    """A request whose length is past the table: nothing is read or written astray, and the length is told."""
    s = Step([40], [10], 16, [[0, 4, 5]])
    raw, layers = pools(1, s.npages, 2, 16, 64)
    want = raw.clone()
    for length in (2 ** 31 - 1, 49 + 16 * 1000, 5, 0, -2 ** 31):
        s.batch.kv_len.fill_(length)
        got, err = s.run(layers)
        assert err == moe.MOE_ERANGE and got == [max(length - 10 + 3, -2 ** 31)]
        assert torch.equal(raw, want)

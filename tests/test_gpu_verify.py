"""Verification of drafted trees against the definition in whole numbers: every index is equal."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.gpu_util import require_gpu
from tests.tree_util import random_parents, verify_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Case:
    """Requests of ns nodes with random trees, probabilities over V tokens and random numbers."""

    def __init__(self, ns, V, drawn, spread=3, seed=0, sharp=2.0, lead=0, tail=0, near=0.7):
        r = np.random.RandomState(seed)
        self.ns, self.V, self.drawn, self.lead = list(ns), V, drawn, lead
        self.T = lead + sum(ns) + tail
        self.start = np.concatenate([[lead], lead + np.cumsum(ns)]).astype(np.int32)
        logits = r.randn(self.T, V) * sharp
        soft = lambda x: (lambda e: (e / e.sum(1, keepdims=True)).astype(np.float32))(np.exp(x - x.max(1, keepdims=True)))  # noqa: E731
        self.target = soft(logits)
        self.draft = soft(logits + near * r.randn(self.T, V))
        self.parents = [random_parents(n, spread, seed + n) if n else [] for n in ns]
        self.parent = np.full(self.T, 3, dtype=np.int32)
        self.token = r.randint(0, V, self.T).astype(np.int32)
        for b, p in enumerate(self.parents):
            used = {}
            for i, up in enumerate(p):
                t = self.start[b] + i
                self.parent[t] = up
                if up >= 0:
                    q = self.draft[self.start[b] + up].astype(np.float64)
                    if drawn:
                        self.token[t] = r.choice(V, p=q / q.sum())
                    else:
                        used[up] = used.get(up, -1) + 1
                        self.token[t] = np.argsort(-q, kind="stable")[min(used[up], V - 1)]
        self.u = r.rand(self.T).astype(np.float32)
        self.u_last = r.rand(len(ns)).astype(np.float32)

    def expect(self, most):
        paths, tokens = np.full((len(self.ns), most), -1, dtype=np.int32), []
        count = []
        for b, n in enumerate(self.ns):
            rows = slice(self.start[b], self.start[b] + n)
            path, token = verify_ref(self.parent[rows].tolist(), self.token[rows], self.u[rows], self.u_last[b],
                                     self.target[rows], self.draft[rows] if self.drawn else None, most)
            paths[b, :len(path)] = path
            count.append(len(path))
            tokens.append(token)
        return paths, count, tokens

    def device(self, stride=None, shift=0, draft_shift=None):
        """(batch, desc) with rows `stride` elements apart, from element `shift` of an allocation on."""
        def rows(x, at):
            w = stride or self.V
            flat = torch.full((self.T * w + at + 4,), float("nan"), device="cuda")
            view = flat[at:at + self.T * w].view(self.T, w)[:, :self.V]
            view.copy_(torch.from_numpy(x))
            return view
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()  # noqa: E731
        B = len(self.ns)
        batch = moe.KvBatch(i32(self.start), i32(np.zeros(B)), i32(np.zeros((B, 1))), self.T, max(self.ns + [1]))
        self.desc = moe.verify_desc(rows(self.target, shift), i32(self.token), i32(self.parent), torch.from_numpy(self.u).cuda(),
                                    torch.from_numpy(self.u_last).cuda(),
                                    draft=rows(self.draft, shift if draft_shift is None else draft_shift) if self.drawn else None)
        return batch, self.desc

    def run(self, most, **kw):
        batch, desc = self.device(**kw)
        B = len(self.ns)
        path, count, token, err = (torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((B, most), (B,), (B,), (1,)))
        err.zero_()
        moe.moe_verify_drafts(batch, desc, path, count, token, err=err)
        return path.cpu().numpy(), count.tolist(), token.tolist(), err.item()

    def check(self, most=None, error=0, **kw):
        most = most or max(self.ns + [1])
        path, count, token, err = self.run(most, **kw)
        want = self.expect(most)
        assert err == error
        assert (path == want[0]).all()
        assert count == want[1] and token == want[2]
        return want


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 31, 127, 128, 129, 1000, 4099])
def test_vocabularies(V, drawn):
    Case([5, 1, 0, 9, 3, 17, 2, 4], V, drawn, seed=V).check()


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("n,spread", [(1, 1), (2, 1), (12, 1), (33, 40), (64, 3), (65, 2), (256, 8), (256, 300)])
def test_trees(n, spread, drawn):
    Case([n] * 3, 300, drawn, spread=spread, seed=n, near=0.2).check()


@pytest.mark.parametrize("drawn", [True, False])
def test_many_requests(drawn):
    """Every length of a path is met, and refusals of one to several children."""
    r = np.random.RandomState(1)
    want = Case(r.randint(0, 12, 400).tolist(), 64, drawn, spread=3, seed=4, near=0.4, lead=3, tail=2).check()
    assert {1, 2, 3, 4} <= set(want[1]) and 0 in want[1]


@pytest.mark.parametrize("shift,stride,draft_shift", [(0, 1003, 0), (1, 1001, 1), (2, 1006, 3), (3, 1000, 0)])
def test_rows_anywhere(shift, stride, draft_shift):
    Case([6, 7, 3], 1000, True, seed=2).check(stride=stride, shift=shift, draft_shift=draft_shift)


def test_a_large_vocabulary():
    for drawn in (True, False):
        Case([4, 2], 140001, drawn, spread=2, seed=9, sharp=1.0).check()


@pytest.mark.parametrize("most", [1, 2, 3])
def test_paths_cut_short(most):
    want = Case([9] * 40, 50, True, spread=1, seed=3, near=0.1).check(most=most)
    assert max(want[1]) == most


@pytest.mark.parametrize("drawn", [True, False])
def test_borders(drawn):
    """Probabilities and random numbers of few bits, where u s q = R and running sums meet the threshold exactly."""
    r = np.random.RandomState(7)
    c = Case([4] * 300, 4, drawn, spread=3, seed=1)
    rows = np.array([[8, 0, 0, 0], [4, 4, 0, 0], [2, 2, 2, 2], [0, 1, 3, 4], [0, 0, 0, 8], [1, 0, 6, 1]], dtype=np.float32) / 8
    c.target, c.draft = rows[r.randint(0, 6, c.T)], rows[r.randint(0, 6, c.T)]
    c.token = r.randint(0, 4, c.T).astype(np.int32)
    c.u = (r.randint(0, 8, c.T) / 8).astype(np.float32)
    c.u_last = (r.randint(0, 8, 300) / 8).astype(np.float32)
    c.check()


@pytest.mark.parametrize("drawn", [True, False])
def test_values_that_are_no_probabilities(drawn):
    r = np.random.RandomState(8)
    c = Case([5] * 60, 40, drawn, spread=3, seed=5)
    for x in (c.target, c.draft):
        x[r.rand(*x.shape) < 0.1] = np.nan
        x[r.rand(*x.shape) < 0.1] = -0.5
        x[r.rand(*x.shape) < 0.02] = np.float32(1e-30)
        x[r.rand(*x.shape) < 0.02] = np.float32(1e-42)
        x[::7] = 0.0
    c.target[3::11, 5] = np.inf
    c.u[::5] = np.nan
    c.u[1::5] = 1.0
    c.u[2::5] = -1.0
    c.u_last[::3] = 1.5
    c.u_last[1::3] = 0.0
    want = c.check()
    assert -1 in want[2]


def test_nothing_left_goes_back_to_the_target():
    """All of a row's mass on refused children."""
    c = Case([3] * 4, 8, False, spread=1, seed=1)
    c.parent[:] = np.tile([-1, 0, 0], 4)
    c.parents = [[-1, 0, 0]] * 4
    c.target[:] = 0.0
    c.target[:, 2], c.target[:, 5] = 0.5, 0.25
    c.token[:] = np.tile([0, 2, 5], 4)
    c.u[:] = 0.999
    c.u_last[:] = [0.1, 0.6, 0.7, 0.9]
    want = c.check()
    assert want[2] == [2, 2, 5, 5] and want[1] == [1] * 4


def test_tokens_and_parents_out_of_range():
    for drawn in (True, False):
        c = Case([8] * 30, 20, drawn, spread=3, seed=6, near=0.1)
        r = np.random.RandomState(2)
        c.token[r.rand(c.T) < 0.2] = 20
        c.token[r.rand(c.T) < 0.1] = -1
        c.token[r.rand(c.T) < 0.05] = 2 ** 31 - 1
        wild = r.rand(c.T) < 0.1
        wild[::8] = False
        c.parent[wild] = r.choice([-1, -2, 9, 7, 2 ** 31 - 1], int(wild.sum()))
        path, count, token, err = c.run(8)
        fixed = c.parent.reshape(30, 8).copy()
        fixed[fixed >= np.arange(8)] = -1  # a node whose parent is not before it is never reached
        c.parent = fixed.reshape(-1)
        want = c.expect(8)
        assert err == 0 and (path == want[0]).all() and count == want[1] and token == want[2]


def test_more_nodes_than_a_tree_may_have():
    c = Case([300, 4], 30, False, spread=1, seed=1)
    path, count, token, err = c.run(300)
    c.ns[0] = 256
    c2 = c.expect(300)
    assert err == moe.MOE_ERANGE
    assert (path == c2[0]).all() and count == c2[1] and token == c2[2]


def test_starts_that_decrease_are_reported():
    c = Case([3, 3], 30, False, seed=1)
    batch, desc = c.device()
    batch.q_start.copy_(torch.tensor([0, 4, 2], dtype=torch.int32))
    out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 4), (2,), (2,), (1,))]
    moe.moe_verify_drafts(batch, desc, *out[:3], err=out[3])
    assert out[3].item() == moe.MOE_ERANGE and out[1].tolist()[1] == 0 and out[2].tolist()[1] == -1


def test_sums_that_leave_the_range_stay_in_it():
    """Rows of ones: the token is some index, and the call ends."""
    for drawn in (True, False):
        c = Case([6] * 5, 5000, drawn, seed=1)
        c.target[:] = 1.0
        c.draft[:, ::2] = 1.0
        path, count, token, err = c.run(6)
        assert err == 0 and all(-1 <= t < 5000 for t in token) and all(1 <= x <= 6 for x in count)


def test_two_streams_and_a_captured_call():
    a, b = Case([6] * 20, 3001, True, seed=11), Case([9] * 10, 2000, False, seed=12)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs, calls = [], []
    for c, s in ((a, sa), (b, sb)):
        batch, desc = c.device()
        B = len(c.ns)
        out = [torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((B, 9), (B,), (B,))]
        outs.append(out)
        calls.append((batch, desc, s))
    torch.cuda.synchronize()
    for _ in range(20):
        for out, (batch, desc, s) in zip(outs, calls):
            moe.moe_verify_drafts(batch, desc, *out, stream=s)
    torch.cuda.synchronize()
    for c, out in zip((a, b), outs):
        want = c.expect(9)
        assert (out[0].cpu().numpy() == want[0]).all() and out[1].tolist() == want[1] and out[2].tolist() == want[2]
    batch, desc, s = calls[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_verify_drafts(batch, desc, *outs[0])
    a.u, a.u_last = np.random.RandomState(1).rand(a.T).astype(np.float32), np.random.RandomState(2).rand(20).astype(np.float32)
    desc.tensors[3].copy_(torch.from_numpy(a.u))
    desc.tensors[4].copy_(torch.from_numpy(a.u_last))
    graph.replay()
    torch.cuda.synchronize()
    want = a.expect(9)
    assert (outs[0][0].cpu().numpy() == want[0]).all() and outs[0][1].tolist() == want[1] and outs[0][2].tolist() == want[2]


@pytest.mark.parametrize("B,V", [(1, 131072), (1, 7), (9, 20000), (19, 5000), (40, 3000)])
def test_every_size_of_a_cluster(B, V):
    """One request to so many that each has a CTA or two; called, captured and replayed."""
    for drawn in (True, False):
        c = Case([5] * B, V, drawn, spread=2, seed=B, near=0.3)
        want = c.check()
        batch, desc = c.device()
        out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, 5), (B,), (B,))]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                moe.moe_verify_drafts(batch, desc, *out)
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        assert (out[0].cpu().numpy() == want[0]).all() and out[1].tolist() == want[1] and out[2].tolist() == want[2]


def test_many_clusters_of_one():
    c = Case([3] * 700, 200, True, spread=2, seed=2, near=0.3)
    c.check()


def test_rows_past_four_gigabytes():
    """The last request's rows lie past 2^32 bytes, and past 2^31 elements."""
    c = Case([4], 65536, True, spread=2, seed=5, near=0.2)
    lead = (1 << 31) // 65536 + 8
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    T = lead + 4
    rows = [torch.empty(T, 65536, device="cuda") for _ in range(2)]
    for big, small in zip(rows, (c.target, c.draft)):
        big[lead:].copy_(torch.from_numpy(small))
    wide = lambda x, fill: np.concatenate([np.full(lead, fill, dtype=x.dtype), x])  # noqa: E731
    desc = moe.verify_desc(rows[0], i32(wide(c.token, 0)), i32(wide(c.parent, 0)), torch.from_numpy(wide(c.u, 0)).cuda(),
                           torch.from_numpy(c.u_last).cuda(), draft=rows[1])
    batch = moe.KvBatch(i32([lead, T]), i32([0]), i32([[0]]), T, 4)
    out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 4), (1,), (1,))]
    moe.moe_verify_drafts(batch, desc, *out)
    want = c.expect(4)
    assert (out[0].cpu().numpy() == want[0]).all() and out[1].tolist() == want[1] and out[2].tolist() == want[2]

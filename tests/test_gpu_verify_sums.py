"""Verification of rows whose sums leave what probabilities can: a sum above 4 counts as 4, in whatever order it is made."""
import math

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_verify import Case

pytestmark = pytest.mark.gpu
ONE = 1 << 60
MOST = 4 * ONE


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def fixed(row):
    """Exact for what is a multiple of 2^-24."""
    return [int(v) for v in (np.asarray(row, dtype=np.float64).clip(0.0, 1.0) * 2.0 ** 60)]


def chance(x):
    return int(math.floor(math.ldexp(float(x), 64)))


def expect(parents, tokens, u, u_last, target, draft, most):
    """(path, next token): include/moe.h's definition with its sums cut at 4, and s at 0."""
    path, v = [0], 0
    while True:
        p = fixed(target[v])
        rest, s, kept = list(p), ONE, None
        for c in range(v + 1, len(parents)) if len(path) < most else []:
            if parents[c] != v:
                continue
            x = int(tokens[c])
            q = None if draft is None else fixed(draft[v])
            if chance(u[c]) * (s if q is None else s * q[x] // ONE) >> 64 < rest[x]:
                kept = c
                break
            if q is None:
                s, rest[x] = max(s - rest[x], 0), 0
            else:
                rest = [max(a - s * b // ONE, 0) for a, b in zip(rest, q)]
                s = min(sum(rest), MOST)
        if kept is None:
            break
        path.append(kept)
        v = kept
    for row in (rest, p):
        total = min(sum(row), MOST)
        if total:
            t, run = chance(u_last) * total >> 64, 0
            for j, x in enumerate(row):
                run += x
                if run > t:
                    return path, j
    return path, -1


def check(c, most):
    path, count, token, err = c.run(most)
    assert err == 0
    for b in range(len(c.ns)):
        rows = slice(c.start[b], c.start[b] + c.ns[b])
        want, nxt = expect(c.parent[rows].tolist(), c.token[rows], c.u[rows], c.u_last[b], c.target[rows],
                           c.draft[rows] if c.drawn else None, most)
        assert path[b].tolist() == want + [-1] * (most - len(want)) and count[b] == len(want) and token[b] == nxt, b


def test_a_refused_pick_is_not_taken_off_a_cut_sum():
    """Halves: R's running sum passes 0.95 x 4 at the eighth index that is left."""
    for B in (1, 40):
        c = Case([2] * B, 5000, False, spread=1, seed=1)
        c.target[:], c.token[:], c.u[:], c.u_last[:] = 0.5, 3, 0.9, 0.95
        _, count, token, _ = c.run(2)
        assert count == [1] * B and token == [8] * B


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,V,n", [(1, 5000, 6), (1, 140001, 4), (9, 20000, 6), (70, 30011, 5), (320, 600, 6), (700, 90, 12)])
def test_rows_of_any_size(B, V, n, drawn):
    """Rows of eighths that sum from a fraction to thousands, at every size of a cluster."""
    r = np.random.RandomState(B + V)
    c = Case([n] * B, V, drawn, spread=4, seed=2) if V < 10000 else Case([n] * B, V, drawn, spread=4, seed=2, sharp=0.5)
    dense = 10.0 ** -r.randint(0, 5, (c.T, 1))
    for x in (c.target, c.draft):
        x[:] = (r.randint(0, 9, x.shape) * (r.rand(*x.shape) < dense) / 8).astype(np.float32)
    c.token = r.randint(0, min(V, 12), c.T).astype(np.int32)
    c.target[:, :12] = (r.randint(0, 9, (c.T, 12)) / 8).astype(np.float32)
    c.draft[:, :12] = (r.randint(1, 9, (c.T, 12)) / 8).astype(np.float32)
    c.u = (r.randint(1, 64, c.T) / 64).astype(np.float32)
    c.u_last = (r.randint(0, 64, B) / 64).astype(np.float32)
    check(c, n)

"""The definition of verification for picked drafts, counted over an even grid of random numbers: the first token after
node 0 has the target's probabilities, to the last point of the grid."""
import itertools

import numpy as np
import pytest

from tests.tree_util import verify_ref

P = np.float32([1 / 8, 1 / 4, 1 / 8, 1 / 4, 1 / 4])


@pytest.mark.parametrize("picks", [[4, 1], [1, 4, 3], [0, 2], [0, 2, 1],
                                   [4, 1, 4],   # a token that is gone: never kept
                                   [9, 3]])     # one outside the vocabulary
def test_picked_drafts_keep_the_targets_distribution(picks):
    """Grids whose points lie on both sides of every threshold R(x) / s, and of the last draw's."""
    n = len(picks) + 1
    axes, s, gone = [], 1.0, set()
    for x in picks:
        p = float(P[x]) if x < 5 and x not in gone else 0.0
        part = next(m for m in range(1, 169) if abs(m * p / s - round(m * p / s)) < 1e-9)
        axes.append(part if p else 1)
        s, gone = s - p, gone | {x}
    left = [float(v) / s if i not in gone else 0.0 for i, v in enumerate(P)]
    axes.append(next(m for m in range(1, 169) if all(abs(m * v - round(m * v)) < 1e-9 for v in left)))
    seen, total = np.zeros(5), 0
    for us in itertools.product(*[[(i + 0.5) / m for i in range(m)] for m in axes]):
        path, nxt = verify_ref([-1] + [0] * (n - 1), [-1] + picks, np.float32([0.0, *us[:-1]]), np.float32(us[-1]), [P] * n, None, n)
        seen[picks[path[1] - 1] if len(path) > 1 else nxt] += 1
        total += 1
    assert (seen == P * total).all(), (seen, P * total)

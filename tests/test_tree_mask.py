"""The bits of keys that a tree's node sees (csrc/tree_mask.h) on the host, as compilers must read them: without
optimisation, with it, and with every step of undefined arithmetic an error."""
import shutil
import subprocess

import numpy as np
import pytest

from serving_router_top_gb300 import build
from tests.tree_util import depths, random_parents, sees, words_of

MAIN = r"""
#include <stdio.h>
#include "tree_mask.h"
int main() {
  int n, words, node, window, node0, end;
  static int depth[512];
  static unsigned row[16], seen[4];
  while (scanf("%d %d %d %d %d %d", &n, &words, &node, &window, &node0, &end) == 6) {
    for (int i = 0; i < n; ++i) if (scanf("%d", depth + i) != 1) return 1;
    for (int w = 0; w < words; ++w) if (scanf("%u", row + w) != 1) return 1;
    moe::attn::seen_keys<2>(row, words, depth, depth[node], window, node0, end, seen);
    printf("%u %u", seen[0], seen[1]);
    moe::attn::seen_keys<4>(row, words, depth, depth[node], window, node0, end, seen);
    printf(" %u %u %u %u\n", seen[0], seen[1], seen[2], seen[3]);
  }
  return 0;
}
"""


@pytest.fixture(scope="module", params=["-O0", "-O2", "-O0 -fwrapv", "-O1 -fsanitize=undefined -fsanitize-trap=undefined"])
def program(request, tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("mask")
    src, exe = where / "main.cpp", where / "main"
    src.write_text(MAIN)
    subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", *request.param.split(), "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    return str(exe)


def cases():
    """(parents, words, node, window, key0, pos0, cap): tiles all over a request of a few to 96 nodes behind pos0 keys."""
    r = np.random.RandomState(0)
    for words in (1, 2, 3):
        for n in (1, 2, 17, 31, 32, 33, 64, 65, 90, 96):
            if n > 32 * words:
                continue
            for pos0 in (0, 1, 31, 32, 100, 1000, 4097, -3, 2 ** 31 - 1 - n):
                for spread in (1, 5, 200):
                    parents = random_parents(n, spread, n + spread)
                    tile = max(pos0, 0) // 128 * 128
                    for key0 in {tile, tile + 64, max(tile - 128, 0), tile + 128, 0}:
                        window = int(r.choice([0, 0, 1, 2, 7, 40, 1000, 2 ** 29 - 1]))
                        cap = int(r.choice([2 ** 29, pos0 + n // 2 if pos0 < 2 ** 20 else 2 ** 29, 640]))
                        # a tile begins before the last key
                        if key0 < min(pos0 + n, cap):
                            yield parents, words, int(r.randint(n)), window, key0, pos0, cap


def test_bits_are_those_of_the_definition(program):
    lines, want, masks = [], [], {}
    for parents, words, node, window, key0, pos0, cap in cases():
        n = len(parents)
        if id(parents) not in masks:
            masks[id(parents)] = parents, sees(parents), depths(parents)
        _, above, deep = masks[id(parents)]
        end = min(cap, max(pos0 + n, 0)) - key0
        lines.append(" ".join(map(str, [n, words, node, window, key0 - pos0, end, *deep,
                                        *words_of(above[node:node + 1], words).view(np.uint32)[0]])))
        row = []
        for j in range(128):
            other = key0 + j - pos0
            sees_it = j < end and (other < 0 or (other < n and above[node, other]))
            if sees_it and window:
                sees_it = (other if other < 0 else deep[other]) > deep[node] - window
            row.append(sees_it)
        w = words_of(np.array([row]), 4).view(np.uint32)[0].tolist()
        want.append(w[:2] + w)
    out = subprocess.run([program], input="\n".join(lines), capture_output=True, text=True)
    assert out.returncode == 0
    got = [list(map(int, line.split())) for line in out.stdout.splitlines()]
    assert len(got) == len(want) > 500
    wrong = [i for i in range(len(want)) if got[i] != want[i]]
    assert not wrong, (len(wrong), lines[wrong[0]], got[wrong[0]], want[wrong[0]])

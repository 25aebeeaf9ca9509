"""Drafted trees for the tests: parents, masks and 64-bit references."""
import math

import numpy as np
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import U_BF16, U_F32, Paged


def random_parents(n, spread, seed):
    """Parent of each of n nodes: one of the `spread` nodes before it; node 0 is the root."""
    r = np.random.RandomState(seed)
    return [-1] + [i - 1 - r.randint(0, min(spread, i)) for i in range(1, n)]


def chains(parents):
    """Each node's way from its root down to itself."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def depths(parents):
    return [len(c) - 1 for c in chains(parents)]


def sees(parents):
    """sees[i, j]: node j is node i or above it."""
    m = np.zeros((len(parents), len(parents)), dtype=bool)
    for i, c in enumerate(chains(parents)):
        m[i, c] = True
    return m


def words_of(bits, words):
    """Rows of truth values as int32 words, the lowest bit first."""
    x = np.zeros((bits.shape[0], 32 * words), dtype=np.uint64)
    x[:, :bits.shape[1]] = bits
    return (x.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(2).astype(np.uint32).view(np.int32)


def rows_of(P: Paged, parents):
    """parent [T] of a cache's rows: those of no request hold junk."""
    p = np.full(P.T, 77, dtype=np.int32)
    for b, t in enumerate(parents):
        p[P.start[b]:P.start[b] + P.ns[b]] = t
    return p


def tree_of(P: Paged, batch, parents):
    """A prepared moe.Tree."""
    t = moe.Tree(batch, torch.from_numpy(rows_of(P, parents)).cuda())
    moe.moe_tree_prepare(batch, t)
    return t


def tree_attention_ref(P: Paged, q, Hq, scale, window, parents):
    """(o, bound) as attn_util.attention_ref's, of tree nodes."""
    G, D = Hq // P.Hkv, P.D
    o = torch.full((P.T, Hq, D), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(o)
    for b in range(P.B):
        n, L = P.ns[b], max(P.lens[b], 0)
        rows = slice(int(P.start[b]), int(P.start[b]) + n)
        base = P.lens[b] - n
        hidden = np.zeros((n, L), dtype=bool)
        hidden[:, max(base, 0):] = ~sees(parents[b])[:, max(-base, 0):]
        if window:
            at = base + np.array(depths(parents[b]), dtype=np.int64)
            where = np.concatenate([np.arange(max(base, 0)), at[max(-base, 0):]])
            hidden |= where <= at.reshape(-1, 1) - window
        hidden = torch.from_numpy(hidden).view(n, 1, L)
        for h in range(P.Hkv):
            qh = q[rows, h * G:(h + 1) * G].double()
            k, v = P.rows("k", b, h), P.rows("v", b, h)
            # what a row does not see counts as nothing, whatever it holds
            s = torch.einsum("tgd,jd->tgj", qh, k) * scale
            w = torch.softmax(s.masked_fill(hidden, -math.inf), -1).masked_fill(hidden, 0.0)
            vv = v.unsqueeze(0).expand(n, L, D).masked_fill(hidden.view(n, L, 1), 0.0)
            o[rows, h * G:(h + 1) * G] = torch.einsum("tgj,tjd->tgd", w, vv)
            mag = torch.einsum("tgj,tjd->tgd", w, vv.abs())
            size = (torch.einsum("tgd,jd->tgj", qh.abs(), k.abs()) * abs(scale)).masked_fill(hidden, 0.0)
            ds = 2 * D * U_F32 * size.amax(-1, keepdim=True) if L else torch.zeros(n, G, 1).double()
            tol[rows, h * G:(h + 1) * G] = mag * (U_BF16 + 2 * ds + 2.0 ** -21 + 2 * L * U_F32)
    return o, tol + o.abs() * U_BF16 * (1 + 2.0 ** -8) + 1e-30


def verify_ref(parents, tokens, u, u_last, target, draft, most):
    """(path, next token) of one request, every step in whole numbers of 2^-60: the definition as include/moe.h gives it."""
    one = 1 << 60

    def fixed(row):
        x = np.nan_to_num(np.asarray(row, dtype=np.float64), nan=0.0, posinf=1.0, neginf=0.0).clip(0.0, 1.0)
        return [int(v) for v in np.floor(x * 2.0 ** 60)]  # exact: a power of two times a double below 2^61

    def chance(x):
        x = float(x)
        x = 0.0 if not x > 0.0 else min(x, 1.0 - 2.0 ** -24)
        return int(math.floor(math.ldexp(x, 64)))

    n = len(parents)
    if n == 0:
        return [], -1
    V = len(target[0])
    path, v = [0], 0
    while True:
        p = fixed(target[v])
        q = None if draft is None else fixed(draft[v])
        rest, s, kept = list(p), one, None
        for c in range(v + 1, n) if len(path) < most else []:
            if parents[c] != v:
                continue
            x = int(tokens[c])
            inside = 0 <= x < V
            r = rest[x] if inside else 0
            odds = s if q is None else s * (q[x] if inside else 0) // one
            if chance(u[c]) * odds >> 64 < r:
                kept = c
                break
            if q is None:
                s -= r
                if inside:
                    rest[x] = 0
            else:
                rest = [max(a - s * b // one, 0) for a, b in zip(rest, q)]
                s = sum(rest)
        if kept is None:
            break
        path.append(kept)
        v = kept
    for row in (rest, p):
        total = sum(row)
        if total:
            t, run = chance(u_last) * total >> 64, 0
            for j, x in enumerate(row):
                run += x
                if run > t:
                    return path, j
    return path, -1

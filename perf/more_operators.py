"""A decoding step of drafted token trees over the paged cache, measured operator by operator.

Requests draft trees of tokens: node 0 is the last token of the request, every other
node follows its parent.  One pass of the model verifies a tree:

* ``append``: norm of each head's queries and keys, rotation by position (a node's is
  that of its depth), keys and values into the cache's pages; the tree's depths and
  masks, which every layer uses, are made in the same pass.
* ``attn``: attention of every node over its request's pages and its own ancestors.
* ``verify``: which drafted tokens the target's probabilities keep, and the next token,
  from given random numbers.
* ``compact``: the keys and values of the kept nodes move together, in every layer.
* ``copy``: pages of a cache copied, in every layer (a fork of a request).

``run`` computes them in plain torch where ``own`` is false, and through the
package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BF = torch.bfloat16


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one request's tree of 16 nodes behind a hidden-2048 layer: latency
        dict(name="append_tree16", op="append", B=1, n=16, ragged=False, spread=6, Hq=16, Hkv=2, D=256, rot=64,
             interleaved=False, page=64, lo=1021, hi=1021, e4m3=False),
        # trees of 8 nodes of a batch of 64 at far positions, 8-bit cache
        dict(name="append_batch64_e4m3", op="append", B=64, n=8, ragged=True, spread=4, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=True, page=16, lo=9, hi=262144, e4m3=True),
        # a prompt chunk of 8192 tokens of a model with norms of queries and keys: no tree
        dict(name="append_prefill8192", op="append", B=2, n=4096, ragged=False, spread=0, Hq=32, Hkv=4, D=128, rot=128,
             interleaved=False, page=64, lo=4096, hi=9001, e4m3=False),
        # one request's tree of 8 nodes over a short context: latency
        dict(name="attn_tree8", op="attn", B=1, n=8, ragged=False, spread=4, Hq=16, Hkv=2, D=256, page=64, lo=717, hi=717,
             window=0, e4m3=False),
        # a batch of 32 trees of up to 16 nodes, contexts from a few tokens to 8192, small pages
        dict(name="attn_batch32", op="attn", B=32, n=16, ragged=True, spread=6, Hq=32, Hkv=8, D=128, page=16, lo=60,
             hi=8192, window=0, e4m3=False),
        # 16 trees of up to 32 nodes over a long 8-bit cache
        dict(name="attn_e4m3", op="attn", B=16, n=32, ragged=True, spread=8, Hq=16, Hkv=2, D=256, page=64, lo=512,
             hi=32768, window=0, e4m3=True),
        # a sliding-window layer, trees of up to 12 nodes, three query heads a key head
        dict(name="attn_sliding", op="attn", B=48, n=12, ragged=True, spread=5, Hq=24, Hkv=8, D=64, page=32, lo=100,
             hi=16384, window=1000, e4m3=False),
        # four trees of 256 nodes: the widest
        dict(name="attn_tree256", op="attn", B=4, n=256, ragged=False, spread=32, Hq=32, Hkv=4, D=128, page=64, lo=4096,
             hi=16000, window=0, e4m3=False),
        # one request's chain of 5 drawn tokens, with the draft's probabilities: latency
        dict(name="verify_chain5", op="verify", B=1, n=6, ragged=False, spread=1, V=131072, drawn=True),
        # a batch of 64 trees of the draft's likeliest tokens, an odd vocabulary
        dict(name="verify_batch64", op="verify", B=64, n=16, ragged=True, spread=5, V=100001, drawn=False),
        # the kept nodes of 64 trees of 32, up to six a tree, in 24 layers
        dict(name="compact_batch64", op="compact", B=64, n=32, keep=6, layers=24, Hkv=8, D=128, page=16, e4m3=False),
        # copy-on-write of 96 pages of a beam or a shared prompt's ends, in 32 layers of an 8-bit cache
        dict(name="copy_96_pages", op="copy", pages=96, layers=32, Hkv=8, D=128, page=64, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "verify", "compact", "copy"])
    if op == "verify":
        n = _log(rng, 1, 64)
        V = _log(rng, 1000, 131072)
        B = max(1, min(_log(rng, 1, 64), 64 * 16 * 131072 // (n * V)))
        return dict(op="verify", B=B, n=n, ragged=rng.random() < 0.5, spread=rng.choice([1, 1, 3, 5, 8]), V=V,
                    drawn=rng.random() < 0.6)
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    e4m3 = rng.random() < 0.4
    if op == "compact":
        n = _log(rng, 2, 256)
        B, layers = _log(rng, 1, 64), _log(rng, 1, 48)
        while B * (n + 2 * page) * layers * Hkv * D > 64 * 64 * 24 * 8 * 128:
            B, layers = max(1, B // 2), max(1, layers // 2)
        return dict(op="compact", B=B, n=n, keep=rng.randint(1, max(1, min(n // 2, 12))), layers=layers, Hkv=Hkv, D=D,
                    page=page, e4m3=e4m3)
    if op == "copy":
        pages, layers = _log(rng, 1, 128), _log(rng, 1, 48)
        while pages * layers * Hkv * D * page > 96 * 32 * 8 * 128 * 64:
            pages, layers = max(1, pages // 2), max(1, layers // 2)
        return dict(op="copy", pages=pages, layers=layers, Hkv=Hkv, D=D, page=page, e4m3=e4m3)
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    spread = rng.choice([1, 3, 5, 8, 32])
    if op == "append":
        B = _log(rng, 1, 64)
        n = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, 256), _log(rng, 1, 4096)])
        if n > 256 or rng.random() < 0.3:
            spread = 0
        while B * n * (G + 1) * Hkv * D > 8192 * 36 * 128:
            B, n = max(1, B // 2), max(1, n // 2)
        hi = max(n, _log(rng, 16, 262144 if B * n <= 1024 else 8192))
        return dict(op="append", B=B, n=n, ragged=rng.random() < 0.5, spread=spread, Hq=G * Hkv, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.5, page=page, lo=max(n, hi // 8),
                    hi=hi, e4m3=e4m3)
    n = rng.choice([_log(rng, 1, 16), _log(rng, 2, 64), _log(rng, 16, 256)])
    B = _log(rng, 1, 48 if n <= 64 else 4)
    if n > 64:
        G, Hkv, D = min(G, 8), min(Hkv, 4), min(D, 128)
    hi = max(n, _log(rng, 16, 65536 if B == 1 and n <= 64 else 16384))
    while B * hi * Hkv * D > 48 * 1024 * 1024 or B * hi * n * G * Hkv > 512 * 1024 * 1024:
        if B == 1 and hi <= max(n, 64):
            break
        B, hi = max(1, B // 2), max(n, hi // 2)
    return dict(op="attn", B=B, n=n, ragged=rng.random() < 0.5, spread=spread, Hq=G * Hkv, Hkv=Hkv, D=D, page=page,
                lo=max(n, hi // 16), hi=hi, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), e4m3=e4m3)


# ------------------------------------------------- lengths and trees: part of the case, so that the work is too

def _trees(c):
    """Tokens of each request in the cache (its nodes included), its nodes, and their parents [B, n] (-1: none)."""
    B, n = c["B"], c["n"]
    hi, lo = c.get("hi", 4 * n + 8), c.get("lo", n + 4)
    r = np.random.RandomState(7919 * B + 31 * hi + n)
    lens = np.clip(np.rint(np.exp(r.uniform(math.log(lo), math.log(hi), B))).astype(np.int64), lo, hi)
    lens[0] = hi
    ns = np.full(B, n, dtype=np.int64)
    if c.get("ragged"):
        ns = r.randint(1, n + 1, B).astype(np.int64)
        ns[-1] = n
    ns = np.minimum(ns, lens)
    # a node's parent is one of the `spread` before it; spread 1 is a chain, 0 a prompt's tokens, with no tree
    i = np.arange(n)
    parent = i - 1 - np.floor(r.rand(B, n) * np.minimum(max(c.get("spread", 1), 1), np.maximum(i, 1))).astype(np.int64)
    parent[:, 0] = -1
    parent[i >= ns.reshape(-1, 1)] = -1
    return lens, ns, parent


def _above(parent, ns):
    """above[b, i, j]: node j is node i or one of its ancestors; depth [B, n]."""
    B, n = parent.shape
    above = np.zeros((B, n, n), dtype=bool)
    depth = np.zeros((B, n), dtype=np.int64)
    for i in range(n):
        up = parent[:, i]
        has = up >= 0
        above[has, i] = above[has, up[has]]
        depth[has, i] = depth[has, up[has]] + 1
        above[:, i, i] = True
    there = np.arange(n) < ns.reshape(-1, 1)
    return above & there.reshape(B, n, 1), depth


def _kept(c):
    """Kept nodes of each tree, [B, keep] with -1 past the count: the root, then nodes past the count, in order."""
    B, n, keep = c["B"], c["n"], c["keep"]
    r = np.random.RandomState(104729 + 17 * B + n)
    count = r.randint(1, keep + 1, B)
    count[0] = keep
    path = np.full((B, keep), -1, dtype=np.int64)
    path[:, 0] = 0
    for b in range(B):
        m = int(count[b])
        path[b, 1:m] = np.sort(r.permutation(np.arange(m, n))[:m - 1]) if n - m >= m - 1 else np.arange(1, m)
    return path, count.astype(np.int64)


def work(c):
    size = 1 if c.get("e4m3") else 2
    if c["op"] == "copy":
        moved = c["pages"] * c["layers"] * 2 * c["Hkv"] * c["D"] * c["page"] * size
        return {"bytes": 2 * moved, "flops": 0}
    if c["op"] == "compact":
        path, count = _kept(c)
        moves = int((path[:, 1:] > np.arange(1, path.shape[1])).sum())
        return {"bytes": 2 * moves * c["layers"] * 2 * c["Hkv"] * c["D"] * size + 8 * int(count.sum()), "flops": 0}
    lens, ns, parent = _trees(c)
    T = int(ns.sum())
    if c["op"] == "verify":  # the rows of the node that a walk ends at
        return {"bytes": c["B"] * c["V"] * 4 * (2 if c["drawn"] else 1), "flops": c["B"] * c["V"] * (4 if c["drawn"] else 2)}
    if c["op"] == "append":
        D = c["D"]
        return {"bytes": T * D * (4 * c["Hq"] + 2 * c["Hkv"] * (2 + size)), "flops": T * (c["Hq"] + c["Hkv"]) * (4 * D + 3 * c["rot"])}
    above, depth = _above(parent, ns)
    keys = rows = 0
    for b in range(c["B"]):
        m, base = int(ns[b]), int(lens[b] - ns[b])
        w = c["window"] or 1 << 30
        d = depth[b, :m]
        near = above[b, :m, :m] & (d.reshape(-1, 1) - d < w)
        keys += min(base, w - 1 - int(d.min())) + m
        rows += int(near.sum()) + int(np.minimum(base, np.maximum(w - 1 - d, 0)).sum())
    return {"bytes": keys * c["Hkv"] * 2 * c["D"] * size + 4 * T * c["Hq"] * c["D"], "flops": 4 * c["D"] * c["Hq"] * rows}


# ------------------------------------------------------------------ the inputs

def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    return {"verify": _verify_inputs, "compact": _pool_inputs, "copy": _pool_inputs}.get(c["op"], _cache_inputs)(c, seed, g)


def _pools(g, c, *lead):
    """Keys and values of [*lead, Hkv, page, D]."""
    shape = (*lead, c["Hkv"], c["page"], c["D"])
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    return (x * 30).to(torch.float8_e4m3fn) if c["e4m3"] else x.to(BF)


def _pool_inputs(c, seed, g):
    if c["op"] == "copy":
        kv = _pools(g, c, c["layers"], 2, 2 * c["pages"] + 1)
        order = np.random.RandomState(int(seed) % (1 << 31)).permutation(2 * c["pages"] + 1)
        return dict(c=c, kv=kv, src=_dev(order[:c["pages"]]), dst=_dev(order[c["pages"]:2 * c["pages"]]))
    B, n, page = c["B"], c["n"], c["page"]
    path, count = _kept(c)
    r = np.random.RandomState(int(seed) % (1 << 31))
    base = r.randint(0, 8 * page, B)
    lens = base + n
    per = -(-lens // page)
    first = base // page  # pages before the trees are not looked at
    table = np.full((B, int(per.max())), -1, dtype=np.int64)
    used = int((per - first).sum())
    kv = _pools(g, c, c["layers"], 2, B * (n // page + 2))
    order = r.permutation(B * (n // page + 2))[:used]
    slots = np.concatenate([np.arange(a, z) for a, z in zip(first, per)])
    table[np.repeat(np.arange(B), per - first), slots] = order
    return dict(c=c, kv=kv, table=_dev(table), lens=_dev(lens), start=_dev(np.arange(B + 1) * n), path=_dev(path),
                count=_dev(count), max_n=n, T=B * n)


def _verify_inputs(c, seed, g):
    B, n, V = c["B"], c["n"], c["V"]
    lens, ns, parent = _trees(c)
    T = int(ns.sum())
    start = np.concatenate([[0], np.cumsum(ns)])
    request, place = np.repeat(np.arange(B), ns), np.concatenate([np.arange(m) for m in ns])
    up = parent[request, place]
    # rank of a node among its parent's children, and the children of every node in their order
    rank = np.array([int((parent[b, :i] == parent[b, i]).sum()) for b, i in zip(request, place)])
    kids = np.full((B, n, int(rank.max()) + 1), -1, dtype=np.int64)
    inner = up >= 0
    kids[request[inner], up[inner], rank[inner]] = place[inner]
    logits = torch.randn(T, V, generator=g, device="cuda") * 2.5
    s = dict(c=c, T=T, B=B, max_n=int(ns.max()), target=torch.softmax(logits, 1), draft=None)
    q = torch.softmax(logits.add_(torch.randn(T, V, generator=g, device="cuda")), 1)
    del logits
    row = torch.from_numpy(start[request] + np.maximum(up, 0)).cuda()  # of the parent
    if c["drawn"]:  # drawn from the draft's probabilities
        total = q.cumsum(1, dtype=torch.float64)
        at = torch.rand(T, 1, generator=g, device="cuda", dtype=torch.float64) * total[row, -1:]
        token = torch.cat([torch.searchsorted(total[int(r)], a) for r, a in zip(row.cpu(), at)])
        s["draft"] = q
    else:           # its likeliest tokens, in their order
        most = torch.topk(q, min(V, kids.shape[2]), dim=1).indices
        token = most[row, torch.from_numpy(rank).cuda()]
    lost = token.clamp(max=V - 1)
    lost[_dev(place, torch.long) == 0] = -1  # the root is no drafted token
    s.update(token=lost.to(torch.int32), parent=_dev(up), u=torch.rand(T, generator=g, device="cuda"),
             u_last=torch.rand(B, generator=g, device="cuda"), start=_dev(start), lens=_dev(lens),
             table=torch.zeros(B, 1, dtype=torch.int32, device="cuda"), kids=_dev(kids, torch.long),
             depth=int(_above(parent, ns)[1].max()) + 1)
    return s


def _cache_inputs(c, seed, g):
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    lens, ns, parent = _trees(c)
    B, n, page, Hq, Hkv, D = c["B"], c["n"], c["page"], c["Hq"], c["Hkv"], c["D"]
    T = int(ns.sum())
    start = np.concatenate([[0], np.cumsum(ns)])
    request, place = np.repeat(np.arange(B), ns), np.concatenate([np.arange(m) for m in ns])
    per = -(-lens // page)
    first = (lens - ns) // page if c["op"] == "append" else np.zeros(B, dtype=np.int64)
    # an append looks at the new tokens' pages only: earlier ones are page 0
    table = np.full((B, int(per.max())), 0 if c["op"] == "append" else -1, dtype=np.int64)
    used = int((per - first).sum()) + 1
    slots = np.concatenate([np.arange(a, z) for a, z in zip(first, per)])
    table[np.repeat(np.arange(B), per - first), slots] = np.random.RandomState(int(seed) % (1 << 31)).permutation(used - 1) + 1
    # a few channels of the keys are large, as after a projection with a bias
    chan = torch.where(torch.rand(Hkv, 1, D, generator=g, device="cuda") < 0.03, 3.0, 0.0)
    kc, vc = normal(used, Hkv, page, D) + chan, normal(used, Hkv, page, D)
    ks, vs = (torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.02 for _ in range(2))
    if c["e4m3"]:
        shape = (1, Hkv, 1, 1)
        kc = (kc / ks.view(shape)).clamp(-448, 448).to(torch.float8_e4m3fn)
        vc = (vc / vs.view(shape)).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        kc, vc = kc.to(BF), vc.to(BF)
    s = dict(c=c, T=T, kc=kc, vc=vc, ks=ks if c["e4m3"] else None, vs=vs if c["e4m3"] else None, table=_dev(table),
             start=_dev(start), lens=_dev(lens), max_n=int(ns.max()), max_len=int(lens.max()), row=_dev(place, torch.long),
             request=_dev(request, torch.long), place=_dev((lens - ns)[request] + place, torch.long),
             base=_dev((lens - ns)[request], torch.long), parent=_dev(parent[request, place]))
    if c["op"] == "append":
        s["qkv"] = (normal(T, (Hq + 2 * Hkv) * D) * (0.5 + normal(T, 1).abs())).to(BF)  # the rows of a joint projection
        s["wq"], s["wk"] = ((1.0 + 0.2 * normal(D)).to(BF) for _ in range(2))
        s["freq"] = 1e4 ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])
        s["freq_dev"] = torch.from_numpy(s["freq"]).cuda()
    else:
        above, depth = _above(parent, ns)  # the plan of the step, which its layers share
        s["above"], s["depth"] = _dev(above, torch.bool), _dev(depth, torch.long)
        s["q"] = (1.5 * normal(T, Hq, D)).to(BF)
        # what no request has written yet is whatever the memory held
        last = table[np.arange(B), per - 1]
        junk = _dev(np.where(lens % page > 0, lens % page, page), torch.long).view(B, 1, 1, 1)
        tail = torch.arange(page, device="cuda").view(1, 1, page, 1) >= junk
        pages = torch.from_numpy(last).cuda()
        for pool in (kc, vc):
            raw = pool.view(torch.uint8 if c["e4m3"] else torch.int16)
            fill = 0x7F if c["e4m3"] else 0x7FC0
            raw[pages] = torch.where(tail, torch.full_like(raw[pages], fill), raw[pages])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles and outputs that a serving loop keeps
        from serving_router_top_gb300 import moe
        c = case
        s["moe"] = moe
        out = lambda *shape, dtype=torch.int32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        if c["op"] in ("compact", "copy"):
            s["layers"] = moe.KvLayers([moe.KvPages(kv[0], kv[1]) for kv in s["kv"]])
        if c["op"] != "copy":
            s["batch"] = moe.KvBatch(s["start"], s["lens"], s["table"], s["T"], s["max_n"])
        if c["op"] == "compact":
            s["new_len"] = out(c["B"])
        if c["op"] == "verify":
            s["desc"] = moe.verify_desc(s["target"], s["token"], s["parent"], s["u"], s["u_last"], draft=s["draft"])
            s["path"], s["count"], s["next"] = out(c["B"], s["depth"]), out(c["B"]), out(c["B"])
        if c["op"] in ("append", "attn"):
            s["pages"] = moe.KvPages(s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"])
            s["tree"] = moe.Tree(s["batch"], s["parent"]) if c["spread"] else None
            s["out"] = out(s["T"], c["Hq"], c["D"], dtype=BF)
        if c["op"] == "append":
            s["rope"] = moe.Rope(c["rot"], inv_freq=s["freq"], interleaved=c["interleaved"])
            s["norm"] = moe.HeadNorm(s["wq"], s["wk"], EPS)
            s["err"] = out(1).zero_()
        if c["op"] == "attn":
            moe.moe_tree_prepare(s["batch"], s["tree"])
            s["ws"] = moe.AttnWorkspace(c["Hq"], c["Hkv"], c["D"])
    return s


def _split(s):
    c = s["c"]
    return s["qkv"].view(s["T"], -1, c["D"]).split([c["Hq"], c["Hkv"], c["Hkv"]], 1)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["c"]["op"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "verify": _plain_verify, "compact": _plain_compact,
                "copy": _plain_copy}[op](s)
    moe, c = s["moe"], s["c"]
    if op == "append":
        q, k, v = _split(s)
        tree = s["tree"]
        if tree is not None:
            moe.moe_tree_prepare(s["batch"], tree, err=s["err"])
        moe.moe_kv_append_norm(s["pages"], s["batch"], s["rope"], s["norm"], q, s["out"], k, v, tree=tree, err=s["err"])
        return {"q": s["out"], "k": s["kc"], "v": s["vc"], **({} if tree is None else {"depth": tree.depth, "above": tree.above})}
    if op == "attn":
        moe.moe_tree_attention(s["pages"], s["batch"], s["tree"], s["q"], s["out"], s["ws"], scale=c["D"] ** -0.5,
                               window=c["window"])
        return s["out"]
    if op == "verify":
        moe.moe_verify_drafts(s["batch"], s["desc"], s["path"], s["count"], s["next"])
        return {"path": s["path"], "count": s["count"], "next": s["next"]}
    if op == "compact":
        moe.moe_kv_compact(s["layers"], s["batch"], s["path"], s["count"], s["new_len"])
        return {"kv": s["kv"], "len": s["new_len"]}
    moe.moe_kv_copy_pages(s["layers"], s["src"], s["dst"])
    return s["kv"]


def _words(bits):
    """[..., n] truth values as int32 words of 32, the first the lowest bit."""
    n = bits.shape[-1]
    x = torch.nn.functional.pad(bits, (0, -n % 32)).unflatten(-1, (-1, 32)).long()
    x = (x << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)


def _plain_tree(s):
    """Depth and ancestors of every row, from the parents."""
    B, n = s["c"]["B"], s["max_n"]
    step = torch.zeros(B, n, n, device="cuda")
    step[s["request"], s["row"], s["row"]] = 1.0
    inner = s["parent"] >= 0
    step[s["request"][inner], s["row"][inner], s["parent"][inner].long()] = 1.0
    for _ in range(max(n - 1, 1).bit_length()):  # the ways of up to 2, 4, 8 .. steps
        step = (step @ step).clamp(max=1.0)
    above = step[s["request"], s["row"]] > 0
    return above.sum(1).to(torch.int32) - 1, above


def _plain_append(s):
    c = s["c"]
    rot = c["rot"]
    q, k, v = _split(s)
    tree = c["spread"] > 0
    if tree:
        depth, above = _plain_tree(s)
    position = s["base"] + depth if tree else s["place"]
    angle = position.double().view(-1, 1, 1) * s["freq_dev"]
    cos, sin = angle.cos().float(), angle.sin().float()

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    page = s["table"][s["request"], s["place"] // c["page"]].long()
    at = s["place"] % c["page"]
    k, v = turned(k, s["wk"]), v.float()
    if c["e4m3"]:
        k = (k / s["ks"].view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / s["vs"].view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kc"].view(torch.uint8)[page, :, at] = k
        s["vc"].view(torch.uint8)[page, :, at] = v
    else:
        s["kc"][page, :, at] = k.to(BF)
        s["vc"][page, :, at] = v.to(BF)
    return {"q": turned(q, s["wq"]).to(BF), "k": s["kc"], "v": s["vc"],
            **({"depth": depth, "above": _words(above)} if tree else {})}


def _plain_attn(s):
    c = s["c"]
    B, Hkv, D, G, n = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], s["max_n"]
    j = torch.arange(s["max_len"], device="cuda")
    there = j < s["lens"].view(B, 1)                                   # [B, L]
    page = s["table"][:, (j // c["page"]).clamp(max=s["table"].shape[1] - 1)].clamp(min=0).long()

    def rows(pool, scale):
        x = pool.view(torch.uint8)[page, :, j % c["page"]].view(torch.float8_e4m3fn) if c["e4m3"] else pool[page, :, j % c["page"]]
        x = x.float() if scale is None else x.float() * scale.view(-1, 1)
        return torch.where(there.view(B, -1, 1, 1), x, 0.0).transpose(1, 2)  # [B, Hkv, L, D]

    q = torch.zeros(B, n, Hkv, G, D, device="cuda")
    q[s["request"], s["row"]] = s["q"].float().view(-1, Hkv, G, D)
    base = s["lens"].long() - s["start"].diff()
    node = j - base.view(B, 1)                                         # [B, L]: which node a key is, < 0 none
    inside = node.clamp(0, n - 1).view(B, 1, -1).expand(B, n, -1)
    seen = torch.where(node.view(B, 1, -1) < 0, True, s["above"][:, :n, :n].gather(2, inside)) & there.view(B, 1, -1)
    if c["window"]:
        at = (base.view(B, 1) + s["depth"][:, :n]).unsqueeze(2)        # positions of the rows and of the keys
        where = torch.where(node < 0, j, base.view(B, 1) + s["depth"].gather(1, node.clamp(0, n - 1))).unsqueeze(1)
        seen &= where > at - c["window"]
    score = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D) @ rows(s["kc"], s["ks"]).transpose(2, 3)
    score = (score * D ** -0.5).view(B, Hkv, G, n, -1).masked_fill(~seen.view(B, 1, 1, n, -1), float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, G * n, -1) @ rows(s["vc"], s["vs"])
    o = o.view(B, Hkv, G, n, D) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4)[s["request"], s["row"]].reshape(-1, c["Hq"], D).to(BF)


def _plain_verify(s):
    B, V = s["B"], s["c"]["V"]
    all_b = torch.arange(B, device="cuda")
    node, last = (torch.zeros(B, dtype=torch.long, device="cuda") for _ in range(2))
    alive = torch.ones(B, dtype=torch.bool, device="cuda")
    path = torch.full((B, s["depth"]), -1, dtype=torch.int32, device="cuda")
    left = torch.zeros(B, V, dtype=torch.float64, device="cuda")       # what the last token is drawn from
    for level in range(s["depth"]):
        path[:, level] = torch.where(alive, node, -1)
        row = s["start"][:-1] + node
        rest = s["target"][row].double()
        q = None if s["draft"] is None else s["draft"][row].double()
        sigma = torch.ones(B, dtype=torch.float64, device="cuda")
        moved = torch.zeros_like(alive)
        to = node
        for k in range(s["kids"].shape[2]):
            child = s["kids"][all_b, node, k]
            tried = alive & ~moved & (child >= 0)
            at = s["start"][:-1] + child.clamp(min=0)
            x = s["token"][at].clamp(min=0).long()
            r = rest[all_b, x]
            qx = 1.0 if q is None else q[all_b, x]
            taken = tried & (s["u"][at].double() * qx * sigma < r)
            refused = tried & ~taken
            if q is None:
                less, total = rest.scatter(1, x.unsqueeze(1), 0.0), sigma - r
            else:
                less = (rest - sigma.unsqueeze(1) * q).clamp(min=0.0)
                total = less.sum(1)
            rest = torch.where(refused.unsqueeze(1), less, rest)
            sigma = torch.where(refused, total, sigma)
            to = torch.where(taken, child, to)
            moved = moved | taken
        left = torch.where((alive & ~moved).unsqueeze(1), rest, left)
        last = torch.where(alive & ~moved, node, last)
        alive, node = moved, to
    left = torch.where(left.sum(1, keepdim=True) > 0, left, s["target"][s["start"][:-1] + last].double())
    run_up = left.cumsum(1)
    found = run_up > s["u_last"].double().unsqueeze(1) * run_up[:, -1:]
    token = torch.where(run_up[:, -1] > 0, found.to(torch.uint8).argmax(1), -1)
    return {"path": path, "count": (path >= 0).sum(1).to(torch.int32), "next": token.to(torch.int32)}


def _plain_compact(s):
    c = s["c"]
    page = c["page"]
    b, d = (s["path"] >= 0).nonzero(as_tuple=True)
    base = (s["lens"] - s["start"].diff()).long()
    raw = s["kv"].view(torch.uint8) if c["e4m3"] else s["kv"]
    old, new = base[b] + s["path"][b, d], base[b] + d
    where = lambda p: s["table"][b, p // page].long()  # noqa: E731
    raw[:, :, where(new), :, new % page] = raw[:, :, where(old), :, old % page]
    return {"kv": s["kv"], "len": (base + s["count"]).to(torch.int32)}


def _plain_copy(s):
    raw = s["kv"].view(torch.uint8) if s["c"]["e4m3"] else s["kv"]
    raw[:, :, s["dst"].long()] = raw[:, :, s["src"].long()]
    return s["kv"]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "verify": _exact_verify, "compact": _exact_compact,
            "copy": _exact_copy}[case["op"]](case, s)


def _exact_append(c, s):
    lens, ns, parent = _trees(c)
    table = s["table"].cpu().numpy()
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    qkv = s["qkv"].double().view(s["T"], Hq + 2 * Hkv, D).clone()
    for heads, w in ((slice(0, Hq), s["wq"]), (slice(Hq, Hq + Hkv), s["wk"])):
        x = qkv[:, heads]
        qkv[:, heads] = w.double() * x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt()
    out, pos, ids, places = {}, [], [], []
    chains = []
    for b in range(c["B"]):
        base = int(lens[b] - ns[b])
        up = []
        for i in range(int(ns[b])):  # the node and those above it
            up.append(([] if not c["spread"] or parent[b, i] < 0 else up[parent[b, i]]) + [i])
            pos.append(base + (len(up[-1]) - 1 if c["spread"] else i))
            ids.append(table[b, (base + i) // page])
            places.append((base + i) % page)
        chains += up
    pos = torch.tensor(pos, dtype=torch.float64, device="cuda")
    pairs = c["rot"] // 2
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + pairs)
        turn = torch.polar(torch.ones_like(pos), pos * float(s["freq"][i])).view(-1, 1)
        z = torch.complex(qkv[:, :Hq + Hkv, a], qkv[:, :Hq + Hkv, b]) * turn
        qkv[:, :Hq + Hkv, a], qkv[:, :Hq + Hkv, b] = z.real, z.imag
    k, v = s["kc"].double(), s["vc"].double()
    kn, vn = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if c["e4m3"]:
        kn = (kn / s["ks"].double().view(1, -1, 1)).clamp(-448, 448)
        vn = (vn / s["vs"].double().view(1, -1, 1)).clamp(-448, 448)
    ids, places = torch.tensor(ids, dtype=torch.long, device="cuda"), torch.tensor(places, device="cuda")
    k[ids, :, places], v[ids, :, places] = kn, vn
    out.update(q=qkv[:, :Hq].contiguous(), k=k, v=v)
    if c["spread"]:
        words = -(-int(ns.max()) // 32)
        bits = np.zeros((s["T"], words), dtype=np.uint32)
        for t, chain in enumerate(chains):
            for i in chain:
                bits[t, i // 32] |= np.uint32(1 << i % 32)
        out.update(depth=torch.tensor([len(x) - 1 for x in chains], dtype=torch.int32), above=torch.from_numpy(bits.view(np.int32)))
    return out


def _exact_attn(c, s):
    lens, ns, parent = _trees(c)
    table = s["table"].cpu().numpy()
    start = np.concatenate([[0], np.cumsum(ns)])
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        L, m = int(lens[b]), int(ns[b])
        base = L - m
        hidden = np.zeros((m, L), dtype=bool)
        chains = []
        for i in range(m):
            chains.append(([] if parent[b, i] < 0 else chains[parent[b, i]]) + [i])
            hidden[i, base:] = True
            hidden[i, base + np.array(chains[i])] = False
        if c["window"]:
            position = np.concatenate([np.arange(base), base + np.array([len(x) - 1 for x in chains])])
            hidden |= position <= position[base:].reshape(-1, 1) - c["window"]
        first = int(np.argmin(hidden.all(0)))  # keys that no row sees are not read
        hidden = torch.from_numpy(hidden[:, first:]).cuda().view(m, 1, L - first)
        ids = torch.from_numpy(table[b, first // page:-(-L // page)].astype(np.int64)).cuda()
        skip = first - first // page * page
        for h in range(Hkv):
            k = s["kc"][:, h].view(torch.uint8 if c["e4m3"] else torch.int16)[ids].view(s["kc"].dtype)
            v = s["vc"][:, h].view(torch.uint8 if c["e4m3"] else torch.int16)[ids].view(s["vc"].dtype)
            k, v = (x.double().reshape(-1, D)[skip:skip + L - first] for x in (k, v))
            if c["e4m3"]:
                k, v = k * float(s["ks"][h]), v * float(s["vs"][h])
            mine = slice(int(start[b]), int(start[b + 1]))
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            score = torch.einsum("thd,jd->thj", s["q"][mine, heads].double(), k) / math.sqrt(D)
            w = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out[mine, heads] = torch.einsum("thj,jd->thd", w, v)
    return out


def _exact_verify(c, s):
    lens, ns, parent = _trees(c)
    start = np.concatenate([[0], np.cumsum(ns)])
    token, u, u_last = (s[k].cpu().numpy() for k in ("token", "u", "u_last"))
    path = np.full((c["B"], s["depth"]), -1, dtype=np.int32)
    nxt = np.full(c["B"], -1, dtype=np.int32)
    row = lambda which, t: s[which][t].double().cpu().numpy()  # noqa: E731
    for b in range(c["B"]):
        v, at = 0, 0
        while True:
            path[b, at] = v
            t0 = int(start[b])
            p = row("target", t0 + v)
            rest, sigma, kept = p.copy(), 1.0, None
            children = [i for i in range(1, int(ns[b])) if parent[b, i] == v]
            q = row("draft", t0 + v) if children and s["draft"] is not None else None
            for i in children:
                x = int(token[t0 + i])
                odds = 1.0 if q is None else float(q[x])
                if float(u[t0 + i]) * odds * sigma < rest[x]:
                    kept = i
                    break
                if q is None:
                    sigma -= float(rest[x])
                    rest[x] = 0.0
                else:
                    rest = np.maximum(rest - sigma * q, 0.0)
                    sigma = math.fsum(rest)
            if kept is None:
                break
            v, at = kept, at + 1
        if not rest.any():
            rest = p
        total = np.cumsum(rest)
        if total[-1] > 0:
            nxt[b] = int(np.searchsorted(total, float(u_last[b]) * total[-1], side="right"))
    return {"path": path, "count": (path >= 0).sum(1).astype(np.int32), "next": nxt}


def _exact_compact(c, s):
    path, count = _kept(c)
    kv = s["kv"].double()
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    for b in range(c["B"]):
        base = int(lens[b]) - c["n"]
        for d in range(int(count[b])):
            old, new = base + int(path[b, d]), base + d
            kv[:, :, int(table[b, new // c["page"]]), :, new % c["page"]] = kv[:, :, int(table[b, old // c["page"]]), :, old % c["page"]].clone()
    return {"kv": kv, "len": (lens - c["n"] + count).astype(np.int32)}


def _exact_copy(c, s):
    kv = s["kv"].double()
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        kv[:, :, z] = s["kv"][:, :, a].double()
    return kv

"""The attention half of a decoder layer beside the MoE layer, measured operator by operator.

Three operators over the state a serving loop keeps (a paged key-value cache, its
page tables, an fp32 residual stream):

* ``append``: rotate the new tokens' queries and keys by their positions and write
  keys and values into the cache's pages (bf16 or E4M3).
* ``attn``: attention of each request's newest tokens over its pages.
* ``norm``: the norm after a block with its gate and residual scale, the residual
  add, and the norm before the next block.

``run`` computes them in plain torch where ``own`` is false, and through the
package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one request's verify window of 4 tokens behind a hidden-2048 layer: latency
        dict(name="append_verify4", op="append", B=1, n=4, ragged=False, Hq=16, Hkv=2, D=256, rot=64, interleaved=False,
             page=64, lo=1021, hi=1021, e4m3=False),
        # a batch-64 decode step of far positions into an 8-bit cache
        dict(name="append_batch64_e4m3", op="append", B=64, n=1, ragged=False, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=True, page=16, lo=5, hi=262144, e4m3=True),
        # a prompt chunk of 8192 tokens
        dict(name="append_prefill8192", op="append", B=2, n=4096, ragged=False, Hq=32, Hkv=4, D=128, rot=128,
             interleaved=False, page=64, lo=4096, hi=9001, e4m3=False),
        # the same verify window's attention over a short context: latency
        dict(name="attn_verify4", op="attn", B=1, n=4, ragged=False, Hq=16, Hkv=2, D=256, page=64, lo=717, hi=717,
             window=0, e4m3=False),
        # one new token of one request over a long context: the split over the length
        dict(name="attn_one_long", op="attn", B=1, n=1, ragged=False, Hq=32, Hkv=4, D=128, page=64, lo=131071, hi=131071,
             window=0, e4m3=False),
        # a batch-64 decode step, contexts from a few tokens to 8192, small pages
        dict(name="attn_batch64", op="attn", B=64, n=1, ragged=False, Hq=32, Hkv=8, D=128, page=16, lo=3, hi=8192,
             window=0, e4m3=False),
        # 16 requests' verify windows over an 8-bit cache
        dict(name="attn_verify_e4m3", op="attn", B=16, n=4, ragged=True, Hq=16, Hkv=2, D=256, page=64, lo=512, hi=32768,
             window=0, e4m3=True),
        # a sliding-window layer, three query heads a key head
        dict(name="attn_sliding", op="attn", B=48, n=1, ragged=False, Hq=24, Hkv=8, D=64, page=32, lo=100, hi=16384,
             window=1000, e4m3=False),
        # two prompt chunks behind their own earlier tokens
        dict(name="attn_chunk", op="attn", B=2, n=512, ragged=True, Hq=32, Hkv=4, D=128, page=64, lo=2048, hi=6000,
             window=0, e4m3=False),
        # between two blocks of a verify window: latency
        dict(name="norm_verify4", op="norm", T=4, H=2048, post=True, gate="none", scale=1.0),
        # batch-64 decode at hidden 4096 with a gate per token and channel
        dict(name="norm_batch64", op="norm", T=64, H=4096, post=False, gate="sigmoid", scale=0.5),
        # a prompt chunk of 8192 tokens with one gate row for every token
        dict(name="norm_prefill8192", op="norm", T=8192, H=2048, post=True, gate="row", scale=0.7071),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "norm"])
    if op == "norm":
        T = _log(rng, 1, 8192)
        H = rng.choice([_log(rng, 64, 4096), 8 * _log(rng, 8, 512), 2048, 4096])
        while T * H > 8192 * 2048:
            T //= 2
        return dict(op="norm", T=T, H=H, post=rng.random() < 0.6, gate=rng.choice(["none", "row", "sigmoid", "token"]),
                    scale=rng.choice([1.0, 0.5, 0.7071]))
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    e4m3 = rng.random() < 0.4
    if op == "append":
        B = _log(rng, 1, 64)
        n = rng.choice([1, 1, 4, _log(rng, 1, 4096)])
        while B * n * (G + 1) * Hkv * D > 8192 * 36 * 128:
            B, n = max(1, B // 2), max(1, n // 2)
        hi = max(n, _log(rng, 16, 262144 if B * n <= 256 else 8192))
        return dict(op="append", B=B, n=n, ragged=rng.random() < 0.5, Hq=G * Hkv, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.5, page=page,
                    lo=max(n, hi // 8), hi=hi, e4m3=e4m3)
    B = _log(rng, 1, 64)
    n = rng.choice([1, 1, 1, 2, 4, _log(rng, 1, 16), _log(rng, 16, 512)])
    if n > 16:
        B = min(B, 2)
    hi = max(n, _log(rng, 16, 131072 if B == 1 and n <= 16 else 16384 if n <= 16 else 6000))
    while B * hi * Hkv * D > 64 * 1024 * 1024:
        hi = max(n, hi // 2)
        B = max(1, B // 2)
    if n > 16:
        G = min(G, 8)
        Hkv = min(Hkv, 4)
        D = min(D, 128)
    return dict(op="attn", B=B, n=n, ragged=rng.random() < 0.5, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, lo=max(n, hi // 16),
                hi=hi, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), e4m3=e4m3)


def _lengths(c):
    """Tokens of each request in the cache (its new ones included) and its new ones: part of the
    case, so that the work does not depend on the seed."""
    r = np.random.RandomState(7919 * c["B"] + 31 * c["hi"] + c["n"])
    lens = np.exp(r.uniform(math.log(c["lo"]), math.log(c["hi"]), c["B"]))
    lens = np.clip(np.rint(lens).astype(np.int64), c["lo"], c["hi"])
    lens[0] = c["hi"]
    n = np.full(c["B"], c["n"], dtype=np.int64)
    if c["ragged"]:
        n = r.randint(1, c["n"] + 1, c["B"]).astype(np.int64)
        n[-1] = c["n"]
    n = np.minimum(n, lens)  # a request has at least its new tokens
    return lens, n


def work(c):
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        gate = {"none": 0, "row": 2 * H}.get(c["gate"], 2 * T * H)
        return {"bytes": T * H * (4 + 4 + 2 + 2) + gate + 2 * H * (2 if c["post"] else 1), "flops": 8 * T * H}
    lens, n = _lengths(c)
    T, size = int(n.sum()), 1 if c["e4m3"] else 2
    if c["op"] == "append":
        return {"bytes": T * c["D"] * (4 * c["Hq"] + 2 * c["Hkv"] * (2 + size)),
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    keys = rows = 0
    for L, m in zip(lens.tolist(), n.tolist()):
        w = c["window"] or L
        keys += min(L, w + m - 1)
        rows += sum(min(p + 1, w) for p in range(L - m, L))
    return {"bytes": keys * c["Hkv"] * 2 * c["D"] * size + 4 * T * c["Hq"] * c["D"], "flops": 4 * c["D"] * c["Hq"] * rows}


# ------------------------------------------------------------------ the inputs

def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s = dict(c=c, x=normal(T, H) * (1.0 + 2.0 * normal(1, H).abs()), y=(normal(T, H) * 0.7).to(bf),
                 w_post=(1.0 + 0.1 * normal(H)).to(bf), w_pre=(1.0 + 0.1 * normal(H)).to(bf), gate=None,
                 x_out=torch.empty(T, H, device="cuda"), xn=torch.empty(T, H, dtype=bf, device="cuda"))
        if c["gate"] == "row":
            s["gate"] = (0.3 * normal(1, H)).to(bf)
        elif c["gate"] != "none":
            s["gate"] = normal(T, H).to(bf)
        return s
    lens, n = _lengths(c)
    B, page, Hq, Hkv, D = c["B"], c["page"], c["Hq"], c["Hkv"], c["D"]
    T = int(n.sum())
    start = np.concatenate([[0], np.cumsum(n)])
    per = -(-lens // page)
    width = int(per.max())
    if c["op"] == "append":  # only the pages that the new tokens fall into are held; earlier ones are page 0
        first = (lens - n) // page
        table, used = np.zeros((B, width), dtype=np.int32), int((per - first).sum()) + 1
    else:
        first = np.zeros(B, dtype=np.int64)
        table, used = np.full((B, width), -1, dtype=np.int32), int(per.sum()) + 1
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(used - 1) + 1
    at = 0
    for b in range(B):
        m = int(per[b] - first[b])
        table[b, first[b]:per[b]] = order[at:at + m]
        at += m
    # a few channels of the keys are large, as after a projection with a bias
    chan = torch.where(torch.rand(Hkv, 1, D, generator=g, device="cuda") < 0.03, 3.0, 0.0)
    kc, vc = normal(used, Hkv, page, D) + chan, normal(used, Hkv, page, D)
    ks, vs = (torch.rand(Hkv, generator=g, device="cuda") * 0.02 + 0.02 for _ in range(2))
    if c["e4m3"]:
        shape = (1, Hkv, 1, 1)
        kc = (kc / ks.view(shape)).clamp(-448, 448).to(torch.float8_e4m3fn)
        vc = (vc / vs.view(shape)).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        kc, vc = kc.to(bf), vc.to(bf)
    s = dict(c=c, T=T, kc=kc, vc=vc, ks=ks if c["e4m3"] else None, vs=vs if c["e4m3"] else None,
             table=torch.from_numpy(table).cuda(), start=torch.from_numpy(start.astype(np.int32)).cuda(),
             lens=torch.from_numpy(lens.astype(np.int32)).cuda(), max_n=int(n.max()), max_len=int(lens.max()),
             request=torch.from_numpy(np.repeat(np.arange(B), n)).cuda(),
             place=torch.from_numpy(np.concatenate([np.arange(m) for m in n])).cuda(),
             position=torch.from_numpy(np.concatenate([np.arange(l - m, l) for l, m in zip(lens, n)])).cuda())
    if c["op"] == "append":
        s["qkv"] = normal(T, (Hq + 2 * Hkv) * D).to(bf)  # the rows of a joint projection
        s["freq"] = 1e4 ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / c["rot"])
        s["freq_dev"] = torch.from_numpy(s["freq"]).cuda()
    else:
        s["q"] = (1.5 * normal(T, Hq, D)).to(bf)
        # what no request has written yet is whatever the memory held
        last = table[np.arange(B), per - 1].astype(np.int64)
        junk = torch.from_numpy(np.where(lens % page > 0, lens % page, page)).cuda().view(B, 1, 1, 1)
        tail = torch.arange(page, device="cuda").view(1, 1, page, 1) >= junk
        for pool in (kc, vc):
            raw = pool.view(torch.uint8 if c["e4m3"] else torch.int16)
            fill = 0x7F if c["e4m3"] else 0x7FC0
            pages = torch.from_numpy(last).cuda()
            raw[pages] = torch.where(tail, torch.full_like(raw[pages], fill), raw[pages])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles that a serving loop keeps
        from serving_router_top_gb300 import moe
        c = case
        s["moe"] = moe
        if c["op"] == "norm":
            s["desc"] = moe.block_norm_desc(y=s["y"], post_norm=c["post"], w_post=s["w_post"], gate=s["gate"],
                                            gate_sigmoid=c["gate"] == "sigmoid", res_scale=c["scale"], w_pre=s["w_pre"],
                                            eps=EPS)
        else:
            s["pages"] = moe.KvPages(s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"])
            s["batch"] = moe.KvBatch(s["start"], s["lens"], s["table"], s["T"], s["max_n"])
            if c["op"] == "append":
                s["rope"] = moe.Rope(c["rot"], inv_freq=s["freq"], interleaved=c["interleaved"])
                s["q_out"] = torch.empty(s["T"], c["Hq"], c["D"], dtype=torch.bfloat16, device="cuda")
                s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            else:
                s["ws"] = moe.AttnWorkspace(c["Hq"], c["Hkv"], c["D"])
                s["o"] = torch.empty(s["T"], c["Hq"], c["D"], dtype=torch.bfloat16, device="cuda")
    return s


def _split(s):
    c = s["c"]
    return s["qkv"].view(s["T"], -1, c["D"]).split([c["Hq"], c["Hkv"], c["Hkv"]], 1)


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    if c["op"] == "norm":
        if not own:
            return _plain_norm(s)
        s["moe"].moe_block_norm(s["desc"], s["x"], s["x_out"], s["xn"], c["T"], c["H"])
        return {"x": s["x_out"], "xn": s["xn"]}
    if c["op"] == "append":
        if not own:
            return _plain_append(s)
        q, k, v = _split(s)
        s["moe"].moe_kv_append(s["pages"], s["batch"], s["rope"], q, s["q_out"], k, v, err=s["err"])
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
    if not own:
        return _plain_attn(s)
    s["moe"].moe_paged_attention(s["pages"], s["batch"], s["q"], s["o"], s["ws"], scale=c["D"] ** -0.5, window=c["window"])
    return s["o"]


def _plain_norm(s):
    c = s["c"]
    z = s["y"].float()
    if c["post"]:
        z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        z = z * (torch.sigmoid(s["gate"].float()) if c["gate"] == "sigmoid" else s["gate"].float())
    x = s["x"] + c["scale"] * z
    xn = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    return {"x": x, "xn": xn.to(torch.bfloat16)}


def _plain_append(s):
    c = s["c"]
    rot = c["rot"]
    q, k, v = _split(s)
    angle = s["position"].double().view(-1, 1, 1) * s["freq_dev"]
    cos, sin = angle.cos().float(), angle.sin().float()

    def turned(x):
        x = x.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    page = s["table"][s["request"], s["position"] // c["page"]].long()
    at = s["position"] % c["page"]
    k, v = turned(k), v.float()
    if c["e4m3"]:
        k = (k / s["ks"].view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / s["vs"].view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kc"].view(torch.uint8)[page, :, at] = k
        s["vc"].view(torch.uint8)[page, :, at] = v
    else:
        s["kc"][page, :, at] = k.to(torch.bfloat16)
        s["vc"][page, :, at] = v.to(torch.bfloat16)
    return {"q": turned(q).to(torch.bfloat16), "k": s["kc"], "v": s["vc"]}


def _plain_attn(s):
    c = s["c"]
    B, Hkv, D, G, n = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], s["max_n"]
    j = torch.arange(s["max_len"], device="cuda")
    there = j < s["lens"].view(B, 1)                                   # [B, L]
    page = s["table"][:, j // c["page"]].clamp(min=0).long()           # [B, L]

    def rows(pool, scale):
        x = pool.view(torch.uint8)[page, :, j % c["page"]].view(torch.float8_e4m3fn) if c["e4m3"] else pool[page, :, j % c["page"]]
        x = x.float() if scale is None else x.float() * scale.view(-1, 1)
        return torch.where(there.view(B, -1, 1, 1), x, 0.0).transpose(1, 2)  # [B, Hkv, L, D]

    q = torch.zeros(B, n, Hkv, G, D, device="cuda")
    q[s["request"], s["place"]] = s["q"].float().view(-1, Hkv, G, D)
    at = torch.full((B, n), -1, device="cuda", dtype=torch.long)
    at[s["request"], s["place"]] = s["position"]
    seen = j <= at.unsqueeze(2)
    if c["window"]:
        seen &= j > at.unsqueeze(2) - c["window"]                      # [B, n, L]
    score = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D) @ rows(s["kc"], s["ks"]).transpose(2, 3)
    score = (score * D ** -0.5).view(B, Hkv, G, n, -1).masked_fill(~seen.view(B, 1, 1, n, -1), float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, G * n, -1) @ rows(s["vc"], s["vs"])
    o = o.view(B, Hkv, G, n, D) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4)[s["request"], s["place"]].reshape(-1, c["Hq"], D).to(torch.bfloat16)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        x, y = s["x"].double(), s["y"].double()
        if case["post"]:
            y = s["w_post"].double() * y / ((y ** 2).sum(1, keepdim=True) / case["H"] + EPS).sqrt()
        if case["gate"] != "none":
            g = s["gate"].double()
            y = y * (1.0 / (1.0 + (-g).exp()) if case["gate"] == "sigmoid" else g)
        x = x + case["scale"] * y
        return {"x": x, "xn": s["w_pre"].double() * x / ((x ** 2).sum(1, keepdim=True) / case["H"] + EPS).sqrt()}
    lens, n = _lengths(case)
    table = s["table"].cpu().numpy()
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    start = np.concatenate([[0], np.cumsum(n)])
    if case["op"] == "append":
        qkv = s["qkv"].double().view(s["T"], Hq + 2 * Hkv, D).clone()
        pos = torch.cat([torch.arange(l - m, l, dtype=torch.float64) for l, m in zip(lens.tolist(), n.tolist())]).cuda()
        pairs = case["rot"] // 2
        for i in range(pairs):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
            turn = torch.polar(torch.ones_like(pos), pos * float(s["freq"][i])).view(-1, 1)
            z = torch.complex(qkv[:, :Hq + Hkv, a], qkv[:, :Hq + Hkv, b]) * turn
            qkv[:, :Hq + Hkv, a], qkv[:, :Hq + Hkv, b] = z.real, z.imag
        k, v = s["kc"].double(), s["vc"].double()
        kn, vn = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if case["e4m3"]:
            kn = (kn / s["ks"].double().view(1, -1, 1)).clamp(-448, 448)
            vn = (vn / s["vs"].double().view(1, -1, 1)).clamp(-448, 448)
        ids, places = [], []
        for b in range(case["B"]):
            p = np.arange(lens[b] - n[b], lens[b])
            ids.append(table[b, p // page])
            places.append(p % page)
        ids = torch.from_numpy(np.concatenate(ids).astype(np.int64)).cuda()
        places = torch.from_numpy(np.concatenate(places)).cuda()
        k[ids, :, places], v[ids, :, places] = kn, vn
        return {"q": qkv[:, :Hq].contiguous(), "k": k, "v": v}
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        L, m = int(lens[b]), int(n[b])
        first = max(0, L - m + 1 - case["window"]) if case["window"] else 0
        ids = torch.from_numpy(table[b, first // page:-(-L // page)].astype(np.int64)).cuda()
        skip = first - first // page * page
        for h in range(Hkv):
            k = s["kc"][:, h].view(torch.uint8 if case["e4m3"] else torch.int16)[ids].view(s["kc"].dtype)
            v = s["vc"][:, h].view(torch.uint8 if case["e4m3"] else torch.int16)[ids].view(s["vc"].dtype)
            k, v = (x.double().reshape(-1, D)[skip:skip + L - first] for x in (k, v))
            if case["e4m3"]:
                k, v = k * float(s["ks"][h]), v * float(s["vs"][h])
            mine = slice(int(start[b]), int(start[b + 1]))
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            score = torch.einsum("thd,jd->thj", s["q"][mine, heads].double(), k) / math.sqrt(D)
            at = torch.arange(L - m, L, device="cuda").view(-1, 1, 1)
            j = torch.arange(first, L, device="cuda")
            hidden = (j > at) | (j <= at - case["window"]) if case["window"] else j > at
            w = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out[mine, heads] = torch.einsum("thj,jd->thd", w, v)
    return out

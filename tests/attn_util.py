"""Inputs and 64-bit references for the attention half of a layer (paged cache, norms)."""
import numpy as np
import torch

from serving_router_top_gb300 import moe

U_BF16 = torch.finfo(torch.bfloat16).eps / 2  # one rounding to bf16
U_F32 = torch.finfo(torch.float32).eps / 2
U_E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2
E4M3_STEP = 2.0 ** -9  # between subnormals


class Paged:
    """A cache of `lens` tokens per request in shuffled pages, the last ns[b] of them new.

    Pools hold junk wherever no request's token lies.  layout "hnd": [page][head][place][D];
    "nhd": [page][place][head][D]; "kv": keys and values of a page side by side."""

    def __init__(self, lens, ns, Hkv, D, page, e4m3=False, layout="hnd", seed=0, lead=0, tail=0, table_extra=2,
                 junk=float("nan"), k_std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.ns, self.Hkv, self.D, self.page, self.e4m3 = list(lens), list(ns), Hkv, D, page, e4m3
        self.B, self.lead = len(lens), lead
        self.T = lead + sum(ns) + tail
        self.start = np.concatenate([[lead], lead + np.cumsum(ns)]).astype(np.int32)
        per = [-(-max(n, 0) // page) for n in lens]
        self.width = max(per + [0]) + table_extra
        npages = sum(per) + 3
        order = torch.randperm(npages - 1, generator=g).numpy() + 1  # page 0 belongs to nobody
        table = np.full((self.B, self.width), -1, dtype=np.int32)
        at = 0
        for b in range(self.B):
            table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
        self.table = table
        dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        shape = {"hnd": (npages, Hkv, page, D), "nhd": (npages, page, Hkv, D), "kv": (npages, 2, Hkv, page, D)}[layout]

        def pool():
            x = (torch.randn(shape, generator=g) * k_std).to(dt)
            return x.permute(0, 2, 1, 3) if layout == "nhd" else x

        if layout == "kv":
            both = pool()
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = pool(), pool()
        self.k_scale = self.v_scale = None
        if e4m3:
            self.k_scale = torch.rand(Hkv, generator=g) * 0.5 + 0.75
            self.v_scale = torch.rand(Hkv, generator=g) * 0.5 + 0.75
        mine = torch.zeros(npages, page, dtype=torch.bool)
        for b in range(self.B):
            for j0 in range(per[b]):
                mine[int(table[b, j0]), :min(page, lens[b] - j0 * page)] = True
        self.mine = mine
        bits = 0x7F if junk != junk else None
        for p in (self.k, self.v):
            if e4m3:
                raw = p.view(torch.uint8)
                raw.masked_fill_(~mine.view(npages, 1, page, 1), 0x7F if bits else 0x7E)
            else:
                p.masked_fill_(~mine.view(npages, 1, page, 1), junk)

    def positions(self):
        return [list(range(l - n, l)) for l, n in zip(self.lens, self.ns)]

    def rows(self, which, b, h):
        """fp64 [len, D] keys or values of a request's head."""
        pool = self.k if which == "k" else self.v
        scale = self.k_scale if which == "k" else self.v_scale
        n = max(self.lens[b], 0)
        x = torch.empty(n, self.D, dtype=torch.float64)
        for j0 in range(-(-n // self.page)):
            m = min(self.page, n - j0 * self.page)
            x[j0 * self.page:j0 * self.page + m] = pool[int(self.table[b, j0]), h, :m].float().double()
        return x if scale is None else x * float(scale[h])

    def device(self):
        """(KvPages, KvBatch) over device copies with the same strides."""
        def up(x):
            base = x._base if x._base is not None else x
            raw = base.view(torch.uint8).cuda().view(x.dtype)
            return raw.as_strided(x.shape, x.stride(), x.storage_offset())
        if self.k._base is not None and self.k._base is self.v._base:
            raw = self.k._base.view(torch.uint8).cuda().view(self.k.dtype)
            self.dk, self.dv = (raw.as_strided(x.shape, x.stride(), x.storage_offset()) for x in (self.k, self.v))
        else:
            self.dk, self.dv = up(self.k), up(self.v)
        sc = [None if s is None else s.cuda() for s in (self.k_scale, self.v_scale)]
        pages = moe.KvPages(self.dk, self.dv, *sc)
        return pages, self.batch()

    def batch(self):
        return moe.KvBatch(torch.from_numpy(self.start).cuda(),
                           torch.tensor(self.lens, dtype=torch.int32).cuda(), torch.from_numpy(self.table).cuda(),
                           self.T, max(self.ns + [0]))


def strided_rows(T, H, D, pad, g, std=1.0):
    """bf16 [T, H, D] rows inside wider rows (pad columns, a multiple of 8, after each token)."""
    x = (torch.randn(T, H * D + pad, generator=g) * std).to(torch.bfloat16)
    return x[:, :H * D].unflatten(1, (H, D))


def attention_ref(P: Paged, q, Hq, scale, window):
    """(o, bound) in fp64 [T, Hq, D]; rows outside every request are NaN.

    bound: the largest error of a kernel with scores summed in fp32 (any order, one more bit for
    the tensor cores' alignment), weights rounded once to bf16 or better and fp32 sums:
      dp/p <= 2 ds + 2^-21 with ds = 2 D u32 scale sum|q||k|,  and each weight's rounding u16,
    on sum p|v| / sum p, then one rounding of the output."""
    G, D = Hq // P.Hkv, P.D
    o = torch.full((P.T, Hq, D), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(o)
    for b in range(P.B):
        n, L = P.ns[b], max(P.lens[b], 0)
        rows = slice(int(P.start[b]), int(P.start[b]) + n)
        at = torch.arange(P.lens[b] - n, P.lens[b]).view(n, 1, 1)
        j = torch.arange(L)
        hidden = j > at
        if window:
            hidden = hidden | (j <= at - window)
        for h in range(P.Hkv):
            qh = q[rows, h * G:(h + 1) * G].double()
            k, v = P.rows("k", b, h), P.rows("v", b, h)
            s = torch.einsum("tgd,jd->tgj", qh, k) * scale
            # what a row does not see counts as nothing, whatever it holds
            w = torch.softmax(s.masked_fill(hidden, -torch.inf), -1).masked_fill(hidden, 0.0)
            vv = v.unsqueeze(0).expand(n, L, D).masked_fill(hidden.view(n, L, 1), 0.0)
            o[rows, h * G:(h + 1) * G] = torch.einsum("tgj,tjd->tgd", w, vv)
            mag = torch.einsum("tgj,tjd->tgd", w, vv.abs())
            size = (torch.einsum("tgd,jd->tgj", qh.abs(), k.abs()) * abs(scale)).masked_fill(hidden, 0.0)
            ds = 2 * D * U_F32 * size.amax(-1, keepdim=True) if L else torch.zeros(n, G, 1).double()
            tol[rows, h * G:(h + 1) * G] = mag * (U_BF16 + 2 * ds + 2.0 ** -21 + 2 * L * U_F32)
    return o, tol + o.abs() * U_BF16 * (1 + 2.0 ** -8) + 1e-30

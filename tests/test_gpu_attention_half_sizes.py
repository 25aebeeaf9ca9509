"""The attention half at the sizes that serving has: thousands of rows, hundreds of thousands of keys."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import E4M3_STEP, U_BF16, U_E4M3, U_F32
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Cache:
    """Shuffled pages on the GPU: `lens` tokens a request, the last `ns` of them new."""

    def __init__(self, lens, ns, Hkv, D, page, e4m3, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        per = [-(-n // page) for n in lens]
        order = np.random.RandomState(seed).permutation(sum(per))
        table, at = np.full((len(lens), max(per)), -1, dtype=np.int32), 0
        for b, n in enumerate(per):
            table[b, :n], at = order[at:at + n], at + n
        self.table = torch.from_numpy(table).cuda()
        self.lens, self.ns, self.page, self.T = lens, ns, page, sum(ns)
        shape = (sum(per), Hkv, page, D)
        self.k, self.v = (torch.randn(shape, generator=self.g, device="cuda").to(E4M3 if e4m3 else torch.bfloat16) for _ in range(2))
        self.k_scale, self.v_scale = ((torch.rand(Hkv, generator=self.g, device="cuda") * 0.5 + 0.75) if e4m3 else None for _ in range(2))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.start = np.concatenate([[0], np.cumsum(ns)])
        self.batch = moe.KvBatch(i32(self.start.tolist()), i32(lens), self.table, self.T, max(ns))
        self.pages = moe.KvPages(self.k, self.v, self.k_scale, self.v_scale)

    def rows(self, pool, scale, b, h):
        """fp64 [len, D] of a request's head."""
        n = self.lens[b]
        x = pool[:, h].view(torch.uint8 if pool.dtype == E4M3 else torch.int16)[self.table[b, :-(-n // self.page)].long()]
        x = x.view(pool.dtype).double().flatten(0, 1)[:n]
        return x if scale is None else x * scale[h].double()


ATTENTION = [
    # lens, new, Hq, Hkv, D, page, window, e4m3
    ([262143], [1], 32, 4, 128, 64, 0, False),
    ([131071, 70001], [1, 1], 16, 2, 64, 16, 0, True),
    ([200000], [4], 16, 2, 256, 64, 0, True),
    ([16384, 9000, 16000], [1, 1, 1], 24, 8, 64, 32, 4096, False),
    ([6000, 5003], [512, 333], 32, 4, 128, 64, 0, False),
    ([6000, 5003], [512, 333], 32, 4, 128, 64, 0, True),
    ([6000, 5003], [512, 333], 32, 4, 64, 64, 0, False),
    ([6000, 5003], [512, 333], 32, 4, 64, 64, 0, True),
    ([4100, 2048], [512, 333], 16, 2, 256, 64, 0, False),
    ([4100, 2048], [512, 333], 16, 2, 256, 64, 0, True),
    ([8192], [2048], 8, 1, 128, 64, 1024, False),
]


@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,page,window,e4m3", ATTENTION)
def test_attention(lens, ns, Hq, Hkv, D, page, window, e4m3):
    c = Cache(lens, ns, Hkv, D, page, e4m3, seed=D + lens[0])
    G, scale = Hq // Hkv, D ** -0.5
    q = (1.5 * torch.randn(c.T, Hq, D, generator=c.g, device="cuda")).to(torch.bfloat16)
    o, ws = torch.empty_like(q), moe.AttnWorkspace(Hq, Hkv, D)
    moe.moe_paged_attention(c.pages, c.batch, q, o, ws, scale, window)
    assert moe.moe_attn_sync_status(ws) == moe.MOE_OK
    for b, (n, L) in enumerate(zip(ns, lens)):
        for h in range(Hkv):
            k, v = c.rows(c.k, c.k_scale, b, h), c.rows(c.v, c.v_scale, b, h)
            for t0 in range(0, n, 128):
                t1 = min(t0 + 128, n)
                rows = slice(int(c.start[b]) + t0, int(c.start[b]) + t1)
                qq = q[rows, h * G:(h + 1) * G].double()
                at = torch.arange(L - n + t0, L - n + t1, device="cuda").view(-1, 1, 1)
                j = torch.arange(L, device="cuda")
                hidden = (j > at) | (j <= at - window) if window else j > at
                w = torch.softmax((qq @ k.T * scale).masked_fill(hidden, -torch.inf), -1)
                ref, mag = w @ v, w @ v.abs()
                # scores: fp32 sums of D products, and over E4M3 keys a column of q off by 2^-22 of the largest;
                # weights: twice that, one rounding; sums: the tensor core adds 16 keys a step
                ds = (2 * D * U_F32 * (qq.abs() @ k.abs().T)).masked_fill(hidden, 0).amax(-1, keepdim=True) * scale
                if e4m3:
                    ds = ds + 2.0 ** -22 * qq.abs().amax(-1, keepdim=True) * k.abs().sum(1).max() * scale
                tol = mag * (U_BF16 + 2 * ds + 2.0 ** -21 + 2 * (L / 8) * U_F32) + ref.abs() * U_BF16 * (1 + 2.0 ** -8)
                got = o[rows, h * G:(h + 1) * G].double()
                assert ((got - ref).abs() <= tol).all(), (b, h, t0, float(((got - ref).abs() / tol).max()))


@pytest.mark.parametrize("B,n,Hq,Hkv,D,rot,il,page,e4m3", [(2, 4096, 32, 4, 128, 128, False, 64, False),
                                                          (2, 4096, 32, 4, 128, 128, True, 64, True),
                                                          (1, 8192, 16, 2, 256, 64, False, 16, True),
                                                          (1, 8191, 6, 3, 64, 32, True, 128, False)])
def test_append(B, n, Hq, Hkv, D, rot, il, page, e4m3):
    c = Cache([n + 809 * (b + 1) for b in range(B)], [n] * B, Hkv, D, page, e4m3, seed=D + rot)
    raw = torch.uint8 if e4m3 else torch.int16
    old = [p.view(raw).clone() for p in (c.k, c.v)]
    qkv = torch.randn(c.T, Hq + 2 * Hkv, D, generator=c.g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    qo, err = torch.empty(c.T, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_kv_append(c.pages, c.batch, moe.Rope(rot, inv_freq=f, interleaved=il), q, qo, k, v, err=err)
    assert int(err) == 0
    pos = torch.cat([torch.arange(L - n, L, device="cuda") for L in c.lens])
    a = pos.double().view(-1, 1, 1) * torch.from_numpy(f).cuda()
    i = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, rot // 2), slice(rot // 2, rot))
    ref, size = qkv.double(), torch.zeros(qkv.shape, dtype=torch.float64, device="cuda")
    x, y = ref[:, :Hq + Hkv, i[0]].clone(), ref[:, :Hq + Hkv, i[1]].clone()
    ref[:, :Hq + Hkv, i[0]], ref[:, :Hq + Hkv, i[1]] = x * a.cos() - y * a.sin(), y * a.cos() + x * a.sin()
    size[:, :Hq + Hkv, i[0]] = size[:, :Hq + Hkv, i[1]] = x.abs() + y.abs()
    rel = 16 * U_F32  # a fraction of a turn off by 2^-24, sincospif, two products and a sum

    def near(got, want, pair, e4m3=False, s=1.0):
        tol = (1 + U_BF16) * rel * pair / s
        if e4m3:
            want = (want / s).clamp(-448, 448)
            tol = tol + (U_E4M3 * want.abs()).clamp(min=E4M3_STEP / 2) + 8 * U_F32 * want.abs()
        else:
            tol = tol + U_BF16 * want.abs()
        assert ((got.double() - want).abs() <= tol).all()

    near(qo, ref[:, :Hq], size[:, :Hq])
    request = torch.arange(B, device="cuda").repeat_interleave(n)
    page_of, place = c.table[request, pos // page].long(), pos % page
    for pool, before, scale, h0 in ((c.k, old[0], c.k_scale, Hq), (c.v, old[1], c.v_scale, Hq + Hkv)):
        got = pool.view(raw)[page_of, :, place].view(pool.dtype).float()
        s = 1.0 if scale is None else scale.double().view(1, -1, 1)
        near(got, ref[:, h0:h0 + Hkv], size[:, h0:h0 + Hkv], e4m3, s)
        now = pool.view(raw).clone()
        now[page_of, :, place] = before[page_of, :, place]
        assert torch.equal(now, before)  # nothing else was written


@pytest.mark.parametrize("T,H,post,gate,sigmoid", [(8192, 2048, True, "row", False), (8192, 4096, False, "token", True),
                                                  (8191, 1000, True, "token", False), (4096, 4095, True, None, False),
                                                  (2048, 16384, True, "token", True), (65536, 256, False, "row", True),
                                                  (100000, 64, True, None, False)])
def test_norm(T, H, post, gate, sigmoid):
    g = torch.Generator(device="cuda").manual_seed(H)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = lambda x: x.to(torch.bfloat16)  # noqa: E731
    x, y = normal(T, H) * 3, bf(normal(T, H))
    w_post, w_pre = bf(1 + 0.1 * normal(H)), bf(1 + 0.1 * normal(H))
    gt = None if gate is None else bf(normal(1 if gate == "row" else T, H))
    d = moe.block_norm_desc(y=y, post_norm=post, w_post=w_post if post else None, gate=gt, gate_sigmoid=sigmoid, res_scale=0.5,
                            w_pre=w_pre)
    out, xn = torch.empty_like(x), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_norm(d, x, out, xn, T, H)
    for t0 in range(0, T, 8192):
        r = slice(t0, t0 + 8192)
        z = y[r].double()
        if post:
            z = w_post.double() * z / (z.square().mean(1, keepdim=True) + 1e-6).sqrt()
        if gt is not None:
            gg = (gt if gate == "row" else gt[r]).double()
            z = z * (torch.sigmoid(gg) if sigmoid else gg)
        want = x[r].double() + 0.5 * z
        # a sum of H squares over threads and lanes, a root, a division, three products and a sum in fp32
        rel = (H / 32 + 64) * U_F32
        tol = rel * (x[r].double().abs() + z.abs()) + U_F32 * want.abs()
        assert ((out[r].double() - want).abs() <= tol).all()
        s = (want.square().mean(1, keepdim=True) + 1e-6).sqrt()
        n = w_pre.double() * want / s
        size = (x[r].double().abs() + z.abs()) * w_pre.double().abs() / s
        assert ((xn[r].double() - n).abs() <= U_BF16 * n.abs() + (1 + U_BF16) * (2 * rel * size + rel * n.abs()) + 1e-30).all()

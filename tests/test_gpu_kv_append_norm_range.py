"""Norms of heads whose squares leave fp32: the definition has no limit there."""
import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import E4M3_STEP, U_BF16, U_E4M3, Paged
from tests.gpu_util import require_gpu
from tests.test_gpu_kv_append_norm import fp32_bound, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rows(T, H, D, seed):
    """Heads of sizes around 2^60 .. 2^126, some with one large column alone, some small, some zero."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g).to(torch.bfloat16).clamp(-3, 3)
    size = torch.tensor([0.0, 2.0 ** -30, 1.0, 2.0 ** 60, 2.0 ** 63, 2.0 ** 64, 2.0 ** 100, 2.0 ** 126])
    pick = torch.randint(0, len(size), (T, H, 1), generator=g)
    x = (x.float() * size[pick]).to(torch.bfloat16)
    alone = torch.randint(0, 4, (T, H), generator=g) == 0
    x[alone] = torch.where(torch.arange(D) == D // 3, x[alone], torch.zeros_like(x[alone]))
    return x


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 0, False), (64, 64, True), (128, 64, False), (256, 256, False)])
@pytest.mark.parametrize("eps", [1e-6, 1e30])
def test_rows_of_any_size(D, rot, interleaved, e4m3, eps):
    P = Paged([40, 30], [29, 23], 2, D, 16, e4m3=e4m3, seed=D)
    q, k = rows(P.T, 5, D, 1), rows(P.T, 2, D, 2)
    g = torch.Generator().manual_seed(3)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) for _ in range(2))
    freq = 1e4 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) if rot else np.zeros(0)
    pages, batch = P.device()
    qo, err = torch.empty(P.T, 5, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_kv_append_norm(pages, batch, moe.Rope(rot, inv_freq=freq, interleaved=interleaved) if rot else None,
                           moe.HeadNorm(wq.cuda(), wk.cuda(), eps), q.cuda(), qo, k.cuda(), torch.zeros_like(k).cuda(), err=err)
    assert err.item() == 0
    at = [(b, i, P.lens[b] - P.ns[b] + i) for b in range(2) for i in range(P.ns[b])]
    pos = [p for _, _, p in at]
    ref, size = reference(q, wq, pos, freq, interleaved, eps)
    bound = fp32_bound(D, size, True)
    assert ((qo.cpu().double() - ref).abs() <= (ref.abs() + bound) * U_BF16 + bound + 2.0 ** -133).all()
    assert (ref.abs().amax(2) > 0.5).float().mean() > (0.3 if eps < 1 else 0.1)
    ref, size = reference(k, wk, pos, freq, interleaved, eps)
    got = torch.stack([P.dk[int(P.table[b, p // 16]), :, p % 16].float().cpu() for b, _, p in at]).double()
    bound = fp32_bound(D, size, True)
    if e4m3:
        s = P.k_scale.double().cpu().view(1, -1, 1)
        ref, bound = ref / s, bound / s + (ref / s).abs() * 2.0 ** -24
        off = (got - ref.clamp(-448, 448)).abs() - (ref.abs() + bound) * U_E4M3 - bound - E4M3_STEP / 2
    else:
        off = (got - ref).abs() - (ref.abs() + bound) * U_BF16 - bound - 2.0 ** -133
    assert (off <= 0).all(), float(off.max())


def test_infinities_stay_in_their_heads():
    """As the definition has it: infinity over infinity is NaN, what is finite over it 0."""
    P = Paged([8], [8], 1, 64, 16, seed=1)
    q = rows(8, 3, 64, 5)
    q[2, 1, 7] = float("inf")
    q[5, 0, 9] = float("nan")
    pages, batch = P.device()
    qo = torch.empty(8, 3, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(8, 1, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_append_norm(pages, batch, None, moe.HeadNorm(), q.cuda(), qo, kv, kv)
    o = qo.cpu().float()
    assert o[2, 1, 7].isnan() and (o[2, 1, torch.arange(64) != 7] == 0).all() and o[5, 0].isnan().all()
    o[2, 1], o[5, 0] = 0, 0
    assert o.isfinite().all()

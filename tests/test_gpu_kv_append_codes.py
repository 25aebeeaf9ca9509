"""E4M3 codes of moe_kv_append: those of x / scale, code for code."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


SCALES = [1.0, 0.02, 0.0371, 3.0, 1 / 3, -0.7, 2.0 ** -20, 1e-6, 448.0, 1e10, 1e20, 1e-20, 5e-20, 3e38, 2.0 ** -127,
          1.1 * 2.0 ** -130, 1e-44, 0.0, float("inf"), float("nan")] + [0.02 + 0.0001234 * i for i in range(12)]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_bf16_value_by_every_scale(D):
    """All 65536 bit patterns through every scale: ties, the smallest codes, saturation, infinities and NaN."""
    H, T = len(SCALES), 65536 // D
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(T, 1, D)
    scale = torch.tensor(SCALES, dtype=torch.float32)
    rows = x.expand(T, H, D).contiguous().cuda()
    pool = lambda: torch.zeros(T // 64, H, 64, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    k, v = pool(), pool()
    i32 = lambda t: torch.as_tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    bt = moe.KvBatch(i32([0, T]), i32([T]), i32(torch.arange(T // 64)).view(1, -1), T, T)
    moe.moe_kv_append(moe.KvPages(k, v, scale.cuda(), scale.cuda()), bt, None, None, None, rows, rows)
    q = x.float() / scale.view(1, H, 1)  # rounded once, to fp32
    want = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    nan = q.isnan()
    for got in (k, v):
        got = got.view(torch.uint8).cpu().permute(0, 2, 1, 3).reshape(T, H, D)
        assert ((got & 0x7F) == 0x7F)[nan].all()
        off = (got != want) & ~nan
        assert not off.any(), [(int(n), SCALES[h]) for h, n in enumerate(off.sum((0, 2))) if n]

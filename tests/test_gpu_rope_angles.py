"""The angle of far positions in moe_kv_append, against arithmetic of 60 digits."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import U_BF16, U_F32
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def sine(turn: Decimal) -> float:
    """sin of a small angle."""
    x = 2 * PI * turn
    return float(x - x ** 3 / 6 + x ** 5 / 120)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("p", [2 ** 31 - 2, 1_000_003, 4097])
def test_angles_close_to_a_whole_turn(p, sign):
    """Frequencies that bring position p within a double's last bit of whole turns: what is left is the sine."""
    getcontext().prec = 60
    r = np.random.RandomState(7)
    f = np.array([float(2 * PI * int(n) / p) for n in np.exp(r.uniform(np.log(p / 1e3), np.log(p), 32))]) * sign
    left = [Decimal(x) * p / (2 * PI) for x in f]
    left = [x - x.to_integral_value() for x in left]
    D, page = 64, 65536
    k = torch.zeros(1, 1, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.full((1, p // page + 1), -1, dtype=torch.int32)
    table[0, -1] = 0
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    bt = moe.KvBatch(i32(0, 1), i32(p + 1), table.cuda(), 1, 1)
    x = torch.zeros(1, 1, D, dtype=torch.bfloat16, device="cuda")
    x[..., :32] = 1.0  # (1, 0) turns to (cos, sin)
    q, err = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_kv_append(moe.KvPages(k, v), bt, moe.Rope(D, inv_freq=f), x, q, x, x, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    want = torch.tensor([sine(t) for t in left], dtype=torch.float64)
    assert (want.abs() > 0).all() and float(want.abs().max()) < 1e-5
    # the table's 64 bits at position p, then the fp32 fraction, sincospif and one rounding
    tol = 6.3 * p * 2.0 ** -65 + (U_BF16 + 16 * U_F32) * want.abs()
    for got in (q[0, 0].cpu().double(), k[0, 0, p % page].cpu().double()):
        assert (got[:32] == 1).all()
        assert ((got[32:] - want).abs() <= tol).all(), float(((got[32:] - want).abs() / tol).max())

"""moe_block_norm against its formula in 64 bits."""
import pytest
import torch

from serving_router_top_gb300 import moe
from tests.attn_util import U_BF16, U_F32
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rows(T, H, pad, off, dtype, g, std=1.0):
    """[T, H] rows at an offset inside wider rows, on the device."""
    base = (torch.randn(T, H + pad + off, generator=g) * std).to(dtype).cuda()
    return base[:, off:off + H]


def reference(x, y, post, w_post, gate, sig, scale, w_pre, eps):
    x = x.double().cpu()
    H = x.shape[1]
    part = torch.zeros_like(x)
    if y is not None:
        z = y.double().cpu()
        if post:
            z = z / (z.square().mean(1, keepdim=True) + eps).sqrt()
            z = z if w_post is None else z * w_post.double().cpu()
        if gate is not None:
            z = z * (torch.sigmoid(gate.double().cpu()) if sig else gate.double().cpu())
        part = scale * z
    out = x + part
    xn = out / (out.square().mean(1, keepdim=True) + eps).sqrt()
    xn = xn if w_pre is None else xn * w_pre.double().cpu()
    # fp32 sums of H squares (relative H u in any order, halved by the root), the sigmoid's fast
    # exponential (2 + 1.2 |g| ulp, |g| < 8) and a few products
    rel = (H / 2 + 64) * U_F32
    tol_x = U_F32 * out.abs() + rel * part.abs()
    # an element's own error, and that of the row's norm
    root = (out.square().mean(1, keepdim=True) + eps).sqrt()
    tol_n = U_BF16 * xn.abs() + (1 + U_BF16) * (
        (tol_x / root) * (1.0 if w_pre is None else w_pre.double().cpu().abs())
        + xn.abs() * (rel + (tol_x.square().mean(1, keepdim=True).sqrt() / root))) + 1e-38
    return out, xn, tol_x + 1e-38, tol_n


CASES = [
    # T, H, pad, off, post, w, gate, sigmoid, scale
    (1, 1, 0, 0, True, True, "token", True, 1.0),
    (3, 7, 0, 0, True, True, "row", False, 0.5),
    (4, 2048, 0, 0, True, True, None, False, 1.0),
    (4, 2048, 8, 0, True, True, "token", True, 0.7),
    (5, 2048, 3, 1, True, True, "token", False, -1.0),
    (2, 2056, 0, 0, False, True, "row", True, 1.0),
    (64, 4096, 0, 0, False, True, "token", True, 0.5),
    (3, 4097, 0, 0, True, False, "row", False, 2.0),
    (2, 5000, 0, 0, True, True, "token", False, 1.0),
    (2, 16384, 0, 0, True, True, "row", True, 1.0),
    (2, 16383, 0, 0, True, True, "token", True, 1.0),
    (300, 264, 16, 8, True, True, "token", True, 1.0),
    (9, 512, 0, 0, False, False, None, False, 1.0),
    (5, 8, 0, 0, True, True, "token", True, 1.0),
    (6, 256, 8, 0, True, True, "row", True, 1.0),
    (5, 520, 0, 0, True, True, "token", True, 1.0),
    (3, 4104, 8, 8, True, True, "token", True, 1.0),
    (3, 8192, 0, 0, True, True, "token", False, 1.0),
    (3, 8200, 0, 0, True, True, "row", True, 1.0),
]


@pytest.mark.parametrize("T,H,pad,off,post,w,gate,sig,scale", CASES)
def test_block_norm(T, H, pad, off, post, w, gate, sig, scale):
    g = torch.Generator().manual_seed(T * 1000 + H)
    bf, eps = torch.bfloat16, 1e-6
    x, y = rows(T, H, pad, off, torch.float32, g, 3.0), rows(T, H, pad, off, bf, g)
    xo, xn = rows(T, H, pad, off, torch.float32, g), rows(T, H, pad, off, bf, g)
    wp, wq = ((1 + 0.2 * torch.randn(H, generator=g)).to(bf).cuda() if w else None for _ in range(2))
    gt = None if gate is None else rows(T if gate == "token" else 1, H, pad, off, bf, g)
    d = moe.block_norm_desc(y=y, post_norm=post, w_post=wp if post else None, gate=gt, gate_sigmoid=sig, res_scale=scale,
                            w_pre=wq, eps=eps)
    moe.moe_block_norm(d, x, xo, xn, T, H)
    out, ref, tx, tn = reference(x, y, post, wp if post else None, gt, sig, scale, wq, eps)
    assert ((xo.cpu().double() - out).abs() <= tx).all()
    assert ((xn.cpu().double() - ref).abs() <= tn).all()
    once = xo.clone(), xn.clone()
    moe.moe_block_norm(d, x, x, xn, T, H)  # in place: the same bits
    assert torch.equal(x, once[0]) and torch.equal(xn, once[1])


def test_columns_beside_the_rows_stay():
    base, nb = torch.full((4, 80), 5.0, device="cuda"), torch.full((4, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(4, 64, device="cuda")
    moe.moe_block_norm(moe.block_norm_desc(), x, base[:, 8:72], nb[:, :64], 4, 64)
    assert torch.equal(base[:, 8:72], x)
    assert (base[:, :8] == 5).all() and (base[:, 72:] == 5).all() and (nb[:, 64:] == 5).all()


def test_one_output_only_and_no_block():
    g = torch.Generator().manual_seed(2)
    x, y = rows(3, 96, 0, 0, torch.float32, g), rows(3, 96, 0, 0, torch.bfloat16, g)
    xo, xn = torch.empty_like(x), torch.empty_like(y)
    d = moe.block_norm_desc(y=y, post_norm=True)
    moe.moe_block_norm(d, x, xo, xn, 3, 96)
    a, b = torch.empty_like(x), torch.empty_like(y)
    moe.moe_block_norm(d, x, a, None, 3, 96)
    moe.moe_block_norm(d, x, None, b, 3, 96)
    assert torch.equal(a, xo) and torch.equal(b, xn)
    moe.moe_block_norm(moe.block_norm_desc(), x, a, b, 3, 96)
    assert torch.equal(a, x)
    out, ref, _, tn = reference(x, None, False, None, None, False, 1.0, None, 1e-6)
    assert ((b.cpu().double() - ref).abs() <= tn).all()


def test_agrees_with_residual_rmsnorm():
    g = torch.Generator().manual_seed(4)
    x, y = rows(16, 2048, 0, 0, torch.float32, g), rows(16, 2048, 0, 0, torch.bfloat16, g)
    xo, xn, xm = torch.empty_like(x), torch.empty_like(y), torch.empty_like(y)
    moe.moe_block_norm(moe.block_norm_desc(y=y), x, xo, xn, 16, 2048)
    moe.moe_residual_rmsnorm(x, y, xm, 16, 2048)
    assert torch.equal(xo, x)
    ulp = (xn.view(torch.int16).int() - xm.view(torch.int16).int()).abs()
    assert int(ulp.max()) <= 1  # the sums of squares run in another order


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_stay_in_their_row(value):
    g = torch.Generator().manual_seed(6)
    x, y = rows(4, 640, 0, 0, torch.float32, g), rows(4, 640, 0, 0, torch.bfloat16, g)
    y[2, 33] = value
    xo, xn = torch.empty_like(x), torch.empty_like(y)
    moe.moe_block_norm(moe.block_norm_desc(y=y, post_norm=True), x, xo, xn, 4, 640)
    ok = torch.tensor([0, 1, 3], device="cuda")
    assert xo[ok].isfinite().all() and xn[ok].isfinite().all() and not xn[2].isfinite().all()


def test_zero_rows():
    z, y = torch.zeros(2, 128, device="cuda"), torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    xo, xn = torch.ones_like(z), torch.ones_like(y)
    moe.moe_block_norm(moe.block_norm_desc(y=y, post_norm=True), z, xo, xn, 2, 128)
    assert (xo == 0).all() and (xn == 0).all()

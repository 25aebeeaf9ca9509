"""The decoder path: attention half and expert half together, in chunks and windows."""
import pytest
import torch

from serving_router_top_gb300 import inputs as I
from serving_router_top_gb300 import moe
from serving_router_top_gb300.decoder import AttentionShape, Decoder
from tests.attn_util import U_BF16
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def small(requests, s, layers=2):
    # every token takes every expert: no routing decision that a rounding could turn
    w = I.small_workload(T=4, H=256, I=128, E=4, k=4, I_shared=128, layers=layers, seed=5)
    return Decoder(w, s, requests=requests, max_len=96, maxT=128)


@pytest.mark.parametrize("s", [AttentionShape(8, 2, 64, 64, page=16), AttentionShape(4, 4, 128, 32, page=8, window=20),
                               AttentionShape(6, 1, 64, 16, page=32, e4m3=True)])
def test_windows_continue_a_prompt(s):
    """Two requests' prompts at once, then windows of 4 and single tokens, against everything in one chunk."""
    g = torch.Generator().manual_seed(0)
    total = [48, 33]
    x = [torch.randn(n, 256, generator=g) for n in total]
    whole = small(2, s)
    res = torch.cat(x).cuda()
    ref = whole.forward(res, whole.batch(total)).float().cpu()
    whole.check()
    ref = [ref[:total[0]], ref[total[0]:]]
    d = small(2, s)
    at, out = [0, 0], [[], []]
    for new in ([40, 20], [4, 4], [1, 0], [2, 4], [1, 5]):
        rows = torch.cat([x[r][at[r]:at[r] + n] for r, n in enumerate(new)]).cuda()
        xn = d.forward(rows, d.batch(new)).float().cpu()
        out[0].append(xn[:new[0]])
        out[1].append(xn[new[0]:])
        at = [a + n for a, n in zip(at, new)]
    d.check()
    assert at == total
    for r in range(2):
        got = torch.cat(out[r])
        # bf16 activations at four places a layer, two layers, other kernels for chunks than for windows:
        # rows agree to a few bf16 roundings of their size
        err = (got - ref[r]).norm(dim=1) / ref[r].norm(dim=1)
        assert float(err.max()) <= 16 * U_BF16


def test_attention_of_a_layer_against_64_bits():
    s = AttentionShape(8, 2, 64, 64, page=16)
    d = small(1, s, layers=1)
    g = torch.Generator().manual_seed(1)
    xn = torch.randn(50, 256, generator=g).to(torch.bfloat16).cuda()
    y = torch.empty_like(xn)
    d.attention(0, xn, d.batch([50]), y)
    d.check()
    qkv = torch.matmul(xn, d.layers[0].qkv).double().cpu().view(50, 12, 64)
    a = torch.arange(50.0, dtype=torch.float64).view(-1, 1, 1) * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    u, w = qkv[:, :10, :32], qkv[:, :10, 32:]
    qk = torch.cat([u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()], -1)
    q, k, v = qk[:, :8], qk[:, 8:], qkv[:, 10:]
    k, v = (t.repeat_interleave(4, 1) for t in (k, v))
    score = torch.einsum("thd,jhd->htj", q, k) / 8
    score = score.masked_fill(torch.ones(50, 50, dtype=torch.bool).triu(1), -torch.inf)
    o = torch.einsum("htj,jhd->thd", torch.softmax(score, -1), v)
    ref = o.reshape(50, -1) @ d.layers[0].out.double().cpu()
    # q and k rounded after the turn, weights, o and y rounded once each: relative to the sums of absolute values
    mag = torch.einsum("htj,jhd->thd", torch.softmax(score, -1), v.abs()).reshape(50, -1) @ d.layers[0].out.double().abs().cpu()
    ds = 2 * U_BF16 * (torch.einsum("thd,jhd->htj", q.abs(), k.abs()) / 8).max()
    assert ((y.double().cpu() - ref).abs() <= mag * (2 * ds + 2 * U_BF16) + ref.abs() * U_BF16 + 1e-6).all()


def test_a_decode_step_in_a_graph():
    """A step captured once and replayed with the lengths moved on the device."""
    s = AttentionShape(8, 2, 64, 64, page=16)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(24, 256, generator=g)
    ref = small(1, s)
    a = ref.forward(x[:16].cuda(), ref.batch([16]))
    want = [ref.forward(x[16 + i:17 + i].cuda(), ref.batch([1])).clone() for i in range(8)]
    d = small(1, s)
    d.forward(x[:16].cuda(), d.batch([16]))
    d.pages.reserve(0, 96)
    bt = d.batch([1])  # at position 16
    rows, src = torch.empty(1, 256, device="cuda"), x[16:17].cuda()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            rows.copy_(src)
            xn = d.forward(rows, bt)
            bt.kv_len.add_(1)
        for i in range(8):
            src.copy_(x[16 + i:17 + i])
            graph.replay()
            stream.synchronize()
            assert torch.equal(xn, want[i]), i
    d.check()
    assert a is not None and moe.moe_attn_sync_status(d.ws) == moe.MOE_OK

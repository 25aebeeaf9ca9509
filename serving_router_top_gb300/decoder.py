"""A whole decoder: attention over a paged cache in front of every MoE layer.

Each layer of a :class:`~serving_router_top_gb300.model.ModelState` gets the
attention half that its expert path comes after, on the same fp32 residual
stream:

    xn      = norm(x_res += MoE output of the layer before)     moe_block_norm
    q, k, v = xn W_qkv                                          library GEMM
    rotate q and k, append k and v to the pages                 moe_kv_append
    o       = attention over the request's pages                moe_paged_attention
    y       = o W_o                                             library GEMM
    xn      = norm(x_res += gate * post-norm(y))                moe_block_norm
    y       = MoE(xn)                                           moe_layer_forward

One call serves new tokens of several requests at once: a prompt chunk, a verify
window, one token, or a mixture, on the current stream.  ``python -m serving_router_top_gb300.decoder``
runs a prompt and decode windows of a small model and prints the times.
"""
from __future__ import annotations

import dataclasses
from typing import Dict, List, Sequence

import torch

from . import inputs as I
from . import moe
from .model import ModelState


@dataclasses.dataclass(frozen=True)
class AttentionShape:
    Hq: int                  # query heads
    Hkv: int                 # key heads
    D: int                   # columns of a head: 64, 128 or 256
    rot: int                 # columns that turn with the position
    page: int = 64           # tokens in a page
    e4m3: bool = False       # 8-bit cache
    window: int = 0          # visible keys, 0: all
    theta: float = 10000.0


@dataclasses.dataclass
class AttentionWeights:
    qkv: torch.Tensor        # bf16 [H, (Hq + 2 Hkv) D]
    out: torch.Tensor        # bf16 [Hq D, H]
    gate: torch.Tensor       # bf16 [1, H], of the attention's output
    norm_in: torch.Tensor    # bf16 [H], before the attention
    norm_out: torch.Tensor   # bf16 [H], after it
    norm_moe: torch.Tensor   # bf16 [H], before the experts


def attention_weights(H: int, s: AttentionShape, seed: int, layer: int) -> AttentionWeights:
    g = torch.Generator(device="cuda").manual_seed(seed * 1009 + layer)
    bf = torch.bfloat16
    normal = lambda *n, std=1.0: (torch.randn(*n, generator=g, device="cuda") * std).to(bf)  # noqa: E731
    near_one = lambda: (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(bf)  # noqa: E731
    return AttentionWeights(normal(H, (s.Hq + 2 * s.Hkv) * s.D, std=H ** -0.5), normal(s.Hq * s.D, H, std=(s.Hq * s.D) ** -0.5),
                            (0.5 + 0.1 * normal(1, H)).to(bf), near_one(), near_one(), near_one())


class Pages:
    """Page tables of the requests and the free pages, on the host; the same pages in every layer's pools."""

    def __init__(self, requests: int, npages: int, page: int, max_len: int):
        self.page, self.free = page, list(range(npages))[::-1]
        self.table = torch.full((requests, -(-max_len // page)), -1, dtype=torch.int32)
        self.held = [0] * requests
        self.device = self.table.cuda()

    def reserve(self, request: int, length: int) -> None:
        """Pages for `length` tokens of a request."""
        self.reserve_all({request: length})

    def reserve_all(self, lengths: Dict[int, int]) -> None:
        """Pages for that many tokens of each request, or none for any of them."""
        left = len(self.free)
        for request, length in lengths.items():
            need = -(-length // self.page)
            left -= max(need - self.held[request], 0)
            if need > self.table.shape[1] or left < 0:
                raise RuntimeError(f"no pages for {length} tokens of request {request}")
        for request, length in lengths.items():
            need = -(-length // self.page)
            for j in range(self.held[request], need):
                self.table[request, j] = self.free.pop()
            self.held[request] = max(self.held[request], need)

    def upload(self) -> None:
        self.device.copy_(self.table)


class Decoder:
    def __init__(self, w: I.Workload, s: AttentionShape, requests: int, max_len: int, maxT: int, eps: float = 1e-6):
        self.st = ModelState(w, maxT=maxT)
        self.s, self.H, self.eps, self.maxT = s, w.shape.H, eps, maxT
        self.layers = [attention_weights(self.H, s, w.seed, l) for l in range(self.st.L)]
        npages = requests * -(-max_len // s.page)
        self.pages = Pages(requests, npages, s.page, max_len)
        dt = torch.float8_e4m3fn if s.e4m3 else torch.bfloat16
        one = torch.ones(s.Hkv, device="cuda") if s.e4m3 else None
        pool = lambda: torch.empty(npages, s.Hkv, s.page, s.D, dtype=dt, device="cuda")  # noqa: E731
        self.kv: List[moe.KvPages] = [moe.KvPages(pool(), pool(), one, one) for _ in range(self.st.L)]
        self.rope = moe.Rope(s.rot, theta=s.theta)
        self.ws = moe.AttnWorkspace(s.Hq, s.Hkv, s.D)
        bf = torch.bfloat16
        self.xn = torch.empty(maxT, self.H, dtype=bf, device="cuda")
        self.y = torch.empty(maxT, self.H, dtype=bf, device="cuda")
        self.q = torch.empty(maxT, s.Hq, s.D, dtype=bf, device="cuda")
        self.o = torch.empty(maxT, s.Hq, s.D, dtype=bf, device="cuda")
        self.lens = [0] * requests

    def batch(self, new: Sequence[int]) -> moe.KvBatch:
        """The next call's requests: new[r] tokens of request r (pages are reserved for them).  A call
        that raises leaves lengths and pages as they were."""
        if len(new) != len(self.lens) or min(new) < 0 or sum(new) > self.maxT:
            raise ValueError(f"new tokens of {len(self.lens)} requests, at most {self.maxT} in all, got {list(new)}")
        lens = [have + n for have, n in zip(self.lens, new)]
        self.pages.reserve_all(dict(enumerate(lens)))
        self.lens = lens
        self.pages.upload()
        start = torch.tensor([0] + list(new), dtype=torch.int32).cumsum(0).to(torch.int32)
        return moe.KvBatch(start.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.pages.device,
                           int(sum(new)), max(new))

    def attention(self, l: int, xn: torch.Tensor, bt: moe.KvBatch, y: torch.Tensor) -> None:
        """y = attention of layer l on the normalised rows xn, whose keys and values join the cache."""
        s, T = self.s, bt.c.T
        qkv = torch.matmul(xn, self.layers[l].qkv).view(T, s.Hq + 2 * s.Hkv, s.D)
        q, k, v = qkv.split([s.Hq, s.Hkv, s.Hkv], 1)
        moe.moe_kv_append(self.kv[l], bt, self.rope, q, self.q[:T], k, v, err=self.ws.error_ptr)
        moe.moe_paged_attention(self.kv[l], bt, self.q[:T], self.o[:T], self.ws, scale=s.D ** -0.5, window=s.window)
        torch.matmul(self.o[:T].view(T, s.Hq * s.D), self.layers[l].out, out=y)

    def forward(self, x_res: torch.Tensor, bt: moe.KvBatch) -> torch.Tensor:
        """All layers on the residual rows x_res (fp32 [T, H], updated in place); the normalised rows."""
        T, H = bt.c.T, self.H
        xn, y = self.xn[:T], self.y[:T]
        prev = None  # output of the block before, added by the next norm
        for l, a in enumerate(self.layers):
            moe.moe_block_norm(moe.block_norm_desc(y=prev, w_pre=a.norm_in, eps=self.eps), x_res, x_res, xn, T, H)
            self.attention(l, xn, bt, y)
            d = moe.block_norm_desc(y=y, post_norm=True, w_post=a.norm_out, gate=a.gate, w_pre=a.norm_moe, eps=self.eps)
            moe.moe_block_norm(d, x_res, x_res, xn, T, H)
            self.st.forward(l, xn, y, T, y_is_fp32=False)
            prev = y
        moe.moe_block_norm(moe.block_norm_desc(y=prev, eps=self.eps), x_res, x_res, xn, T, H)
        return xn

    def check(self) -> None:
        for what, rc in (("attention", moe.moe_attn_sync_status(self.ws)), ("experts", moe.moe_sync_status(self.st.ws))):
            if rc != moe.MOE_OK:
                raise moe.MoeError(rc, what)


def main() -> None:
    w = I.small_workload(T=4, H=2048, I=512, E=64, k=8, I_shared=512, layers=4)
    s = AttentionShape(Hq=16, Hkv=2, D=256, rot=64)
    prompt, window, steps = 2048, 4, 16
    d = Decoder(w, s, requests=1, max_len=prompt + window * (steps + 2), maxT=prompt)
    x = torch.randn(prompt, d.H, device="cuda")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    d.forward(x[:window].clone(), d.batch([window]))  # first-call set-up
    ev[0].record()
    d.forward(x, d.batch([prompt]))
    ev[1].record()
    batches = [d.batch([window]) for _ in range(steps)]
    ev[2].record()
    for b in batches:
        d.forward(x[:window].clone(), b)
    ev[3].record()
    d.check()
    print(f"{d.st.L} layers, hidden {d.H}, {s.Hq} query and {s.Hkv} key heads of {s.D}: prompt of {prompt} tokens "
          f"{ev[0].elapsed_time(ev[1]):.2f} ms, a window of {window} {ev[2].elapsed_time(ev[3]) / steps * 1e3:.0f} us")


if __name__ == "__main__":
    main()

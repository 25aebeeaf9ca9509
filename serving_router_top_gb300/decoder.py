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
window, one token, or a mixture, on the current stream.  Drafted tokens may branch:

    bt, tree = d.tree_batch(parents)      a node a row, after each request's tokens
    xn       = d.forward(x, bt, tree)     moe_kv_append_norm, moe_tree_attention
    d.accept(bt, moe.verify_desc(...))    moe_verify_drafts on the target's probabilities,
                                          moe_kv_compact of the nodes it kept

and ``d.fork`` lets a request go on from another's tokens.  ``python -m serving_router_top_gb300.decoder``
runs a prompt, decode windows and trees of a small model and prints the times.
"""
from __future__ import annotations

import dataclasses
import weakref
from typing import Dict, List, Optional, Sequence, Tuple

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
    qk_norm: bool = False    # norms of each head's queries and keys


@dataclasses.dataclass
class AttentionWeights:
    qkv: torch.Tensor        # bf16 [H, (Hq + 2 Hkv) D]
    out: torch.Tensor        # bf16 [Hq D, H]
    gate: torch.Tensor       # bf16 [1, H], of the attention's output
    norm_in: torch.Tensor    # bf16 [H], before the attention
    norm_out: torch.Tensor   # bf16 [H], after it
    norm_moe: torch.Tensor   # bf16 [H], before the experts
    norm_q: torch.Tensor     # bf16 [D], of each query head, with qk_norm
    norm_k: torch.Tensor     # bf16 [D], of each key head


def attention_weights(H: int, s: AttentionShape, seed: int, layer: int) -> AttentionWeights:
    g = torch.Generator(device="cuda").manual_seed(seed * 1009 + layer)
    bf = torch.bfloat16
    normal = lambda *n, std=1.0: (torch.randn(*n, generator=g, device="cuda") * std).to(bf)  # noqa: E731
    near_one = lambda n=H: (1.0 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(bf)  # noqa: E731
    return AttentionWeights(normal(H, (s.Hq + 2 * s.Hkv) * s.D, std=H ** -0.5), normal(s.Hq * s.D, H, std=(s.Hq * s.D) ** -0.5),
                            (0.5 + 0.1 * normal(1, H)).to(bf), near_one(), near_one(), near_one(), near_one(s.D), near_one(s.D))


class Pages:
    """Page tables of the requests and the free pages, on the host; the same pages in every layer's pools."""

    def __init__(self, requests: int, npages: int, page: int, max_len: int):
        self.page, self.free = page, list(range(npages))[::-1]
        self.table = torch.full((requests, -(-max_len // page)), -1, dtype=torch.int32)
        self.held = [0] * requests
        self.users = [0] * npages  # requests that hold a page
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
                self.users[self.table[request, j]] += 1
            self.held[request] = max(self.held[request], need)

    def release(self, request: int) -> None:
        """None of its pages belong to the request any more; those of no other request are free."""
        for j in range(self.held[request]):
            id = int(self.table[request, j])
            self.users[id] -= 1
            if self.users[id] == 0:
                self.free.append(id)
        self.table[request] = -1
        self.held[request] = 0

    def fork(self, source: int, request: int, length: int) -> List[Tuple[int, int, int]]:
        """`request`, which holds no pages, gets the first `length` tokens of `source`: its whole pages are shared, as
        nothing is written to them any more, and a last one that is not full is to be copied: (from, to, tokens)."""
        whole, rest = divmod(length, self.page)
        if self.held[request] or length > self.held[source] * self.page or source == request:
            raise ValueError(f"request {request} cannot go on from {length} tokens of request {source}")
        if rest and not self.free:
            raise RuntimeError(f"no page for the last tokens of request {request}")
        for j in range(whole):
            self.table[request, j] = self.table[source, j]
            self.users[self.table[request, j]] += 1
        self.held[request] = whole
        if not rest:
            return []
        self.table[request, whole] = self.free.pop()
        self.users[self.table[request, whole]] += 1
        self.held[request] = whole + 1
        return [(int(self.table[source, whole]), int(self.table[request, whole]), rest)]

    def upload(self) -> None:
        self.device.copy_(self.table)


class Decoder:
    # trees that accept() has not seen: their batch, and the nodes of each request, 0 once it was released
    trees: Tuple[Tuple["weakref.ref[moe.KvBatch]", List[int]], ...] = ()

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
        self.kv_layers = moe.KvLayers(self.kv)
        self.norms = [moe.HeadNorm(a.norm_q, a.norm_k, eps) if s.qk_norm else None for a in self.layers]
        self.rope = moe.Rope(s.rot, theta=s.theta)
        self.ws = moe.AttnWorkspace(s.Hq, s.Hkv, s.D)
        bf = torch.bfloat16
        self.xn = torch.empty(maxT, self.H, dtype=bf, device="cuda")
        self.y = torch.empty(maxT, self.H, dtype=bf, device="cuda")
        self.q = torch.empty(maxT, s.Hq, s.D, dtype=bf, device="cuda")
        self.o = torch.empty(maxT, s.Hq, s.D, dtype=bf, device="cuda")
        self.lens = [0] * requests

    def open_tree(self, request: int) -> bool:
        """Whether the request's last tokens are a tree's nodes, of which accept() has yet to tell what stays."""
        return any(nodes[request] for _, nodes in self.trees)

    def batch(self, new: Sequence[int]) -> moe.KvBatch:
        """The next call's requests: new[r] tokens of request r (pages are reserved for them), none for one whose
        tree waits for accept().  A call that raises leaves lengths and pages as they were."""
        if len(new) != len(self.lens) or min(new) < 0 or sum(new) > self.maxT:
            raise ValueError(f"new tokens of {len(self.lens)} requests, at most {self.maxT} in all, got {list(new)}")
        for r, n in enumerate(new):
            if n and self.open_tree(r):
                raise ValueError(f"the tree of request {r} has not been verified")
        lens = [have + n for have, n in zip(self.lens, new)]
        self.pages.reserve_all(dict(enumerate(lens)))
        self.lens = lens
        self.pages.upload()
        start = torch.tensor([0] + list(new), dtype=torch.int32).cumsum(0).to(torch.int32)
        return moe.KvBatch(start.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.pages.device,
                           int(sum(new)), max(new))

    def tree_batch(self, parents: Sequence[Sequence[int]]) -> Tuple[moe.KvBatch, moe.Tree]:
        """The next call's trees: parents[r] for each node of request r, -1 for its root.  The nodes count among the
        request's tokens until accept() tells which of them stay; until then it takes no other tokens and is not
        forked.  What other requests do in between is theirs."""
        new = [len(p) for p in parents]
        if max(new) > 256 or any(not -1 <= up < i for p in parents for i, up in enumerate(p)):
            raise ValueError("a tree has at most 256 nodes, each behind its parent")
        bt = self.batch(new)
        tree = moe.Tree(bt, torch.tensor([up for p in parents for up in p], dtype=torch.int32).cuda())
        moe.moe_tree_prepare(bt, tree, err=self.ws.error_ptr)
        # those that nobody can accept any more and that hold up no request go
        self.trees = tuple(t for t in self.trees if any(t[1]) or t[0]() is not None) + ((weakref.ref(bt), new),)
        return bt, tree

    def accept(self, bt: moe.KvBatch, desc: moe.VerifyDesc, most: Optional[int] = None) -> Tuple[List[List[int]], List[int]]:
        """After forward() of tree_batch()'s trees, once: the nodes of each request that the target keeps (at most `most`),
        and its next token.  Keys and values of the others are gone, and the lengths of the trees' requests are those of
        what was kept.  A request that was released meanwhile keeps nothing."""
        mine = [nodes for batch, nodes in self.trees if batch() is bt]
        if not mine:
            raise ValueError("a batch of trees that has not been verified is wanted")
        most = max(bt.c.max_n, 1) if most is None else most
        if most < 1:
            raise ValueError("at least a tree's first node is kept")
        B, nodes = len(self.lens), mine[0]
        path = torch.empty(B, most, dtype=torch.int32, device="cuda")
        count, token = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
        moe.moe_verify_drafts(bt, desc, path, count, token, err=self.ws.error_ptr)
        if sum(nodes) < bt.c.T:  # the places of a released request may be another's by now
            here = torch.tensor([n > 0 for n in nodes]).cuda()
            count.masked_fill_(~here, 0)
            token.masked_fill_(~here, -1)
        moe.moe_kv_compact(self.kv_layers, bt, path, count, err=self.ws.error_ptr)
        kept = count.tolist()
        for r, n in enumerate(nodes):
            self.lens[r] -= n - kept[r]
        self.trees = tuple(t for t in self.trees if t[0]() is not bt)
        return [p[:n] for p, n in zip(path.tolist(), kept)], token.tolist()

    def fork(self, source: int, request: int) -> None:
        """Request `request`, which has no tokens, goes on from the tokens of `source`, whose tree if any is verified."""
        if self.lens[request]:
            raise ValueError(f"request {request} has tokens of its own")
        if self.open_tree(source):
            raise ValueError(f"the tree of request {source} has not been verified")
        self.pages.release(request)
        for a, z, n in self.pages.fork(source, request, self.lens[source]):
            i32 = lambda x: torch.tensor([x], dtype=torch.int32).cuda()  # noqa: E731
            moe.moe_kv_copy_pages(self.kv_layers, i32(a), i32(z), tokens=i32(n), err=self.ws.error_ptr)
        self.lens[request] = self.lens[source]

    def release(self, request: int) -> None:
        """The request has no tokens any more, nor a tree.  What forward() is still to run finds no pages of it."""
        self.pages.release(request)
        self.pages.upload()
        self.lens[request] = 0
        for _, nodes in self.trees:
            nodes[request] = 0

    def attention(self, l: int, xn: torch.Tensor, bt: moe.KvBatch, y: torch.Tensor, tree: Optional[moe.Tree] = None) -> None:
        """y = attention of layer l on the normalised rows xn, whose keys and values join the cache."""
        s, T = self.s, bt.c.T
        qkv = torch.matmul(xn, self.layers[l].qkv).view(T, s.Hq + 2 * s.Hkv, s.D)
        q, k, v = qkv.split([s.Hq, s.Hkv, s.Hkv], 1)
        if tree is None and self.norms[l] is None:
            moe.moe_kv_append(self.kv[l], bt, self.rope, q, self.q[:T], k, v, err=self.ws.error_ptr)
        else:
            moe.moe_kv_append_norm(self.kv[l], bt, self.rope, self.norms[l], q, self.q[:T], k, v, tree=tree, err=self.ws.error_ptr)
        if tree is None:
            moe.moe_paged_attention(self.kv[l], bt, self.q[:T], self.o[:T], self.ws, scale=s.D ** -0.5, window=s.window)
        else:
            moe.moe_tree_attention(self.kv[l], bt, tree, self.q[:T], self.o[:T], self.ws, scale=s.D ** -0.5, window=s.window)
        torch.matmul(self.o[:T].view(T, s.Hq * s.D), self.layers[l].out, out=y)

    def forward(self, x_res: torch.Tensor, bt: moe.KvBatch, tree: Optional[moe.Tree] = None) -> torch.Tensor:
        """All layers on the residual rows x_res (fp32 [T, H], updated in place); the normalised rows."""
        T, H = bt.c.T, self.H
        xn, y = self.xn[:T], self.y[:T]
        prev = None  # output of the block before, added by the next norm
        for l, a in enumerate(self.layers):
            moe.moe_block_norm(moe.block_norm_desc(y=prev, w_pre=a.norm_in, eps=self.eps), x_res, x_res, xn, T, H)
            self.attention(l, xn, bt, y, tree)
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
    d = Decoder(w, s, requests=1, max_len=prompt + 16 * (steps + 2), maxT=prompt)
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
    parents = [[-1, 0, 0, 0, 1, 1, 2, 4]]
    vocabulary = torch.randn(d.H, 32000, device="cuda") * d.H ** -0.5
    draws = [torch.rand(n, device="cuda") for n in (len(parents[0]), 1)]
    tokens = torch.randint(0, 32000, (len(parents[0]),), dtype=torch.int32, device="cuda")
    kept = 0
    ev2 = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for step in range(steps + 1):
        if step == 1:
            ev2[0].record()
        bt, tree = d.tree_batch(parents)
        xn = d.forward(x[:len(parents[0])].clone(), bt, tree)
        target = torch.softmax(xn.float() @ vocabulary, 1)
        paths, _ = d.accept(bt, moe.verify_desc(target, tokens, tree.parent, *draws))
        kept += len(paths[0])
    ev2[1].record()
    d.check()
    print(f"{d.st.L} layers, hidden {d.H}, {s.Hq} query and {s.Hkv} key heads of {s.D}: prompt of {prompt} tokens "
          f"{ev[0].elapsed_time(ev[1]):.2f} ms, a window of {window} {ev[2].elapsed_time(ev[3]) / steps * 1e3:.0f} us, "
          f"a tree of {len(parents[0])} with its verification {ev2[0].elapsed_time(ev2[1]) / steps * 1e3:.0f} us "
          f"({kept} tokens kept in {steps + 1})")


if __name__ == "__main__":
    main()

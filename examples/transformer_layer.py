#!/usr/bin/env python3
"""One rank's share of an MoE transformer layer, over prompts and then token by token.

Tensor parallel over W ranks with the token rows sharded between the products, expert parallel over the same ranks; this
process is one rank, and the peers' rows are simulated in its GPU's memory.

  prompt:  rms_norm -> AllGather + QKV product -> attn_prompt -> output product + ReduceScatter -> rms_norm with the
           residual -> router logits -> moe_gate -> AllToAll dispatch -> experts -> AllToAll combine
  tokens:  rms_norm with the residual -> QKV product -> append to the paged cache -> attn_decode, captured in one graph

    python examples/transformer_layer.py [--tokens 4096] [--hidden 1024] [--steps 64]
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import signal_gated_tiled_amd as sgt  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@dataclass
class Layer:
    """This rank's weights and the sizes of the layer."""
    W: int
    rank: int
    hidden: int
    Hq: int           # of this rank
    Hkv: int
    D: int
    experts: int
    topk: int
    norm1: torch.Tensor
    norm2: torch.Tensor
    qkv: torch.Tensor     # hidden x (Hq + 2 Hkv) D
    o: torch.Tensor       # Hq D x hidden
    router: torch.Tensor  # hidden x experts
    bias: torch.Tensor    # experts
    expert: torch.Tensor  # experts x hidden x hidden (all ranks' experts: the peers are simulated)


def make_layer(seed: int, W: int = 4, rank: int = 1, hidden: int = 512, Hq: int = 8, Hkv: int = 2, D: int = 64,
               experts: int = 16, topk: int = 4) -> Layer:
    g = torch.Generator().manual_seed(seed)

    def w(*shape, fan=None, dtype=BF16):
        return (torch.randn(*shape, generator=g) * ((fan or shape[0]) ** -0.5)).to(dtype).cuda()

    return Layer(W, rank, hidden, Hq, Hkv, D, experts, topk, (1 + 0.1 * torch.randn(hidden, generator=g)).to(BF16).cuda(),
                 (1 + 0.1 * torch.randn(hidden, generator=g)).to(BF16).cuda(), w(hidden, (Hq + 2 * Hkv) * D),
                 w(Hq * D, hidden), w(hidden, experts), (0.1 * torch.randn(experts, generator=g)).cuda(),
                 w(experts, hidden, hidden, fan=hidden))


def flags(n: int) -> torch.Tensor:
    return torch.zeros(n, dtype=I32, device="cuda")


def split_heads(L: Layer, qkv: torch.Tensor):
    """q, k and v of a QKV product's rows, as views."""
    x = qkv.view(-1, L.Hq + 2 * L.Hkv, L.D)
    return x[:, :L.Hq], x[:, L.Hq:L.Hq + L.Hkv], x[:, L.Hq + L.Hkv:]


def prompt(ctx: sgt.Context, L: Layer, x_shards, cu: torch.Tensor, partials):
    """The layer over packed prompts (offsets cu).  x_shards: every rank's rows of the residual stream; partials: what
    the peers' output products add to this rank's rows.  Returns what each step left."""
    W, T_r, H, r = L.W, x_shards[0].shape[0], L.hidden, L.rank
    T = W * T_r
    normed = [torch.empty_like(x) for x in x_shards]
    for x, y in zip(x_shards, normed):   # (each rank its own rows)
        sgt.rms_norm(x, L.norm1, y)
    gathered = torch.empty(T, H, dtype=BF16, device="cuda")
    qkv = torch.empty(T, L.qkv.shape[1], dtype=BF16, device="cuda")
    ctx.ag_gemm(normed, L.qkv, gathered, qkv, flags(sgt.ag_flag_count(W, T, H)), rank=r, out_dtype=sgt.SGT_BF16)

    q, k, v = split_heads(L, qkv)
    attn = torch.empty(T, L.Hq, L.D, dtype=BF16, device="cuda")
    sgt.attn_prompt(q, k, v, attn, cu, cu)

    tile = min(T_r & -T_r, 128)   # the ReduceScatter's signal tiles have to fit the rank's rows
    ng, npf = sgt.rs_flag_count(W, T, H, rs_tile=tile)
    summed = torch.empty(T_r, H, device="cuda")
    ctx.gemm_rs(attn.view(T, -1), L.o, [None if p == r else partials[p] for p in range(W)],
                torch.empty(T, H, device="cuda"), summed, flags(ng), flags(npf), rank=r, rs_tile=tile)

    stream, rows = torch.empty_like(x_shards[r]), torch.empty_like(x_shards[r])
    sgt.rms_norm(summed, L.norm2, rows, residual=x_shards[r], sum_out=stream)

    # every rank routes its own rows; the peers' stand in here with their normed inputs
    all_rows = [rows if p == r else normed[p] for p in range(W)]
    ids = [torch.empty(T_r, L.topk, dtype=I32, device="cuda") for _ in range(W)]
    gate = [torch.empty(T_r, L.topk, device="cuda") for _ in range(W)]
    logits = [x.float() @ L.router.float() for x in all_rows]
    for p in range(W):
        sgt.moe_gate(logits[p], ids[p], gate[p], score="sigmoid", bias=L.bias, n_group=4, topk_group=2, scale=2.0)

    E_r = L.experts // W
    nf = sgt.a2a_flag_count(W, T_r, L.experts)
    back = []
    for p in range(W):   # rank p's experts: what is dispatched to them, and their answers to this rank
        recv = torch.zeros(E_r, W, T_r, H, dtype=BF16, device="cuda")
        ctx.a2a_dispatch(all_rows, ids, recv, torch.empty(E_r, W, T_r, dtype=I32, device="cuda"),
                         torch.zeros(E_r, W, dtype=torch.int64, device="cuda"), flags(nf), L.experts, rank=p)
        back.append(torch.stack([recv[e, r] @ L.expert[p * E_r + e] for e in range(E_r)]))
    moe = torch.empty(T_r, H, device="cuda")
    ctx.a2a_combine(back, ids[r], gate[r], torch.empty(L.experts, T_r, H, dtype=BF16, device="cuda"),
                    torch.empty(T_r, L.topk, dtype=I32, device="cuda"), moe, flags(nf), W, rank=r)
    ctx.sync()
    return dict(normed=normed[r], qkv=qkv, attn=attn, summed=summed, stream=stream, rows=rows, logits=logits[r],
                ids=ids[r], gate=gate[r], moe=moe)


class Tokens:
    """This rank's attention of new tokens over a paged cache: one step per call, as a captured graph."""

    def __init__(self, L: Layer, qkv: torch.Tensor, lens, steps: int, page: int = 16):
        B = len(lens)
        self.L, self.page = L, page
        per = -(-(max(lens) + steps) // page)
        order = torch.randperm(B * per, generator=torch.Generator().manual_seed(5))
        self.table = order.to(I32).view(B, per).cuda()
        self.k = torch.zeros(B * per, page, L.Hkv, L.D, dtype=BF16, device="cuda")
        self.v = torch.zeros_like(self.k)
        _, k, v = split_heads(L, qkv)
        at = 0
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            pages = self.table[b, j // page].long()
            self.k[pages, j % page], self.v[pages, j % page] = k[at:at + n], v[at:at + n]
            at += n
        self.lens = torch.tensor(lens, dtype=I32, device="cuda")
        self.x, self.add = (torch.zeros(B, L.hidden, dtype=BF16, device="cuda") for _ in range(2))
        self.row, self.qkv = torch.zeros_like(self.x), torch.zeros(B, L.qkv.shape[1], dtype=BF16, device="cuda")
        self.out = torch.zeros(B, L.Hq, L.D, dtype=BF16, device="cuda")
        self.lse = torch.zeros(B, L.Hq, device="cuda")
        self.work = torch.zeros(sgt.attn_decode_workspace(B, L.Hq, L.Hkv, L.D), dtype=torch.uint8, device="cuda")
        self.graph = None

    def step(self):
        """The residual stream's rows x, to which `add` is added first; out: the attention of the tokens' heads."""
        L = self.L
        sgt.rms_norm(self.x, L.norm1, self.row, residual=self.add, sum_out=self.add)
        torch.mm(self.row, L.qkv, out=self.qkv)
        q, k, v = split_heads(L, self.qkv)
        at = self.lens.long()
        pages = self.table.gather(1, (at // self.page)[:, None])[:, 0].long()
        self.k[pages, at % self.page], self.v[pages, at % self.page] = k, v
        self.lens += 1
        sgt.attn_decode(q, self.k, self.v, self.table, self.lens, self.out, self.work, lse=self.lse)

    def replay(self):
        """The same step from a graph, captured on the first call."""
        if self.graph is None:
            state = [t.clone() for t in (self.k, self.v, self.lens, self.add)]
            self.step()   # once outside the graph, so that libraries set themselves up, and taken back
            for t, s in zip((self.k, self.v, self.lens, self.add), state):
                t.copy_(s)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.step()
        self.graph.replay()


def inputs(L: Layer, lens, seed: int):
    """Every rank's rows of the residual stream, the prompts' offsets, the peers' partial sums."""
    T = sum(lens)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, L.hidden, generator=g).to(BF16).cuda()
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=I32, device="cuda")
    partials = [torch.randn(T // L.W, L.hidden, generator=g).cuda() for _ in range(L.W)]
    return list(x.view(L.W, T // L.W, L.hidden)), cu, partials


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    L = make_layer(1, hidden=a.hidden, Hq=8, Hkv=1, D=128, experts=64, topk=8)
    T = max(a.tokens // (128 * L.W), 1) * 128 * L.W
    lens = [T // 2, T // 4, T // 8 + 1, T - T // 2 - T // 4 - T // 8 - 1]
    x, cu, partials = inputs(L, lens, 2)
    with sgt.Context(0) as ctx:
        for i in range(3):
            torch.cuda.synchronize()
            t = time.perf_counter()
            got = prompt(ctx, L, x, cu, partials)
            torch.cuda.synchronize()
            t = time.perf_counter() - t
        print("prompts of %s tokens: one rank's share of the layer (and its peers' norms, gates and experts) in %.2f ms"
              % (lens, t * 1e3), flush=True)
    tok = Tokens(L, got["qkv"], lens, a.steps + 2)
    tok.x.normal_()
    tok.replay()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        tok.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    print("%d tokens at a time behind them: %.1f us a step" % (len(lens), t * 1e6), flush=True)


if __name__ == "__main__":
    main()

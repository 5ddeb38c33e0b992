"""The layer operators together, as a program uses them.

decode: one attention + expert block of a token-by-token step over NVFP4
weights and a paged NVFP4 cache, captured in a graph and replayed.
train:  one step of a routed linear layer in MXFP8, forward and backward:
route, grouped product, combine, and the gradients of the tokens, the experts'
weights and the router's logits.

    python examples/moe_block.py [--seqs 8] [--context 4096] [--steps 16] [--tokens 4096]
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import nvfp4_block_scaled_amax_amd as mxq                # noqa: E402
from nvfp4_block_scaled_amax_amd import api             # noqa: E402


class Shape(NamedTuple):
    hidden: int = 2048
    inter: int = 768
    experts: int = 128
    top_k: int = 8
    heads: int = 32
    kv_heads: int = 4
    head_dim: int = 128
    page: int = 64


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class DecodeBlock:
    """Weights in NVFP4, and the caches and page table of n_seqs sequences that
    hold `context` positions each so far and at most max_len."""

    def __init__(self, s: Shape, n_seqs: int, context: int, max_len: int, seed: int = 0):
        self.s = s
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, device="cuda", generator=g) * std).bfloat16()

        qkv = (s.heads + 2 * s.kv_heads) * s.head_dim
        self.w_qkv = api.nvfp4_quantize_per_tensor(normal(qkv, s.hidden, std=s.hidden ** -0.5))
        self.w_out = api.nvfp4_quantize_per_tensor(
            normal(s.hidden, s.heads * s.head_dim, std=(s.heads * s.head_dim) ** -0.5))
        self.w_router = api.nvfp4_quantize_per_tensor(
            normal(s.experts, s.hidden, std=s.hidden ** -0.5))
        self.gateup = api.nvfp4_quantize_gateup_pair(
            normal(s.experts, s.inter, s.hidden, std=s.hidden ** -0.5),
            normal(s.experts, s.inter, s.hidden, std=s.hidden ** -0.5))
        self.down = api.nvfp4_quantize_gateup_pair(
            normal(s.experts, s.hidden, s.inter, std=s.inter ** -0.5))

        # Every sequence's pages, in an order that is not the table's.
        per_seq = -(-max_len // s.page)
        n_pages = n_seqs * per_seq
        self.table = torch.randperm(n_pages, device="cuda", generator=g).view(n_seqs, per_seq)
        self.lens = torch.full((n_seqs,), context, dtype=torch.int64, device="cuda")
        self.cache = [self._empty_cache(n_pages) for _ in "kv"]
        pos = torch.arange(context, device="cuda").repeat(n_seqs, 1)
        rows = self._rows(pos).view(-1, s.kv_heads)
        for c in self.cache:                   # what earlier steps would have appended
            api.nvfp4_cache_append(normal(n_seqs * context, s.kv_heads, s.head_dim, std=1.0),
                                   rows, c)

    def _empty_cache(self, n_pages):
        s, n = self.s, n_pages * self.s.kv_heads * self.s.page
        return api.NVFP4(torch.zeros(n, s.head_dim // 2, dtype=torch.uint8, device="cuda"),
                         torch.zeros(n, s.head_dim // 16, dtype=torch.uint8, device="cuda"),
                         torch.zeros(n, device="cuda"))

    def _rows(self, pos):
        """Cache rows of positions pos [n_seqs][n] of every sequence."""
        pages = self.table.gather(1, pos // self.s.page)
        return api.nvfp4_cache_rows(pages.view(-1), (pos % self.s.page).view(-1),
                                    self.s.kv_heads, self.s.page)

    def step(self, x):
        """x [n_seqs][hidden] BF16 -> (the block's output, what it passed between
        its operators).  Appends one position to every sequence."""
        s, n = self.s, x.shape[0]
        h = norm(x)
        qkv = api.nvfp4_matvec(h, *self.w_qkv).view(n, -1, s.head_dim)
        q, k, v = (t.contiguous() for t in qkv.split([s.heads, s.kv_heads, s.kv_heads], 1))
        rows = self._rows(self.lens[:, None])
        api.nvfp4_cache_append(k, rows, self.cache[0])
        api.nvfp4_cache_append(v, rows, self.cache[1])
        self.lens += 1
        att = api.nvfp4_attention(q[:, None], *self.cache, self.table, self.lens, s.kv_heads,
                                  s.page).out
        x = x + api.nvfp4_matvec(att.view(n, -1), *self.w_out)
        h2 = norm(x)
        logits = api.nvfp4_matvec(h2, *self.w_router, out_dtype=torch.float32)
        routing = api.moe_route(logits, s.top_k)
        y = api.nvfp4_expert_layer(h2, routing, self.gateup, self.down)
        return x + y, dict(q=q, k=k, v=v, rows=rows, att=att, h2=h2, logits=logits,
                           routing=routing, y=y)


class TrainStep(NamedTuple):
    out: torch.Tensor            # [T][N]
    d_tokens: torch.Tensor       # [T][K]
    d_experts: torch.Tensor      # [E][N][K] FP32
    d_logits: torch.Tensor       # [T][E]


def _mxfp8_weight(w):
    """[E][N][K] BF16 -> rowwise MXFP8 codes and scales."""
    E, N, K = w.shape
    q = api.mxfp8_quantize_rowcol(w.reshape(E * N, K), colwise=False)
    return q.row_codes.view(E, N, K), q.row_scales.view(E, N, K // 32)


def train_step(tokens, logits, weights, d_out, top_k) -> TrainStep:
    """out[t] = sum_c w[t][c] W_e tokens[t] over the top_k experts e that logits
    choose, in MXFP8 with BF16 results, and its gradients under d_out."""
    r = api.moe_route(logits, top_k)
    x = tokens[r.row_tokens]
    xc, xs, x_t = api.mxfp8_grouped_quantize_rowcol_t(x, r.seg_offsets)
    y = api.mxfp8_grouped_gemm(xc, xs, *_mxfp8_weight(weights), r.seg_offsets)
    out = api.moe_combine(y, r.token_rows, r.weights)

    d_y, d_w = api.moe_combine_backward(d_out, y, r.token_rows, r.weights, r.seg_offsets)
    dc, ds, d_t = api.mxfp8_grouped_quantize_rowcol_t(d_y, r.seg_offsets)
    d_x = api.mxfp8_grouped_gemm(dc, ds, *_mxfp8_weight(weights.transpose(1, 2).contiguous()),
                                 r.seg_offsets)
    # Every copy of a token adds to its gradient: the return with weights of one.
    d_tokens = api.moe_combine(d_x, r.token_rows, torch.ones_like(r.weights))
    d_experts = api.mxfp8_grouped_wgrad(d_t, x_t)
    return TrainStep(out, d_tokens, d_experts, api.moe_route_backward(d_w, logits, r.experts))


def timed(run, n):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    run()
    start.record()
    for _ in range(n):
        run()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / n


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--seqs", type=int, default=8)
    p.add_argument("--context", type=int, default=4096)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--tokens", type=int, default=4096)
    a = p.parse_args()
    mxq.lib()
    s = Shape()

    block = DecodeBlock(s, a.seqs, a.context, a.context + 2 * a.steps + 8)
    x = torch.randn(a.seqs, s.hidden, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):              # the allocator's and the library's first calls
        block.step(x)
    torch.cuda.current_stream().wait_stream(side)
    eager = timed(lambda: block.step(x), 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.step(x)
    ms = timed(graph.replay, a.steps)
    print(f"decode: {a.seqs} sequences of {int(block.lens[0])} positions, {ms * 1e3:.0f} us a step "
          f"in a graph ({eager * 1e3:.0f} us eager), output rms {out.float().square().mean().sqrt():.3f}")

    tokens = torch.randn(a.tokens, s.hidden, device="cuda").bfloat16()
    logits = torch.randn(a.tokens, s.experts, device="cuda").bfloat16()
    w = (torch.randn(s.experts, s.inter, s.hidden, device="cuda") * s.hidden ** -0.5).bfloat16()
    d_out = torch.randn(a.tokens, s.inter, device="cuda").bfloat16()
    ms = timed(lambda: train_step(tokens, logits, w, d_out, s.top_k), 4)
    print(f"train: {a.tokens} tokens, {ms * 1e3:.0f} us a step (forward and backward)")


if __name__ == "__main__":
    main()

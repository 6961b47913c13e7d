"""An attention block in 4 bits, as a serving loop runs it on one MI355X.

    python examples/w4a8kv4_attention.py [--steps 32]

Prompts of different lengths enter the cache in one call, then every sequence gets one
token a step. Each call of ``AttentionBlock`` is the pre-norm block

    h   = x + residual                     add_rmsnorm_int8: the sum, the norm and the 8-bit
    a   = int8(norm(h))                    activations in one pass
    qkv = a Wqkv^T                         linear_w4a8_quantized: 4-bit weights
    cache <- k, v                          kv4_append: the projection's slices, 4 bits each
    o   = attention(q, cache)              kv4_attention: prompts, single tokens and mixtures
    out = o Wo^T                           linear: 4-bit weights, 16-bit activations

and returns ``(out, h)``, the next block's x and residual. (Positions are left out: nothing
here rotates queries and keys.) The decode step is also captured in a graph and replayed.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import quantized_gemm_rtn_amd as wq  # noqa: E402


def quantized(N, K, gen, device):
    """A random layer in 4 bits: packed codes, scales, zero-points."""
    w = torch.randn(N, K, device=device, generator=gen) / K ** 0.5
    q = wq.quantize_rtn(w)
    return wq.pack(q["codes"]), q["scales"].contiguous(), q["zeros"].contiguous()


class AttentionBlock:
    """One block's weights; its cache is the caller's, and so are the batch's arrays."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, outliers=8, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.norm = (1 + 0.1 * torch.randn(hidden, device=device, generator=gen)).half()
        # the channels that the activations' calibration found largest
        self.outliers = torch.randperm(hidden, device=device, generator=gen)[:outliers].sort().values.int()
        self.qkv = quantized((q_heads + 2 * kv_heads) * head_dim, hidden, gen, device)
        self.o = quantized(hidden, q_heads * head_dim, gen, device)

    def project(self, x, residual):
        """(q, k, v, h) of tokens x [T, hidden]; q, k and v are slices of one tensor."""
        xq, sx, xo, h = wq.add_rmsnorm_int8(x, self.norm, residual, outliers=self.outliers)
        qkv = wq.linear_w4a8_quantized(xq, sx, xo, self.outliers, *self.qkv)
        heads = qkv.view(x.shape[0], self.q_heads + 2 * self.kv_heads, self.head_dim)
        return *heads.split([self.q_heads, self.kv_heads, self.kv_heads], 1), h

    def __call__(self, x, residual, cache, page_table, seq_start, ctx_len, max_q, max_ctx):
        q, k, v, h = self.project(x, residual)
        wq.kv4_append(k, v, cache, page_table, seq_start, ctx_len, max_new=max_q)
        o = wq.kv4_attention(q, cache, page_table, seq_start, ctx_len, max_q=max_q, max_ctx=max_ctx)
        return wq.linear(o.view(x.shape[0], -1), *self.o), h


def captured(fn):
    """``fn`` in a graph; returns the graph and fn's outputs, which each replay rewrites."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()  # sizes the allocator's pool before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    return graph, out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=32)
    steps = ap.parse_args().steps
    hidden, q_heads, kv_heads, head_dim, page = 4096, 32, 8, 128, 64
    lengths = [1500, 37, 800, 1, 2048, 300, 64, 1021]
    B, T = len(lengths), sum(lengths)
    block = AttentionBlock(hidden, q_heads, kv_heads, head_dim)
    pages = -(-(max(lengths) + steps) // page)
    cache = wq.kv4_cache(B * pages, page, kv_heads, head_dim)
    page_table = torch.randperm(B * pages, device="cuda").int().view(B, pages)
    ctx_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")

    x, residual = torch.randn(T, hidden, device="cuda").half(), torch.randn(T, hidden, device="cuda").half()
    for name in ("first call", "prompts"):
        torch.cuda.synchronize()
        begin = time.perf_counter()
        out, h = block(x, residual, cache, page_table, starts, ctx_len, max(lengths), max(lengths))
        torch.cuda.synchronize()
        print(f"{name}: {T} tokens of {B} sequences, {(time.perf_counter() - begin) * 1e3:.2f} ms")

    # one token a sequence: the block's outputs of the last tokens go in again
    last = starts[1:].long() - 1
    x, residual = out[last].contiguous(), h[last].contiguous()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def step():
        ctx_len.add_(1)
        out, h = block(x, residual, cache, page_table, one, ctx_len, 1, pages * page)
        x.copy_(out)
        residual.copy_(h)
        return x

    start_len = ctx_len.clone()
    graph, _ = captured(step)
    ctx_len.copy_(start_len)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    print(f"decode: {steps} steps of {B} tokens, {(time.perf_counter() - begin) / steps * 1e6:.1f} us a step; "
          f"finite: {bool(torch.isfinite(x).all())}")
    per_token = kv_heads * wq.kv4_page_bytes(page, head_dim) // page
    print(f"cache: {per_token} bytes a token, {4 * kv_heads * head_dim} in 16 bits")


if __name__ == "__main__":
    main()

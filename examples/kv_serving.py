"""A serving loop over the 8-bit key/value cache: one attention layer, its projections as MXFP8 products.

Every step gives the requests their cache blocks and the new tokens their places (kv_block_tables),
projects the tokens' hidden states to queries, keys and values with one MXFP8 GEMM, writes the keys and
values into the cache (kv_cache_append), attends over it (kv_attention) and projects the result back.
Weights and hidden states are random; requests start with a prompt, go on token by token and leave.

  python examples/kv_serving.py [--requests 16] [--prompt 1000] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_mx_gb300 as mx  # noqa: E402


class Layer:
    """Attention of `heads` query and `kv_heads` key/value heads on hidden states of `hidden` values, with
    a cache of `blocks` blocks for up to `requests` requests of `longest` tokens."""

    def __init__(self, hidden, heads, kv_heads, head_dim, blocks, block_tokens, requests, longest, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def weight(n, k):  # quantized once, as the B operand of a product
            w = (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(torch.bfloat16)
            return mx.mx_quantize(w, layout=mx.ROWWISE)[:2]
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.block_tokens = hidden, heads, kv_heads, head_dim, block_tokens
        self.qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, heads * head_dim)
        cache = (blocks, kv_heads, block_tokens, head_dim)
        self.codes = [torch.empty(cache, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scale = [torch.empty(cache[:2], device="cuda") for _ in range(2)]
        self.tables = torch.full((requests, -(-longest // block_tokens)), -1, dtype=torch.int32, device="cuda")
        self.free = torch.arange(blocks, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), blocks, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def project(self, x, weight, n):
        """x [tokens][k] times a quantized weight [n][k]; the products take rows in 128s."""
        tokens, k = x.shape
        rows = -(-tokens // 128) * 128
        if rows != tokens:
            x = torch.cat([x, x.new_zeros(rows - tokens, k)])
        q, s, _, _ = mx.mx_quantize(x.contiguous(), layout=mx.ROWWISE)
        return mx.mx_gemm(q, s, mx.E4M3, *weight, mx.E4M3, rows, n, k)[:tokens]

    def leave(self):
        """All requests leave, and give their blocks back."""
        after = torch.zeros_like(self.lengths)
        self.free_count = mx.kv_block_tables(self.tables, self.lengths, after, self.free, self.free_count, 0,
                                             self.block_tokens)[3][:1]
        self.lengths = after

    def step(self, x, after, most_new):
        """Hidden states x of the new tokens, the requests' lengths with them (int32, on the device), and the
        most new tokens of a request.  Returns (queries, attention's result, its lse, the layer's result);
        raises, with everything as it was, if the cache has too few blocks."""
        q_start, slots, positions, info = mx.kv_block_tables(
            self.tables, self.lengths, after, self.free, self.free_count, x.shape[0], self.block_tokens)
        qkv = self.project(x, self.qkv, (self.heads + 2 * self.kv_heads) * self.head_dim)
        if int(info[1]):  # (read here, while the projection runs)
            raise RuntimeError(f"{int(info[1])} cache blocks are missing: nothing was moved, the step cannot go on")
        q, k, v = qkv.view(x.shape[0], -1, self.head_dim).split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        mx.kv_cache_append(k, v, slots, *self.codes, *self.scale)
        out, lse = mx.kv_attention(q, *self.codes, *self.scale, self.tables, after, q_start, most_new)
        self.lengths, self.free_count = after, info[:1]
        return q, out, lse, self.project(out.view(x.shape[0], -1), self.out, self.hidden)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000, help="the longest prompt; the others are shorter")
    ap.add_argument("--steps", type=int, default=32, help="single-token steps after the prompts")
    a = ap.parse_args(argv)
    n, longest = a.requests, a.prompt + a.steps
    blocks = n * -(-longest // 64)
    layer = Layer(4096, 32, 8, 128, blocks, 64, n, longest)
    gen = torch.Generator("cuda").manual_seed(1)
    prompts = [max(1, a.prompt * (i + 1) // n) for i in range(n)]

    def hidden(tokens):
        return torch.randn(tokens, 4096, generator=gen, device="cuda").to(torch.bfloat16)
    layer.step(hidden(sum(prompts)), torch.tensor(prompts, dtype=torch.int32, device="cuda"), max(prompts))
    x = hidden(n)
    for _ in range(2):  # (the first single-token step loads its kernels)
        torch.cuda.synchronize()
        began = time.perf_counter()
        for _ in range(a.steps // 2):
            x = layer.step(x, layer.lengths + 1, 1)[3]
        torch.cuda.synchronize()
        spent = time.perf_counter() - began
    held = sum(-(-(p + 2 * (a.steps // 2)) // 64) for p in prompts)
    left = int(layer.free_count)
    layer.leave()
    assert mx.mx_check() == mx.MX_OK
    assert left == blocks - held and int(layer.free_count) == blocks and bool(torch.isfinite(x).all())
    print("%d requests, prompts of %d to %d tokens: %.1f us a single-token step of the layer, %d of %d blocks held"
          % (n, min(prompts), max(prompts), 1e6 * spent / max(1, a.steps // 2), held, blocks))


if __name__ == "__main__":
    main()

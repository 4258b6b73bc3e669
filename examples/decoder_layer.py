"""One decoder layer that serves requests of any length from a cache of 8-bit blocks: prompts and
single tokens in one ragged batch.  lora_linear, qk_norm_rope, kv_cache_write, cache_attention,
and linear with the residual for the output projection and the MLP.

    python examples/decoder_layer.py [--requests 16] [--prompt 300] [--steps 32] [--codes e4m3]

reads the prompts, then decodes: a step for all requests, captured into a graph, and prints what a
step takes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import direct_implicit_gemm_amd as L  # noqa: E402


class DecoderLayer:
    """Weights, and the cache of `blocks` blocks of `block` tokens that all requests share.

    channels in and out, q_heads query heads over k_heads key heads of head_dim, an MLP of `inner`
    values; each request has room for `room` tokens (its row of the table)."""

    def __init__(self, channels, q_heads, k_heads, head_dim, inner, requests, room, block=32,
                 codes=torch.float8_e4m3fn, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, by):
            return (torch.randn(*shape, generator=g) * by).to(dtype).cuda()

        self.q_heads, self.k_heads, self.head_dim = q_heads, k_heads, head_dim
        heads = (q_heads + 2 * k_heads) * head_dim
        self.w_qkv, self.b_qkv = normal(heads, channels, by=channels ** -0.5), normal(heads, by=0.05)
        self.w_out = normal(channels, q_heads * head_dim, by=(q_heads * head_dim) ** -0.5)
        self.w_up, self.b_up = normal(inner, channels, by=channels ** -0.5), normal(inner, by=0.05)
        self.w_down = normal(channels, inner, by=inner ** -0.5)
        self.q_norm = (1 + normal(head_dim, by=0.2).float()).to(dtype)
        self.k_norm = (1 + normal(head_dim, by=0.2).float()).to(dtype)
        self.freqs = L.rotary_frequencies(head_dim)
        # blocks of a request lie anywhere; a block's heads each have their tokens side by side
        width = -(-room // block)
        blocks = requests * width
        shape = (blocks, k_heads, block, head_dim)
        self.k_cache = torch.zeros(shape, dtype=codes, device="cuda").transpose(1, 2)
        self.v_cache = torch.zeros(shape, dtype=codes, device="cuda").transpose(1, 2)
        self.k_scale = torch.zeros(blocks, k_heads, device="cuda")
        self.v_scale = torch.zeros(blocks, k_heads, device="cuda")
        self.table = torch.randperm(blocks, generator=g).view(requests, width).int().cuda()

    def __call__(self, x, starts, lengths, positions, max_rows):
        """x [T, channels]: the next tokens of every request (rows starts[r] .. starts[r + 1] - 1,
        at `positions`), which has lengths[r] tokens with them."""
        d, hq, hk = self.head_dim, self.q_heads, self.k_heads
        qkv = L.lora_linear(x, self.w_qkv, self.b_qkv, None, None, None, None, None)
        q, k, v = (p.view(len(x), -1, d) for p in qkv.split([hq * d, hk * d, hk * d], 1))
        q, k = L.qk_norm_rope(q, k, positions, self.freqs, self.q_norm, self.k_norm)
        cache = (self.k_cache, self.v_cache, self.k_scale, self.v_scale)
        L.kv_cache_write(k, v, *cache, starts, lengths, self.table)
        out = L.cache_attention(q, *cache, starts, lengths, self.table, max_rows=max_rows)
        x = L.linear(out.view(len(x), hq * d), self.w_out, residual=x)
        up = L.linear(x, self.w_up, self.b_up, act="gelu_tanh")
        return L.linear(up, self.w_down, residual=x)


def positions_of(starts, lengths, T):
    """Where each row stands in its request."""
    row = torch.arange(T, dtype=torch.int32, device="cuda")
    entry = torch.searchsorted(starts, row, right=True) - 1
    return (lengths[entry] - starts[entry + 1] + row).int()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=16)
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--channels", type=int, default=1280)
    p.add_argument("--codes", choices=["e4m3", "i8"], default="e4m3")
    p.add_argument("--dtype", choices=["bf16", "f16", "f32"], default="bf16")
    o = p.parse_args()
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[o.dtype]
    codes = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}[o.codes]
    layer = DecoderLayer(o.channels, o.channels // 64, max(1, o.channels // 256), 64, 4 * o.channels,
                         o.requests, o.prompt + o.steps + 8, codes=codes, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(1)

    def tokens(n):
        return torch.randn(n, o.channels, device="cuda", generator=g).to(dtype)

    # prompts of different lengths, read in at once
    rows = torch.linspace(max(1, o.prompt // 3), o.prompt, o.requests).int()
    starts = torch.cat([torch.zeros(1), rows.cumsum(0)]).int().cuda()
    lengths = rows.cuda()
    T = int(rows.sum())
    layer(tokens(T), starts, lengths, positions_of(starts, lengths, T), int(rows.max()))
    # then a token of each at a time
    starts = torch.arange(o.requests + 1, dtype=torch.int32, device="cuda")
    x = tokens(o.requests)

    def step():
        lengths.add_(1)
        return layer(x, starts, lengths, lengths - 1, 1)

    step()                                  # outside the graph, first
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(o.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 1e3 / o.steps
    print(f"{o.requests} requests of up to {o.prompt} tokens, {o.channels} channels {o.dtype}, cache "
          f"in {o.codes}: {us:.1f} us a step, {o.requests * 1e6 / us:.0f} tokens/s of one layer, "
          f"|y| {float(y.float().abs().mean()):.3f}")


if __name__ == "__main__":
    main()

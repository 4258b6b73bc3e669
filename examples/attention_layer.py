"""One attention layer that serves many prompts behind a shared prefix, with each request's
adapter: lora_linear, qk_norm_rope, prefix_attention, lora_linear.

    python examples/attention_layer.py [--requests 8] [--prefix 960] [--steps 32] [--dtype bf16]

reads the prefix once, then the prompts, then decodes: a step for all requests is four calls of
the library (seven kernels, captured into a graph), and prints what a step takes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import direct_implicit_gemm_amd as L  # noqa: E402


class AttentionLayer:
    """Weights, adapters, and the keys and values seen so far.

    channels in and out, q_heads query heads over k_heads key heads of head_dim; n_adapters of
    `rank` for both projections (requests choose one, or -1); room for `prefix` shared keys and
    `room` own keys of each of `requests` requests."""

    def __init__(self, channels, q_heads, k_heads, head_dim, n_adapters, rank, requests, prefix,
                 room, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, by):
            return (torch.randn(*shape, generator=g) * by).to(dtype).cuda()

        self.q_heads, self.k_heads, self.head_dim = q_heads, k_heads, head_dim
        self.requests, self.room = requests, room
        inner, outer = q_heads * head_dim, (q_heads + 2 * k_heads) * head_dim
        self.w_qkv = normal(outer, channels, by=channels ** -0.5)
        self.b_qkv = normal(outer, by=0.05)
        self.w_out = normal(channels, inner, by=inner ** -0.5)
        self.a_qkv = normal(n_adapters, rank, channels, by=channels ** -0.5)
        self.up_qkv = normal(n_adapters, outer, rank, by=0.3 * rank ** -0.5)
        self.a_out = normal(n_adapters, rank, inner, by=inner ** -0.5)
        self.up_out = normal(n_adapters, channels, rank, by=0.3 * rank ** -0.5)
        self.scales = (0.5 + torch.rand(n_adapters, generator=g)).cuda()
        self.q_norm = (1 + normal(head_dim, by=0.2).float()).to(dtype)
        self.k_norm = (1 + normal(head_dim, by=0.2).float()).to(dtype)
        self.freqs = L.rotary_frequencies(head_dim)
        # keys and values lie one request after another; the prefix in a cache of its own
        self.prefix_k = torch.zeros(prefix, k_heads, head_dim, dtype=dtype, device="cuda")
        self.prefix_v = torch.zeros_like(self.prefix_k)
        self.keys = torch.zeros(requests, room, k_heads, head_dim, dtype=dtype, device="cuda")
        self.values = torch.zeros_like(self.keys)

    def _project(self, x, w, bias, a, up, starts, adapters):
        return L.lora_linear(x, w, bias, a, up, self.scales, starts, adapters)

    def _attend(self, x, positions, slots, keys, values, attention, starts, adapters):
        """x [T, channels] at `positions`, whose keys and values go to rows `slots`."""
        d, hq, hk = self.head_dim, self.q_heads, self.k_heads
        qkv = self._project(x, self.w_qkv, self.b_qkv, self.a_qkv, self.up_qkv, starts, adapters)
        q, k, v = (p.view(len(x), -1, d) for p in qkv.split([hq * d, hk * d, hk * d], 1))
        q, _, _ = L.qk_norm_rope(q, k, positions, self.freqs, self.q_norm, self.k_norm, v=v,
                                 slots=slots, k_out=keys.view(-1, hk, d),
                                 v_out=values.view(-1, hk, d))
        out = attention(q)
        return self._project(out.reshape(len(x), hq * d), self.w_out, None, self.a_out,
                             self.up_out, starts, adapters)

    def read_prefix(self, x):
        """x [prefix, channels], the shared tokens: they have no adapter."""
        n = len(x)
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        none = torch.tensor([-1], dtype=torch.int32, device="cuda")
        length = torch.tensor([n], dtype=torch.int32, device="cuda")
        return self._attend(
            x, at, at, self.prefix_k, self.prefix_v,
            lambda q: L.prefix_attention(q[None], None, None, self.prefix_k[None],
                                         self.prefix_v[None], length), starts, none)

    def read(self, x, first, adapters):
        """x [requests, n, channels]: the next n tokens of every request, which has `first`
        (int32 [requests], device) of its own already.  adapters: int32 [requests]."""
        B, n, _ = x.shape
        step = torch.arange(n, dtype=torch.int32, device="cuda")
        own = first[:, None] + step
        slots = own + self.room * torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
        positions = len(self.prefix_k) + own
        starts = n * torch.arange(B + 1, dtype=torch.int32, device="cuda")
        lengths = first + n
        y = self._attend(
            x.reshape(B * n, -1), positions.reshape(-1), slots.reshape(-1), self.keys, self.values,
            lambda q: L.prefix_attention(q.view(B, n, self.q_heads, self.head_dim), self.prefix_k,
                                         self.prefix_v, self.keys, self.values, lengths),
            starts, adapters)
        return y.view(B, n, -1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--prefix", type=int, default=960)
    p.add_argument("--prompt", type=int, default=20)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--channels", type=int, default=1280)
    p.add_argument("--dtype", choices=["bf16", "f16", "f32"], default="bf16")
    o = p.parse_args()
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[o.dtype]
    layer = AttentionLayer(o.channels, o.channels // 64, o.channels // 64, 64, 4, 16, o.requests,
                           o.prefix, o.prompt + o.steps + 8, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)

    def tokens(*shape):
        return torch.randn(*shape, o.channels, device="cuda", generator=g).to(dtype)

    adapters = (torch.arange(o.requests, device="cuda") % 5 - 1).int()
    first = torch.zeros(o.requests, dtype=torch.int32, device="cuda")
    layer.read_prefix(tokens(o.prefix))
    layer.read(tokens(o.requests, o.prompt), first, adapters)
    first += o.prompt
    x = tokens(o.requests, 1)
    layer.read(x, first, adapters)          # a step outside the graph, first
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.read(x, first, adapters)
        first += 1
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(o.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 1e3 / o.steps
    print(f"{o.requests} requests behind {o.prefix} shared tokens, {o.channels} channels "
          f"{o.dtype}: {us:.1f} us a step, {o.requests * 1e6 / us:.0f} tokens/s of one layer, "
          f"|y| {float(y.float().abs().mean()):.3f}")


if __name__ == "__main__":
    main()

"""One decoder layer served from a paged cache: 4-bit projections around rotary positions, the cache
write and attention, with random weights.

    python examples/serve_layer.py

Admits requests of different lengths in chunks, then decodes token by token with the step captured
in a graph, and prints the time of each."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matmul_mlx_amd as qaff  # noqa: E402


class Layer:
    """Attention and feed-forward weights, quantized to 4 bits in groups of 64."""

    def __init__(self, width, heads, kv_heads, dim, hidden, gen, dtype=torch.bfloat16):
        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5
            return qaff.QWeight(*qaff.quantize(w.to(dtype), 64, 4), 4, 64)

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv = weight((heads + 2 * kv_heads) * dim, width)
        self.o = weight(width, heads * dim)
        self.gate, self.up, self.down = weight(hidden, width), weight(hidden, width), weight(width, hidden)
        self.inv_freq = (10000.0 ** (-torch.arange(0, dim, 2, device="cuda") / dim)).float()

    def __call__(self, x, plan, cache, max_new):
        """x [tokens, width] of a step's new tokens, whose keys and values join the cache."""
        h, kv = self.heads, self.kv_heads
        qkv = self.qkv.mm(_norm(x)).view(-1, h + 2 * kv, self.dim)
        q = qaff.rope_append(qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:], plan.positions, self.inv_freq, plan.slots,
                             cache.k, cache.v)
        o = qaff.paged_attention(q, cache.k, cache.v, cache.tables, plan.cu_new, plan.kv_lens, max_new=max_new)
        x = x + self.o.mm(o.view(-1, h * self.dim))
        y = _norm(x)
        return x + self.down.mm(torch.nn.functional.silu(self.gate.mm(y)) * self.up.mm(y))


class Cache:
    """The pages of all requests. Lengths, tables and the list of free pages stay on the GPU, so a
    step reads nothing back; `take` drops the pages that a step took from the front of the list."""

    def __init__(self, layer, pages, page, requests, longest, dtype=torch.bfloat16):
        self.page = page
        # K and V pages alternate in one allocation
        both = torch.empty(pages, 2, layer.kv_heads, page, layer.dim, dtype=dtype, device="cuda")
        self.k, self.v = both[:, 0], both[:, 1]
        self.tables = torch.full((requests, -(-longest // page)), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.index = torch.arange(pages, device="cuda")

    def plan(self, new, tokens):
        return qaff.paged_plan(self.lens, new, self.free, self.tables, self.page, tokens)

    def take(self, plan, new):
        at = self.index + plan.pages_used.long()
        self.free.copy_(torch.where(at < at.numel(), self.free[at.clamp(max=at.numel() - 1)], -1))
        self.lens += new


def _norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def step(layer, cache, x, new, max_new):
    plan = cache.plan(new, x.shape[0])
    y = layer(x, plan, cache, max_new)
    cache.take(plan, new)
    return y


def prefill(layer, cache, prompts, chunk):
    """Takes the prompts ([length, width] each) in steps of up to `chunk` tokens a request; returns
    the output of each prompt's last token."""
    at, last = [0] * len(prompts), [None] * len(prompts)
    while any(a < p.shape[0] for a, p in zip(at, prompts)):
        new = [min(chunk, p.shape[0] - a) for a, p in zip(at, prompts)]
        x = torch.cat([p[a:a + n] for a, n, p in zip(at, new, prompts)])
        y = step(layer, cache, x, torch.tensor(new, dtype=torch.int32).cuda(), max(new))
        end = 0
        for b, n in enumerate(new):
            end += n
            if n:
                last[b] = y[end - 1]
        at = [a + n for a, n in zip(at, new)]
    return torch.stack(last)


class Decoder:
    """A captured step of one token a request: replay() takes x's values and overwrites them with the
    layer's output. What the graph reads (x, the ones) lives as long as it."""

    def __init__(self, layer, cache, x):
        self.x, self.one = x, torch.ones_like(cache.lens)
        state = cache.tables, cache.lens, cache.free
        saved = [t.clone() for t in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # one step outside the capture; what it changes is put back
            step(layer, cache, x, self.one, 1)
            for t, s in zip(state, saved):
                t.copy_(s)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            x.copy_(step(layer, cache, x, self.one, 1))

    def replay(self):
        self.graph.replay()


def main():
    gen = torch.Generator(device="cuda").manual_seed(1)
    layer = Layer(4096, 32, 8, 128, 14336, gen)
    lens = [1537 + 211 * b for b in range(16)]
    steps, page, chunk = 64, 16, 512
    longest = max(lens) + steps
    cache = Cache(layer, sum(-(-(n + steps) // page) for n in lens) + 8, page, len(lens), longest)
    prompts = [torch.randn(n, 4096, generator=gen, device="cuda").bfloat16() for n in lens]

    def timed(f):
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        r = f()
        b.record()
        torch.cuda.synchronize()
        return r, a.elapsed_time(b)

    prefill(layer, Cache(layer, 64, page, 1, 600), prompts[0][None, :600], chunk)  # loads the kernels
    x, ms = timed(lambda: prefill(layer, cache, prompts, chunk))
    print(f"{sum(lens)} prompt tokens of {len(lens)} requests in chunks of up to {chunk}: {ms:.2f} ms")
    decoder = Decoder(layer, cache, x)
    _, ms = timed(lambda: [decoder.replay() for _ in range(steps)])
    print(f"{steps} decode steps of {len(lens)} requests: {1000 * ms / steps:.1f} us a step")
    assert cache.lens.tolist() == [n + steps for n in lens] and x.isfinite().all()


if __name__ == "__main__":
    main()

"""An attention layer on quantised weights and a paged, quantised cache.

    python examples/attention_layer.py [--fmt bf16|f16|int8|int4] [--steps N] [--seqs B] [--prompt L]

Prompts of ragged lengths go through the fused q, k, v projection, the rotation
in place, the cache and prompt attention; then every sequence takes single
tokens, whose step (projection, rotation into the cache, paged attention, output
projection) is captured once in a CUDA graph and replayed.  The last step's
attention is compared with prompt attention over the whole sequences.  Weights
are random EXL3 layers, activations random.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exl3_trellis_quantized_gb300 as E  # noqa: E402
from exl3_trellis_quantized_gb300 import synthetic  # noqa: E402


class Projection:
    """An EXL3 linear on the GPU whose outputs have about the size of its inputs."""

    def __init__(self, k, widths, bits, cb, seed, device):
        layer = synthetic.make_layer(k, widths, bits, cb, seed)
        self.bits, self.cb, self.cols = bits, cb, layer.shard_cols
        self.trellis, self.suh = layer.trellis.to(device), layer.suh.to(device)
        self.svh = (layer.svh.float() * k**-0.5).half().to(device)

    def __call__(self, x):
        return E.linear(x, self.trellis, self.bits, self.cb, self.suh, self.svh, self.cols, out_dtype=x.dtype)


class AttentionLayer:
    """Sequences 0 .. seqs - 1, each with room for max_len tokens in the cache."""

    def __init__(self, hidden, heads, kv_heads, head_dim, seqs, max_len, fmt="int8", page=64, bits=4, window=0,
                 base=10000.0, seed=1, device="cuda"):
        self.heads, self.kv_heads, self.head_dim, self.page, self.window = heads, kv_heads, head_dim, page, window
        self.max_len = max_len
        kv = kv_heads * head_dim
        self.qkv = Projection(hidden, [heads * head_dim, kv, kv], bits, "mcg", seed, device)
        self.out = Projection(heads * head_dim, [hidden], bits, "mcg", seed + 1, device)
        self.phases, self.amplitude = E.rope_phases(head_dim, base=base, device=device)
        pages = (max_len + page - 1) // page
        self.cache = E.KVCache.empty(seqs * pages, page, kv_heads, head_dim, fmt, device=device)
        self.table = torch.randperm(seqs * pages, device=device).to(torch.int32).view(seqs, pages)
        self.kv_lens = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.one_each = torch.arange(seqs + 1, dtype=torch.int32, device=device)

    def slots(self, seq, position):
        """Cache rows of tokens at ``position`` of sequences ``seq``."""
        at = position.long()
        return self.table[seq.long(), at // self.page].long() * self.page + at % self.page

    def heads_of(self, y):
        rows = y.view(y.shape[0], -1, self.head_dim)
        return rows.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def prompt(self, x, lens, keep=True):
        """Attention of whole prompts [sum(lens), hidden], whose keys and values go into the cache unless not ``keep``."""
        device = x.device
        y = self.qkv(x)
        cu = torch.tensor([0] + lens, dtype=torch.int32, device=device).cumsum(0, dtype=torch.int32)
        seq = torch.arange(len(lens), device=device).repeat_interleave(torch.tensor(lens, device=device))
        position = (torch.arange(x.shape[0], device=device) - cu[seq]).to(torch.int32)
        turned = y.view(y.shape[0], -1, self.head_dim)[:, :self.heads + self.kv_heads]  # q and k lie side by side
        E.rope(turned, position, self.phases, amplitude=self.amplitude, out=turned)
        q, k, v = self.heads_of(y)
        if keep:
            E.kv_write(self.cache, k, v, self.slots(seq, position))
            self.kv_lens.copy_(cu[1:] - cu[:-1])
        return E.attention_prompt(q, k, v, cu, max(lens), window=self.window)

    def step(self, x):
        """Attention of the next token of every sequence, x [seqs, hidden]; nothing in here waits for the GPU."""
        q, k, v = self.heads_of(self.qkv(x))
        slots = self.slots(self.one_each[:-1], self.kv_lens)
        q = E.kv_write(self.cache, k, v, slots, q=q, positions=self.kv_lens, phases=self.phases, amplitude=self.amplitude)
        self.kv_lens += 1
        return E.attention_paged(q, self.cache, self.table, self.one_each, self.kv_lens, 1, self.max_len,
                                 window=self.window)

    def project(self, attention):
        return self.out(attention.flatten(1))


def run(fmt="int8", steps=32, seqs=8, prompt=500, hidden=2048, heads=16, kv_heads=4, head_dim=128, seed=3):
    """(the last step's attention, the same by prompt attention, microseconds a step)."""
    device = torch.device("cuda")
    dtype = torch.float16 if fmt == "f16" else torch.bfloat16
    g = torch.Generator(device=device).manual_seed(seed)
    lens = [max(1, prompt - 61 * b) for b in range(seqs)]
    layer = AttentionLayer(hidden, heads, kv_heads, head_dim, seqs, max(lens) + steps, fmt)
    prompts = [torch.randn((n, hidden), generator=g, device=device).to(dtype) for n in lens]
    tokens = torch.randn((steps, seqs, hidden), generator=g, device=device).to(dtype)

    layer.project(layer.prompt(torch.cat(prompts), lens))

    x = tokens[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # the first step as it is, and the graph of every later one
        attention = layer.step(x)
        layer.project(attention)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            attention = layer.step(x)
            layer.project(attention)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    with torch.cuda.stream(stream):
        for t in range(1, steps):
            x.copy_(tokens[t])
            graph.replay()
    torch.cuda.synchronize()
    micros = (time.perf_counter() - begin) * 1e6 / max(1, steps - 1)

    whole = [torch.cat([p, tokens[:, b]]) for b, p in enumerate(prompts)]
    lens = [n + steps for n in lens]
    every = layer.prompt(torch.cat(whole), lens, keep=False)
    last = torch.tensor(lens, device=device).cumsum(0) - 1
    if E.device_status() != 0:
        raise RuntimeError("a kernel gave up waiting")
    return attention, every[last], micros


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--fmt", default="int8", choices=sorted(E.KV_FORMATS))
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--seqs", type=int, default=8)
    p.add_argument("--prompt", type=int, default=500)
    a = p.parse_args()
    got, want, micros = run(a.fmt, max(2, a.steps), a.seqs, a.prompt)
    off = (got.float() - want.float()).norm() / want.float().norm()
    print(f"{a.fmt}: {a.seqs} sequences, {a.steps} steps, {micros:.1f} us a step; "
          f"step against prompt attention: {float(off):.2e} of the norm")


if __name__ == "__main__":
    main()

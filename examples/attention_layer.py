"""An attention layer on quantised weights and a paged, quantised cache.

    python examples/attention_layer.py [--fmt bf16|f16|int8|int4] [--steps N] [--seqs B] [--prompt L] [--shared S] [--norm]

Prompts of ragged lengths go through the fused q, k, v projection, the rotation
(with --norm the norms of query and key heads too) in place, the cache and prompt
attention; then every sequence takes single tokens, whose step (pages and slots
from the lengths, projection, rotation into the cache, paged attention, output
projection) is captured once in a CUDA graph and replayed.  With --shared all
prompts begin with the same S tokens, which only the first sequence writes: the others
begin on its pages and read them together.  The last step's attention is compared
with prompt attention over the whole sequences.  Weights are random EXL3 layers,
activations random.
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
    """Sequences 0 .. seqs - 1, each of up to max_len tokens in the cache."""

    def __init__(self, hidden, heads, kv_heads, head_dim, seqs, max_len, fmt="int8", page=64, bits=4, window=0,
                 base=10000.0, norm=None, seed=1, device="cuda"):
        """norm: the rows' type, for norms of query and key heads (random weights); None: no norms."""
        self.heads, self.kv_heads, self.head_dim, self.page, self.window = heads, kv_heads, head_dim, page, window
        self.max_len = max_len
        kv = kv_heads * head_dim
        self.qkv = Projection(hidden, [heads * head_dim, kv, kv], bits, "mcg", seed, device)
        self.out = Projection(heads * head_dim, [hidden], bits, "mcg", seed + 1, device)
        self.phases, self.amplitude = E.rope_phases(head_dim, base=base, device=device)
        pages = seqs * ((max_len + page - 1) // page)
        self.cache = E.KVCache.empty(pages, page, kv_heads, head_dim, fmt, device=device)
        self.tables = E.KVTables.empty(seqs, max_len, pages, page, device=device)
        self.one_each = torch.ones(seqs, dtype=torch.int32, device=device)
        self.q_weight = self.k_weight = self.qk_weight = None
        if norm is not None:
            g = torch.Generator(device=device).manual_seed(seed)
            self.q_weight, self.k_weight = ((1 + 0.2 * torch.randn(head_dim, generator=g, device=device)).to(norm)
                                            for _ in range(2))
            self.qk_weight = torch.cat([self.q_weight.expand(heads, -1), self.k_weight.expand(kv_heads, -1)])
        self.groups, self.prefix, self.max_prefix = None, None, 0
        self.shared_pages, self.running = 0, torch.ones(seqs, dtype=torch.bool)  # of shared prefixes, on the host

    def heads_of(self, y):
        rows = y.view(y.shape[0], -1, self.head_dim)
        return rows.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def prompt(self, x, lens, keep=True):
        """Attention of whole prompts [sum(lens), hidden], whose keys and values go into the cache unless not ``keep``."""
        if keep and self.groups is not None:
            raise ValueError("tokens behind a shared beginning go through step")
        device = x.device
        y = self.qkv(x)
        new = torch.tensor(lens, dtype=torch.int32, device=device)
        if keep:
            cu, position, slots, _ = E.kv_plan(self.tables, new, x.shape[0])
        else:
            cu = torch.tensor([0] + lens, dtype=torch.int32, device=device).cumsum(0, dtype=torch.int32)
            seq = torch.arange(len(lens), device=device).repeat_interleave(new)
            position = (torch.arange(x.shape[0], device=device) - cu[seq]).to(torch.int32)
        turned = y.view(y.shape[0], -1, self.head_dim)[:, :self.heads + self.kv_heads]  # q and k lie side by side
        E.rope(turned, position, self.phases, amplitude=self.amplitude, out=turned, weight=self.qk_weight)
        q, k, v = self.heads_of(y)
        if keep:
            E.kv_write(self.cache, k, v, slots)
        return E.attention_prompt(q, k, v, cu, max(lens), window=self.window)

    def share(self, tokens, hint=None):
        """All sequences begin with the first ``tokens`` (whole pages) of sequence 0, on its pages; none but it has any yet.
        hint: attention_shared's max_prefix, the tokens unless given."""
        if self.window > 0:
            raise ValueError("attention behind a shared beginning has no window")
        if tokens < 1 or tokens % self.page:
            raise ValueError("a shared beginning is whole pages")
        t, pages = self.tables, tokens // self.page
        t.block_table[1:, :pages] = t.block_table[0, :pages]
        t.held[1:] = pages
        t.kv_lens[1:] = tokens
        self.shared_pages = pages
        self.groups = torch.tensor([0, t.batch], dtype=torch.int32, device=t.kv_lens.device)
        self.prefix = torch.tensor([tokens], dtype=torch.int32, device=t.kv_lens.device)
        self.max_prefix = tokens if hint is None else hint

    def step(self, x, new=None, max_new=1):
        """Attention of the next tokens of every sequence (one each, or new[b] of at most max_new), x [tokens, hidden];
        nothing in here waits for the GPU.  Behind a shared beginning sequences that have ended take none: their rows
        are not in x, and their new[b] is 0."""
        q, k, v = self.heads_of(self.qkv(x))
        cu, position, slots, _ = E.kv_plan(self.tables, self.one_each if new is None else new, x.shape[0])
        q = E.kv_write(self.cache, k, v, slots, q=q, positions=position, phases=self.phases, amplitude=self.amplitude,
                       q_weight=self.q_weight, k_weight=self.k_weight)
        args = (q, self.cache, self.tables.block_table, cu, self.tables.kv_lens)
        if self.groups is None:
            return E.attention_paged(*args, max_new, self.max_len, window=self.window)
        return E.attention_shared(*args, self.groups, self.prefix, max_new, self.max_len, self.max_prefix,
                                  sharers=int(self.running.sum()))

    def end(self, ended):
        """Sequences end (bool [seqs]): their own pages are free again.  Those of a shared beginning are when the last of
        its sequences ends, and only then may sequences begin anew."""
        shared = None
        if self.groups is not None:
            now = ended.cpu() & self.running
            self.running &= ~now
            shared = torch.full_like(self.tables.held, self.shared_pages)
            if self.running.any():
                self.one_each.masked_fill_(ended, 0)
            else:
                shared[int(now.int().argmax())] = 0
                self.one_each.fill_(1)
                self.running.fill_(True)
                self.groups, self.prefix, self.max_prefix = None, None, 0
        E.kv_release(self.tables, ended, shared)

    def project(self, attention):
        return self.out(attention.flatten(1))


def run(fmt="int8", steps=32, seqs=8, prompt=500, hidden=2048, heads=16, kv_heads=4, head_dim=128, seed=3, shared=0,
        norm=False, hint=None):
    """(the last step's attention, the same by prompt attention, microseconds a step)."""
    device = torch.device("cuda")
    dtype = torch.float16 if fmt == "f16" else torch.bfloat16
    g = torch.Generator(device=device).manual_seed(seed)
    lens = [max(1, prompt - 61 * b) for b in range(seqs)]
    page = 64
    shared = shared // page * page
    layer = AttentionLayer(hidden, heads, kv_heads, head_dim, seqs, shared + max(lens) + steps, fmt, page=page,
                           norm=dtype if norm else None)
    begin = torch.randn((shared, hidden), generator=g, device=device).to(dtype)
    prompts = [torch.randn((n, hidden), generator=g, device=device).to(dtype) for n in lens]
    tokens = torch.randn((steps, seqs, hidden), generator=g, device=device).to(dtype)

    if shared:
        layer.prompt(begin, [shared] + [0] * (seqs - 1))
        layer.share(shared, hint)
        attention = layer.step(torch.cat(prompts), torch.tensor(lens, dtype=torch.int32, device=device), max(lens))
        layer.project(attention)
    else:
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
    start = time.perf_counter()
    with torch.cuda.stream(stream):
        for t in range(1, steps):
            x.copy_(tokens[t])
            graph.replay()
    torch.cuda.synchronize()
    micros = (time.perf_counter() - start) * 1e6 / max(1, steps - 1)

    whole = [torch.cat([begin, p, tokens[:, b]]) for b, p in enumerate(prompts)]
    lens = [shared + n + steps for n in lens]
    every = layer.prompt(torch.cat(whole), lens, keep=False)
    last = torch.tensor(lens, device=device).cumsum(0) - 1
    layer.end(torch.ones(seqs, dtype=torch.bool, device=device))
    if int(layer.tables.free_count) != layer.cache.num_pages:
        raise RuntimeError("pages are missing")
    if E.device_status() != 0:
        raise RuntimeError("a kernel gave up waiting")
    return attention, every[last], micros


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--fmt", default="int8", choices=sorted(E.KV_FORMATS))
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--seqs", type=int, default=8)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--shared", type=int, default=0, help="tokens that all prompts begin with (whole pages of 64)")
    p.add_argument("--norm", action="store_true", help="norms of query and key heads")
    a = p.parse_args()
    got, want, micros = run(a.fmt, max(2, a.steps), a.seqs, a.prompt, shared=a.shared, norm=a.norm)
    off = (got.float() - want.float()).norm() / want.float().norm()
    print(f"{a.fmt}: {a.seqs} sequences, {a.steps} steps, {micros:.1f} us a step; "
          f"step against prompt attention: {float(off):.2e} of the norm")


if __name__ == "__main__":
    main()

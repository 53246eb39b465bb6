"""A prompt, its continuation and a fork of it through the quantized projections and the paged 8-bit KV cache.

Attention layers of a decoder with Q4_K projections (by default the 7B shapes: hidden 3584, 28 query heads, 4 KV heads of
128; random weights and inputs, no rotary embedding):

    RMSNorm + Q8 (mq_quantize_q8) -> q | k | v -> mqkv_append -> mqkv_attention -> Q8 -> o -> residual

The prompt goes through the GEMMs in one piece; a decode step is captured once as a CUDA graph and replayed (pages and
lengths are taken on the device).  Then the conversation is forked, both continue, one ends, and the pool is compacted.

    python examples/kv_decode.py [--layers 4] [--prompt 3314] [--tokens 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_q8_activation_quantize_gb300 import binding as B  # noqa: E402
from quantized_q8_activation_quantize_gb300 import inputs, kv  # noqa: E402


class Attention:
    """The attention layers of a decoder and the cache they share, for up to `n_seqs` conversations."""

    def __init__(self, layers, hidden, heads, kv_heads, dim, n_seqs, max_tokens, page=64, seed=1):
        self.layers, self.hidden, self.heads, self.kv_heads, self.dim = layers, hidden, heads, kv_heads, dim
        self.n = (heads * dim, kv_heads * dim, kv_heads * dim)
        r = np.random.default_rng(seed)

        def q4k(n, k):
            return torch.from_numpy(inputs.q4k_weights(r, n, k).reshape(n, -1)).cuda()
        self.w = [{"qkv": [q4k(n, hidden) for n in self.n], "o": q4k(hidden, heads * dim),
                   "norm": torch.ones(hidden, device="cuda")} for _ in range(layers)]
        pages = n_seqs * -(-max_tokens // page)
        self.pool, self.refs = kv.alloc_pool(pages, layers, kv_heads, dim, page)
        self.cache = kv.cache(self.pool, self.refs, layers, kv_heads, dim, page)
        self.table = torch.full((n_seqs, -(-max_tokens // page)), -1, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.all = kv.sequences(self.table, self.len)
        self.pages_ws = kv.alloc_pages_workspace(self.cache, self.all)
        self.max_tokens = max_tokens
        self.scratch = {}

    def seqs(self, count):
        """The first `count` conversations."""
        return kv.sequences(self.table[:count], self.len[:count])

    def buffers(self, tokens, count):
        key = tokens, count
        if key not in self.scratch:
            ws = kv.alloc_attention_workspace(self.cache, self.seqs(count), self.heads, tokens, tokens // count, self.max_tokens,
                                              torch.float32)
            self.scratch[key] = (B.alloc_plane(tokens, self.hidden), B.alloc_plane(tokens, self.n[0]),
                                 torch.empty((tokens, self.heads, self.dim), device="cuda"),
                                 [torch.empty((tokens, n), device="cuda") for n in (*self.n, self.hidden)], ws)
        return self.scratch[key]

    def step(self, x, count):
        """x [tokens, hidden]: as many new tokens for each of the first `count` conversations; their hidden states after the
        layers.  Nothing of it waits for the device, so it can be captured."""
        tokens, seqs = x.shape[0], self.seqs(count)
        plane, plane_o, att, (q, k, v, o), ws = self.buffers(tokens, count)
        each = tokens // count
        add = torch.full((count,), each, dtype=torch.int32, device="cuda") if each != 1 else None
        kv.mqkv_extend(self.cache, seqs, add, self.pages_ws)
        for i, w in enumerate(self.w):
            B.mq_quantize_q8(x, tokens, self.hidden, w["norm"], 1e-6, plane)
            for wt, n, y in zip(w["qkv"], self.n, (q, k, v)):
                B.matmul("q4k", wt, n, self.hidden, plane, tokens, y)
            heads = [t.view(tokens, -1, self.dim) for t in (q, k, v)]
            kv.mqkv_append(self.cache, seqs, i, heads[1], heads[2])
            kv.mqkv_attention(self.cache, seqs, i, heads[0], att, None, each, self.max_tokens, ws)
            B.mq_quantize_q8(att, tokens, self.n[0], None, 0.0, plane_o)
            B.matmul("q4k", w["o"], self.hidden, self.n[0], plane_o, tokens, o)
            x = x + o
        return x

    def captured(self, count):
        """A decode step (one token each) as a CUDA graph: (graph, input, output)."""
        x = torch.zeros((count, self.hidden), device="cuda")
        self.buffers(count, count)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.step(x, count)
        return graph, x, y


def run(layers=4, hidden=3584, heads=28, kv_heads=4, dim=128, prompt=3314, tokens=32, page=64, say=print):
    """The whole path; returns what its test looks at."""
    torch.manual_seed(0)
    model = Attention(layers, hidden, heads, kv_heads, dim, 3, prompt + 2 * tokens + 2, page)
    x = torch.randn((prompt, hidden), device="cuda")
    start = time.perf_counter()
    last = model.step(x, 1)[-1:]
    torch.cuda.synchronize()
    say(f"prompt of {prompt} tokens, {layers} layers: {1e3 * (time.perf_counter() - start):.2f} ms (first call)")

    def decode(graph, x_in, y_out, h, count):
        x_in.copy_(torch.nn.functional.normalize(h, dim=1) * hidden ** 0.5)     # stands in for norm, head, sampling and embedding
        graph.replay()
        return y_out.clone()

    one = model.captured(1)
    h = decode(*one, last, 1)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(tokens - 1):
        h = decode(*one, h, 1)
    torch.cuda.synchronize()
    say(f"decode: {1e6 * (time.perf_counter() - start) / max(1, tokens - 1):.1f} us per token")

    # the conversation goes on three times from here; equal inputs give equal states but for rounding (where a sequence's work
    # is split depends on its place in the batch)
    kv.mqkv_fork(model.cache, model.all, torch.tensor([0, 0], dtype=torch.int32, device="cuda"),
                 torch.tensor([1, 2], dtype=torch.int32, device="cuda"), model.pages_ws)
    shared = int((model.refs == 3).sum())
    three = model.captured(3)
    h3 = decode(*three, h.expand(3, -1), 3)
    spread = float((h3 - h3[:1]).abs().max() / h3.square().mean().sqrt())
    say(f"forked twice: {shared} pages shared, the continuations differ by {spread:.1e} of the states' size")

    # the second one ends; the pool is moved together; the first goes on as if nothing had happened
    kv.mqkv_release(model.cache, model.all, torch.tensor([1], dtype=torch.int32, device="cuda"))
    keep = [t.clone() for t in (model.pool, model.refs, model.table, model.len)]
    before = decode(*one, h3[:1], 1)
    for t, old in zip((model.pool, model.refs, model.table, model.len), keep):
        t.copy_(old)
    kv.mqkv_compact(model.cache, model.all, model.pages_ws)
    after = decode(*one, h3[:1], 1)
    live = int((model.refs > 0).sum())
    say(f"compacted: {live} pages live, the last of them at {int(model.refs.nonzero().max())}")
    kv.mqkv_device_status()
    return {"spread": spread, "shared": shared, "same_after_compact": bool((before == after).all()), "state": after,
            "len": model.len.tolist(), "live": live}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=3314)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args()
    run(layers=a.layers, prompt=a.prompt, tokens=a.tokens)

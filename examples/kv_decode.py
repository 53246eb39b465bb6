"""A prompt, its continuation, a fork of it and a beam search through the quantized projections and the paged 8-bit KV cache.

Attention layers of a decoder with Q4_K projections (by default the 7B shapes: hidden 3584, 28 query heads, 4 KV heads of
128; random weights and inputs):

    residual + RMSNorm + Q8 (mqd_add_quantize_q8) -> q | k | v -> rotary positions and append (mqkv_append_rope) -> mqkv_attention -> Q8 -> o

The prompt goes through the GEMMs in one piece; a decode step is captured once as a CUDA graph and replayed (pages and
lengths are taken on the device).  Then the conversation is forked, both continue, one ends, and the pool is compacted.
At last the prompt is continued by beam search: a step with its head, its selection (mqd_beam_select) and the reordering of the cached
sequences (mqkv_reorder) is one graph too.

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
from quantized_q8_activation_quantize_gb300 import decoder, inputs, kv  # noqa: E402


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
        self.plan = decoder.rope_plan(dim)
        self.norm = torch.ones(hidden, device="cuda")
        self.scratch = {}

    @staticmethod
    def sections(tokens):
        """What the Q4_K matmul of as many tokens reads of its plane."""
        return B.PLANE_FOR_GEMV if B.matmul_path("q4k", tokens) == "gemv" else B.PLANE_FOR_GEMM

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
                                 [torch.empty((tokens, n), device="cuda") for n in (*self.n, self.hidden, self.hidden)], ws)
        return self.scratch[key]

    def step(self, x, count):
        """x [tokens, hidden]: as many new tokens for each of the first `count` conversations; their hidden states after the
        layers.  Nothing of it waits for the device, so it can be captured.  The plane of the states' norm is left for a head."""
        tokens, seqs = x.shape[0], self.seqs(count)
        plane, plane_o, att, (q, k, v, o, h), ws = self.buffers(tokens, count)
        each, sections = tokens // count, self.sections(tokens)
        add = torch.full((count,), each, dtype=torch.int32, device="cuda") if each != 1 else None
        kv.mqkv_extend(self.cache, seqs, add, self.pages_ws)
        for i, w in enumerate(self.w):
            if i == 0:
                B.mq_quantize_q8_ex(x, tokens, self.hidden, w["norm"], 1e-6, sections, plane)
            else:
                decoder.mqd_add_quantize_q8(o, x if i == 1 else h, h, w["norm"], 1e-6, sections, plane)
            for wt, n, y in zip(w["qkv"], self.n, (q, k, v)):
                B.matmul("q4k", wt, n, self.hidden, plane, tokens, y)
            heads = [t.view(tokens, -1, self.dim) for t in (q, k, v)]
            kv.mqkv_append_rope(self.cache, seqs, i, self.plan, heads[0], heads[0], heads[1], heads[2])
            kv.mqkv_attention(self.cache, seqs, i, heads[0], att, None, each, self.max_tokens, ws)
            B.mq_quantize_q8_ex(att, tokens, self.n[0], None, 0.0, sections, plane_o)
            B.matmul("q4k", w["o"], self.hidden, self.n[0], plane_o, tokens, o)
        decoder.mqd_add_quantize_q8(o, x if self.layers == 1 else h, h, self.norm, 1e-6, sections, plane)
        return h

    def captured(self, count):
        """A decode step (one token each) as a CUDA graph: (graph, input, output)."""
        x = torch.zeros((count, self.hidden), device="cuda")
        self.buffers(count, count)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.step(x, count)
        return graph, x, y


class Search:
    """Beam search from a prompt with `beams` rows of a model's cache; random embeddings and head.  A step's logits are scaled down to a spread of a few units."""

    def __init__(self, model, beams, vocab, stop=-1, seed=2):
        self.model, self.beams, self.vocab, self.stop = model, beams, vocab, stop
        r = np.random.default_rng(seed)
        self.head = torch.from_numpy(inputs.q4k_weights(r, vocab, model.hidden).reshape(vocab, -1)).cuda()
        self.table = torch.from_numpy(r.standard_normal((vocab, model.hidden)).astype(np.float32)).cuda()
        self.scale = 2.0 / (1.4 * model.hidden ** 0.5)
        self.logits = torch.zeros((beams, vocab), device="cuda")
        self.scores = torch.full((1, beams), -torch.inf, device="cuda")
        self.row, self.token = (torch.zeros((1, beams), dtype=torch.int32, device="cuda") for _ in range(2))
        self.cand = [torch.empty((1, 2 * beams), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
        self.rows = torch.arange(beams, dtype=torch.int32, device="cuda")
        self.ws = decoder.alloc_beam_workspace(1, beams, vocab, 2 * beams)

    def select(self):
        """The beams' continuations by their logits: next scores, rows and tokens, and the cache's rows after them."""
        decoder.mqd_beam_select(self.logits, self.scores, self.cand, (self.scores, self.row, self.token), self.stop, self.ws)
        kv.mqkv_reorder(self.model.cache, self.model.seqs(self.beams), self.row.view(-1), self.model.pages_ws)

    def step(self, x):
        """One token x [beams, hidden] of every beam, and the next ones' embeddings."""
        m = self.model
        m.step(x, self.beams)
        B.matmul("q4k", self.head, self.vocab, m.hidden, m.buffers(self.beams, self.beams)[0], self.beams, self.logits)
        self.logits.mul_(self.scale)
        self.select()
        x.copy_(self.table[self.token.view(-1).clamp(min=0).long()])

    def run(self, prompt, steps):
        """prompt: token ids.  The beams' tokens (a list each, without the prompt; shorter where a search has run out) and their scores.  The
        first `beams` rows of the cache are the search's: what they hold is released first."""
        m = self.model
        kv.mqkv_release(m.cache, m.seqs(self.beams), self.rows)
        first = self.table[torch.as_tensor(prompt, device="cuda")]
        m.step(first, 1)
        plane = B.alloc_plane(1, m.hidden)
        last = m.buffers(len(prompt), 1)[3][4][-1:]
        B.mq_quantize_q8_ex(last, 1, m.hidden, m.norm, 1e-6, m.sections(1), plane)
        B.matmul("q4k", self.head, self.vocab, m.hidden, plane, 1, self.logits[:1])
        self.logits.mul_(self.scale)
        self.scores.fill_(-torch.inf)                          # one beam is alive
        self.scores[0, 0] = 0
        self.select()
        taken = [(self.row.view(-1).clone(), self.token.view(-1).clone())]
        x = self.table[self.token.view(-1).clamp(min=0).long()]
        m.buffers(self.beams, self.beams)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(x)
        for _ in range(steps - 1):
            graph.replay()
            taken.append((self.row.view(-1).clone(), self.token.view(-1).clone()))
        tokens = []
        for b in range(self.beams):
            path, at = [], b
            for row, token in reversed(taken):
                if at >= 0 and int(row[at]) >= 0:
                    path.append(int(token[at]))
                at = int(row[at]) if at >= 0 else -1
            tokens.append(path[::-1])
        return tokens, self.scores[0].tolist()


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
    lens = model.len.tolist()

    # and a search of its own, three beams from the beginning of a text
    kv.mqkv_release(model.cache, model.all, torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    vocab = 2048
    paths, scores = Search(model, 3, vocab).run(np.random.default_rng(3).integers(0, vocab, min(prompt, 100)).tolist(), 4)
    say(f"beam search: {', '.join(f'{p} at {s:.2f}' for p, s in zip(paths, scores))}")
    kv.mqkv_device_status()
    return {"spread": spread, "shared": shared, "same_after_compact": bool((before == after).all()), "state": after,
            "len": lens, "live": live, "paths": paths, "scores": scores}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=3314)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args()
    run(layers=a.layers, prompt=a.prompt, tokens=a.tokens)

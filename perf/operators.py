"""Measured cases of the paged 8-bit KV cache: attention over it, appending to it and reading it back, and the
bookkeeping and copying of its pages.

A cache is a pool of pages; a page holds ``page`` tokens of every layer.  Layer slab of a page, in bytes:
K codes [kv_heads][page][dim], V codes [kv_heads][page][dim], f32 scales [2][kv_heads][page / 32], padded to a
multiple of 256.  A code byte is q + 128 with q in [-127, 127] and stands for q times the scale of its block of 32
tokens, its head and its half (K or V).  Sequences name their pages in a page table.

Every case is a dict of plain values; lengths follow from the case alone (``lens`` seeds them), contents from the
seed.  The 28 query heads, 4 KV heads of 128, 28 layers and the 3314-token prompt are the 7B shapes of this
repository's inputs; the other head layouts and lengths are generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32


def _attention(name, **kw):
    c = {"name": name, "op": "attention", "dtype": "f32", "heads": 28, "kv_heads": 4, "dim": 128, "page": 64, "layers": 2,
         "seqs": 1, "len_lo": 1, "len_hi": 1, "q_lo": 1, "q_hi": 1, "causal": True, "window": 0, "lens": 1}
    return {**c, **kw}


def _append(name, **kw):
    c = {"name": name, "op": "append", "dtype": "f32", "kv_heads": 4, "dim": 128, "page": 64, "layers": 2, "seqs": 1,
         "len_lo": 0, "len_hi": 0, "q_lo": 1, "q_hi": 1, "lens": 1}
    return {**c, **kw}


def _pages(name, **kw):
    c = {"name": name, "op": "fork", "kv_heads": 4, "dim": 128, "page": 64, "layers": 28, "seqs": 1, "children": 1,
         "len_lo": 1, "len_hi": 1, "keep": 1.0, "lens": 1}
    return {**c, **kw}


def listed():
    return [
        # one user's next token early in a chat: a single short sequence, where latency is all
        _attention("attn_one_token", len_lo=517, len_hi=517, lens=11),
        # a server's decode step: a ragged batch, f32 activations as this library's GEMVs write them
        _attention("attn_decode_batch", seqs=48, len_lo=100, len_hi=16384, lens=12),
        # two users with very long contexts: the cache is split along its length
        _attention("attn_decode_long", dtype="bf16", seqs=2, len_lo=200001, len_hi=262143, page=128, lens=13),
        # checking five drafted tokens per sequence at once, under a sliding window, small heads
        _attention("attn_verify_window", dtype="f16", heads=32, kv_heads=8, dim=64, page=32, seqs=24, len_lo=900, len_hi=9000, q_lo=5, q_hi=5,
                   window=4000, lens=14),
        # the 3314-token prompt of the 7B workload, straight through
        _attention("attn_prompt", len_lo=3314, len_hi=3314, q_lo=3314, q_hi=3314, lens=15),
        # ragged prompt chunks behind histories of other lengths, 16-bit activations: the largest
        _attention("attn_chunks", dtype="bf16", seqs=3, len_lo=5003, len_hi=8191, q_lo=1500, q_hi=2999, page=128, lens=16),
        # one new token for each sequence of a decode batch, inside blocks that already hold others
        _append("append_decode", seqs=64, len_lo=33, len_hi=4097, lens=17),
        # the keys and values of the 3314-token prompt
        _append("append_prompt", len_lo=0, len_hi=0, q_lo=3314, q_hi=3314, lens=18),
        # ragged chunks of many prompts, 16-bit, eight heads
        _append("append_chunks", dtype="bf16", kv_heads=8, page=128, seqs=16, len_lo=0, len_hi=3001, q_lo=700, q_hi=4095, lens=19),
        # one conversation continued in two ways
        _pages("fork_one", seqs=1, children=2, len_lo=3314, len_hi=3314, lens=20),
        # a batch of prompts, each sampled four times
        _pages("fork_batch", seqs=16, children=4, len_lo=100, len_hi=2000, lens=21),
        # a pool with holes, after two thirds of its sequences have ended, moved together
        _pages("compact_pool", op="compact", seqs=96, len_lo=100, len_hi=1500, keep=0.34, lens=22),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    pages = {"page": rng.choice([32, 64, 128, 256]), "lens": rng.randrange(1, 1 << 30)}
    heads, kv_heads, dim = rng.choice([(28, 4, 128), (32, 8, 128), (32, 8, 64), (16, 16, 64), (8, 1, 128), (40, 8, 128), (14, 2, 64), (12, 12, 128)])
    kind = rng.choice(["decode", "decode", "verify", "prefill", "prefill", "append", "append", "fork", "compact"])
    if kind in ("decode", "verify", "prefill"):
        top = {"decode": 400_000, "verify": 120_000, "prefill": 20_000}[kind] * 4 // max(4, kv_heads)
        seqs = _log_int(rng, 1, 64 if kind != "prefill" else 4)
        hi = _log_int(rng, 2, max(2, top // seqs))
        lo = _log_int(rng, 1, hi)
        q_hi = 1 if kind == "decode" else rng.randint(2, 12) if kind == "verify" else _log_int(rng, 13, max(14, min(hi, 2500)))
        q_lo = q_hi if kind != "prefill" else _log_int(rng, 1, q_hi)
        window = 0 if rng.random() < 0.7 else _log_int(rng, 1, hi)
        c = _attention("", dtype=rng.choice(list(TYPES)), heads=heads, kv_heads=kv_heads, dim=dim, seqs=seqs, len_lo=lo, len_hi=hi,
                       q_lo=q_lo, q_hi=q_hi, causal=rng.random() < 0.85, window=window, **pages)
    elif kind == "append":
        seqs = _log_int(rng, 1, 128)
        q_hi = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, 240_000 // (seqs * kv_heads)))
        hi = _log_int(rng, 1, 5000) - 1
        c = _append("", dtype=rng.choice(list(TYPES)), kv_heads=kv_heads, dim=dim, seqs=seqs, len_lo=rng.randint(0, hi), len_hi=hi,
                    q_lo=_log_int(rng, 1, q_hi), q_hi=q_hi, **pages)
    else:
        layers = rng.choice([1, 2, 12, 28])
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 2, max(2, min(4000, 1_500_000 // (seqs * layers))))
        kv = min(kv_heads, 8)
        c = _pages("", op=kind, kv_heads=kv, dim=dim, layers=layers, seqs=seqs + (4 if kind == "compact" else 0), children=rng.randint(1, 4),
                   len_lo=_log_int(rng, 1, hi), len_hi=hi, keep=round(rng.uniform(0.1, 0.9), 2), **pages)
    del c["name"]
    top = [max(work(x)[k] for x in listed()) for k in ("bytes", "flops")]
    while any(work(c)[k] > t for k, t in zip(("bytes", "flops"), top)):  # no drawn case costs more than the largest listed one
        c["len_hi"] = max(c["len_lo"], c["len_hi"] // 2)
        c["seqs"] = max(1, c["seqs"] * 3 // 4) + (4 if kind == "compact" and c["seqs"] < 8 else 0)
        c["len_lo"] = c["len_lo"] // 2
    return c


def _lengths(case):
    """(cached tokens with the new ones, new tokens) of every sequence; the ranges' ends both occur where there are two."""
    r = np.random.RandomState(case["lens"])
    n = case["seqs"]
    ln = np.rint(np.exp(r.uniform(math.log(case["len_lo"] + 1), math.log(case["len_hi"] + 1), n))).astype(np.int64) - 1
    q = r.randint(case.get("q_lo", 1), case.get("q_hi", 1) + 1, n).astype(np.int64)
    if n > 1:
        ln[0], ln[-1] = case["len_lo"], case["len_hi"]
    if case["op"] == "append":  # the range is of what stands there before
        return ln + q, q
    return np.maximum(ln, q), q


def _geometry(case):
    H, T, D = case["kv_heads"], case["page"], case["dim"]
    off_v, off_s = H * T * D, 2 * H * T * D
    slab = -(-(off_s + 2 * H * (T // BLOCK) * 4) // 256) * 256
    return off_s, slab, slab * case["layers"]


def _codes(case, pool):
    """[page, layer, K or V, head, token, dim] of the code bytes."""
    H, T, D, L = case["kv_heads"], case["page"], case["dim"], case["layers"]
    off_s, slab, _ = _geometry(case)
    return pool.view(-1, L, slab)[:, :, :off_s].unflatten(2, (2, H, T, D))


def _scales(case, pool):
    """[page, layer, K or V, head, block] of the scales."""
    H, T, L = case["kv_heads"], case["page"], case["layers"]
    off_s, slab, _ = _geometry(case)
    return pool.view(-1, L, slab)[:, :, off_s:off_s + 8 * H * (T // BLOCK)].view(torch.float32).unflatten(2, (2, H, T // BLOCK))


def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    ln, nq = _lengths(case)
    T, H, D, n = case["page"], case["kv_heads"], case["dim"], case["seqs"]
    fork = case["op"] == "fork"
    rows = n * (1 + case["children"]) if fork else n
    used = -(-ln // T)
    most = int(max(1, used.max()))
    spare = n * case["children"] if fork else 3
    n_pages = int(used.sum()) + spare + 2
    _, slab, page_bytes = _geometry(case)
    pool = torch.randint(0, 256, (n_pages, page_bytes), generator=g, device="cuda", dtype=torch.uint8)
    codes, scales = _codes(case, pool), _scales(case, pool)
    # a block's codes reach to both ends of [-127, 127], whatever its scale
    codes.clamp_(min=1)
    scales.copy_(torch.rand(scales.shape, generator=g, device="cuda") * 0.03 + 0.005)
    # the pages of a sequence lie anywhere in the pool
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = np.full((rows, most), -1, np.int64)
    at = 0
    for b in range(n):
        table[b, :used[b]] = np.arange(at, at + used[b])
        at += used[b]
    table = torch.from_numpy(table).cuda()
    table = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lens[:n] = torch.from_numpy(ln).cuda().to(torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    s = {"case": case, "pool": pool, "table": table, "lens": lens, "refs": refs, "layer": case["layers"] - 1}
    if case["op"] in ("attention", "append"):
        cu = np.concatenate([[0], np.cumsum(nq)])
        s["cu"] = torch.from_numpy(cu).cuda().to(torch.int32)
        s["tokens"], s["max_q"], s["max_kv"] = int(cu[-1]), int(nq.max()), int(max(1, ln.max()))
        dtype = TYPES[case["dtype"]]
    if case["op"] == "attention":
        s["q"] = _normal(g, (s["tokens"], case["heads"], D), dtype)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "append":
        # keys and values beside each other, as one projection writes them; a few channels of the keys are larger
        kv = _normal(g, (s["tokens"], 2, H, D))
        kv[:, 0, :, ::D // 4] *= 6
        kv = kv.to(dtype)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        start = (ln - nq) // BLOCK * BLOCK
        back = ln - start
        s["start"] = torch.from_numpy(start).cuda().to(torch.int32)
        s["cu_back"] = torch.from_numpy(np.concatenate([[0], np.cumsum(back)])).cuda().to(torch.int32)
        s["max_blocks"] = int((-(-back // BLOCK)).max())
        s["k_back"] = torch.empty((int(back.sum()), H, D), dtype=torch.float32, device="cuda")
        s["v_back"] = torch.empty_like(s["k_back"])
    if fork:
        s["parent"] = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(case["children"])
        s["child"] = torch.arange(n, rows, dtype=torch.int32, device="cuda")
    if case["op"] == "compact":
        gone = max(1, int(round(n * (1 - case["keep"]))))
        ids = torch.from_numpy(np.random.RandomState(case["lens"] + 1).permutation(n)[:gone].copy()).cuda().to(torch.int32)
        table2, lens2, refs2 = _released(case, table, lens, refs, ids)
        table.copy_(table2), lens.copy_(lens2), refs.copy_(refs2)
        s["table0"], s["refs0"] = table.clone(), refs.clone()
    return s


def _kept(s):
    """What a user of the library keeps from call to call: the cache's and the sequences' descriptions and the workspace."""
    if "kv" not in s:
        from quantized_q8_activation_quantize_gb300 import kv
        c = s["case"]
        s["cache"] = kv.cache(s["pool"], s["refs"], c["layers"], c["kv_heads"], c["dim"], c["page"])
        s["seqs"] = kv.sequences(s["table"], s["lens"])
        if c["op"] == "attention":
            s["ws"] = kv.alloc_attention_workspace(s["cache"], s["seqs"], c["heads"], s["tokens"], s["max_q"], s["max_kv"], s["q"].dtype)
        if c["op"] in ("fork", "compact"):
            s["ws"] = kv.alloc_pages_workspace(s["cache"], s["seqs"])
        s["kv"] = kv
    return s["kv"]


def run(s):
    return {"attention": _run_attention, "append": _run_append, "fork": _run_fork, "compact": _run_compact}[s["case"]["op"]](s)


# ------------------------------------------------------------------ attention ---

def _run_attention(s):
    case = s["case"]
    if own:
        _kept(s).mqkv_attention(s["cache"], s["seqs"], s["layer"], s["q"], s["out"], s["cu"], s["max_q"], s["max_kv"], s["ws"],
                                causal=case["causal"], window=case["window"])
        return s["out"]
    k, v = _dense(case, s["pool"], s["table"], s["layer"], torch.arange(s["max_kv"], device="cuda").expand(case["seqs"], -1))
    lens, cu = s["lens"].long(), s["cu"].long()
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    G = case["heads"] // case["kv_heads"]
    q = torch.zeros((case["seqs"], s["max_q"], case["kv_heads"], G, case["dim"]), device="cuda")
    q[b, i] = s["q"].float().unflatten(1, (case["kv_heads"], G)) * (1 / math.sqrt(case["dim"]))
    p = torch.einsum("bqhgd,bkhd->bhgqk", q, k)
    kpos = torch.arange(s["max_kv"], device="cuda")[None, None, :]
    qpos = (lens - cu.diff())[:, None, None] + torch.arange(s["max_q"], device="cuda")[None, :, None]
    seen = (kpos < lens[:, None, None]).expand(-1, s["max_q"], -1)
    seen = seen & (kpos <= qpos) if case["causal"] else seen
    seen = seen & (kpos > qpos - case["window"]) if case["window"] else seen
    p.masked_fill_(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1).permute(0, 3, 1, 2)[..., None]
    o = torch.einsum("bhgqk,bkhd->bqhgd", p, v)
    o = torch.where(total > 0, o / total, 0.0)
    return o[b, i].flatten(1, 2).to(s["q"].dtype)


def _dense(case, pool, table, layer, pos):
    """Keys and values in 32 bits at positions pos [sequence, n]: two of [sequence, n, head, dim]."""
    T = case["page"]
    page = torch.gather(table[:pos.shape[0]].long(), 1, (pos // T).clamp(max=table.shape[1] - 1)).clamp(min=0)
    slot = pos % T
    codes, scales = _codes(case, pool)[:, layer], _scales(case, pool)[:, layer]
    kv = (codes[page, :, :, slot].float() - 128.0) * scales[page, :, :, slot // BLOCK][..., None]
    return kv[:, :, 0], kv[:, :, 1]


# -------------------------------------------------------------- append, read ---

def _run_append(s):
    case = s["case"]
    if own:
        kv = _kept(s)
        kv.mqkv_append(s["cache"], s["seqs"], s["layer"], s["k"], s["v"], s["cu"])
        kv.mqkv_read(s["cache"], s["seqs"], s["layer"], s["k_back"], s["v_back"], s["cu_back"], s["start"])
        return s["k_back"], s["v_back"]
    T, n = case["page"], case["seqs"]
    lens, cu, start = s["lens"].long(), s["cu"].long(), s["start"].long()
    new = cu.diff()
    first = lens - new - start  # slots of the first block that hold earlier tokens
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b] + first[b]
    x = torch.zeros((n, s["max_blocks"] * BLOCK, 2, case["kv_heads"], case["dim"]), device="cuda")
    x[b, i] = torch.stack([s["k"].float(), s["v"].float()], 1)
    x = x.unflatten(1, (-1, BLOCK))  # [sequence, block, slot, K or V, head, dim]
    pos = start[:, None] + torch.arange(s["max_blocks"] * BLOCK, device="cuda")
    page = torch.gather(s["table"].long(), 1, (pos // T).clamp(max=s["table"].shape[1] - 1)).clamp(min=0).unflatten(1, (-1, BLOCK))
    slot = (pos % T).unflatten(1, (-1, BLOCK))
    codes, scales = _codes(case, s["pool"])[:, s["layer"]], _scales(case, s["pool"])[:, s["layer"]]
    q0 = codes[page, :, :, slot].float() - 128.0
    d0 = scales[page[:, :, 0], :, :, slot[:, :, 0] // BLOCK]  # [sequence, block, K or V, head]
    j = torch.arange(s["max_blocks"] * BLOCK, device="cuda").unflatten(0, (-1, BLOCK))[None]
    old = j < first[:, None, None]
    live = (pos < lens[:, None]).unflatten(1, (-1, BLOCK)) & ~old
    d0 = torch.where(old.any(2)[..., None, None], d0, 0.0)
    d = torch.maximum(d0, x.abs().amax((2, 5)) / 127.0)
    away = lambda y: torch.trunc(y + torch.copysign(torch.full_like(y, 0.5), y))  # noqa: E731
    inv = torch.where(d > 0, 1.0 / d, 0.0)[:, :, None, :, :, None]
    shrink = torch.where(d > d0, d0 / d, 1.0)[:, :, None, :, :, None]
    q = torch.where(live[..., None, None, None], away(x * inv).clamp(-127, 127), away(q0 * shrink))
    write = live | old
    where = torch.where(write, torch.arange(write.numel(), device="cuda").view(write.shape), -1).flatten().sort().values
    where = where[-int(s["k_back"].shape[0]):]  # as many slots as there are tokens to write
    codes[page.flatten()[where], :, :, slot.flatten()[where]] = (q + 128.0).to(torch.uint8).flatten(0, 2)[where]
    blocks = torch.where(write.any(2), torch.arange(write[:, :, 0].numel(), device="cuda").view(write.shape[:2]), -1).flatten()
    blocks = torch.where(blocks >= 0, blocks, blocks.amax())  # a block that is not there writes the last one again
    scales[page[:, :, 0].flatten()[blocks], :, :, (slot[:, :, 0] // BLOCK).flatten()[blocks]] = d.flatten(0, 1)[blocks]
    cu = s["cu_back"].long()
    t = torch.arange(s["k_back"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = start[b] + t - cu[b]
    page, slot = s["table"].long()[b, pos // T], pos % T
    kv = (codes[page, :, :, slot].float() - 128.0) * scales[page, :, :, slot // BLOCK][..., None]
    return kv[:, 0], kv[:, 1]


# --------------------------------------------------------------------- pages ---

def _released(case, table, lens, refs, ids):
    """The tables after the sequences `ids` have given their pages back."""
    ids = ids.long()
    have = (lens[ids].long() + case["page"] - 1) // case["page"]
    held = torch.arange(table.shape[1], device="cuda")[None] < have[:, None]
    refs = refs.index_add(0, table[ids].long().clamp(min=0).flatten(), -held.int().flatten())
    return table.index_fill(0, ids, -1), lens.index_fill(0, ids, 0), refs


def _run_fork(s):
    """The children of the last fork end, and every parent is forked into as many new ones."""
    case = s["case"]
    if own:
        kv = _kept(s)
        kv.mqkv_release(s["cache"], s["seqs"], s["child"])
        kv.mqkv_fork(s["cache"], s["seqs"], s["parent"], s["child"], s["ws"])
    else:
        T, L = case["page"], case["layers"]
        table, lens, refs = _released(case, s["table"], s["lens"], s["refs"], s["child"])
        parent, child = s["parent"].long(), s["child"].long()
        ln = lens[parent].long()
        full, part = ln // T, ln % T > 0
        free = torch.argsort((refs > 0).int(), stable=True)  # the free pages, the lowest first
        page = free[(part.long().cumsum(0) - 1).clamp(min=0)]
        slot = torch.arange(table.shape[1], device="cuda")[None]
        share = slot < full[:, None]
        tail = (slot == full[:, None]) & part[:, None]
        old = table[parent].long().clamp(min=0)
        refs = refs.index_add(0, old.flatten(), share.int().flatten()).index_add(0, page, part.int())
        table[child] = torch.where(share, old, torch.where(tail, page[:, None], -1)).int()
        lens[child] = ln.int()
        # the used blocks of the tail pages, and all of their scales; a fork without one copies a page onto itself
        src = old.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
        dst = torch.where(part, page, src)
        blocks = torch.arange(T, device="cuda") // BLOCK * BLOCK < (ln % T)[:, None]
        codes, scales = _codes(case, s["pool"]), _scales(case, s["pool"])
        codes[dst] = torch.where(blocks[:, None, None, None, :, None], codes[src], codes[dst])
        scales[dst] = scales[src]
        s["table"].copy_(table), s["lens"].copy_(lens), s["refs"].copy_(refs)
    # page memory as the 32-bit words that are copied
    return s["table"], s["lens"], s["refs"], s["pool"].view(torch.int32)


def _run_compact(s):
    """The tables as the ended sequences left them, and the live pages moved to the front of the pool."""
    s["table"].copy_(s["table0"]), s["refs"].copy_(s["refs0"])
    if own:
        _kept(s).mqkv_compact(s["cache"], s["seqs"], s["ws"])
    else:
        refs = s["refs"]
        live = refs > 0
        at = torch.arange(refs.numel(), device="cuda")
        n = live.sum()
        hole, mover = ~live & (at < n), live & (at >= n)
        half = refs.numel() // 2 + 1
        dst, src = torch.argsort((~hole).int(), stable=True)[:half], torch.argsort((~mover).int(), stable=True)[:half]
        real = at[:half] < mover.sum()
        # pairs past the last move the first one again, or page 0 onto itself where there is none
        none = mover.sum() == 0
        dst, src = torch.where(real, dst, torch.where(none, 0, dst[0])), torch.where(real, src, torch.where(none, 0, src[0]))
        s["pool"][dst] = s["pool"][src]
        place = at.scatter(0, src, dst)
        held = torch.arange(s["table"].shape[1], device="cuda")[None] < ((s["lens"].long() + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
        s["table"].copy_(torch.where(held, place[s["table"].long().clamp(min=0)], s["table"].long()))
        moved = refs.scatter(0, src, torch.where(real, 0, torch.where(none, refs[0], 0)).int())
        refs.copy_(moved.scatter(0, dst, refs[src]))
    return s["table"], s["refs"], s["pool"].view(torch.int32)


# ---------------------------------------------------------------------- work ---

def work(case):
    ln, nq = _lengths(case)
    H, D, T, L = case["kv_heads"], case["dim"], case["page"], case["layers"]
    if case["op"] == "attention":
        size = 4 if case["dtype"] == "f32" else 2
        pairs, read = 0, 0
        for n, q in zip(ln, nq):
            pos = n - q + np.arange(q)
            last = np.clip(np.minimum(pos, n - 1) if case["causal"] else np.full(q, n - 1), -1, n - 1)
            first = np.maximum(pos - case["window"] + 1, 0) if case["window"] else np.zeros(q, np.int64)
            seen = np.maximum(last - first + 1, 0)
            pairs += int(seen.sum())
            if seen.max() > 0:
                read += int(last[seen > 0].max() - first[seen > 0].min() + 1)
        return {"bytes": 2 * int(nq.sum()) * case["heads"] * D * size + read * 2 * H * (D + 4 / BLOCK) + 4 * read / T, "flops": 4 * D * case["heads"] * pairs}
    if case["op"] == "append":
        size = 4 if case["dtype"] == "f32" else 2
        new, back = int(nq.sum()), int((ln - (ln - nq) // BLOCK * BLOCK).sum())
        per = 2 * H * D
        # the new values in, their codes out, and what earlier tokens share their block with in and out again; then all of it read back in 32 bits
        return {"bytes": per * (new * (size + 1) + 2 * (back - new) + back * 5), "flops": per * (4 * new + back)}
    slab = 2 * H * (T * D + T // BLOCK * 4)
    if case["op"] == "fork":
        tail = -(-(ln % T) // BLOCK) * BLOCK * (ln % T > 0)
        moved = int((tail * 2 * H * D + (tail > 0) * 2 * H * (T // BLOCK) * 4).sum()) * L
        return {"bytes": case["children"] * (2 * moved + 12 * int((-(-ln // T)).sum())), "flops": 0}
    gone = max(1, int(round(case["seqs"] * (1 - case["keep"]))))
    ids = np.random.RandomState(case["lens"] + 1).permutation(case["seqs"])[:gone]
    used = -(-ln // T)
    total, live = int(used.sum()) + 5, int(used.sum() - used[ids].sum())
    # of the live pages the share that lies past the new end moves: pages lie anywhere, so the expected number
    return {"bytes": 2 * slab * L * live * (1 - live / total) + 8 * int(used.sum()), "flops": 0}


# --------------------------------------------------------------------- exact ---

def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return None  # nothing is computed: bytes move
    f8 = torch.float64
    H, D, T, layer = case["kv_heads"], case["dim"], case["page"], s["layer"]
    off_s, slab, _ = _geometry(case)
    table, lens, cu = s["table"].cpu().numpy(), s["lens"].cpu().numpy(), s["cu"].cpu().numpy()

    def history(b, n, h, half):
        """The first n tokens of a sequence's K (half 0) or V (1) of one head: codes and the scale of each token."""
        pages = torch.from_numpy(table[b, :-(-n // T)].astype(np.int64)).cuda()
        base = s["pool"].view(-1, case["layers"], slab)[pages, layer]
        q = base[:, (half * H + h) * T * D:][:, :T * D].reshape(-1, D)[:n].to(f8) - 128
        d = base[:, off_s + (half * H + h) * (T // BLOCK) * 4:][:, :(T // BLOCK) * 4].contiguous().view(torch.float32).reshape(-1)
        return q, d.to(f8).repeat_interleave(BLOCK)[:n]

    if case["op"] == "attention":
        out = torch.zeros(s["q"].shape, dtype=f8, device="cuda")
        group = case["heads"] // H
        for b in range(case["seqs"]):
            n, lo, hi = int(lens[b]), int(cu[b]), int(cu[b + 1])
            if n == 0 or hi == lo:
                continue
            at = torch.arange(n - (hi - lo), n, device="cuda")[:, None]
            j = torch.arange(n, device="cuda")[None]
            hidden = (j > at) if case["causal"] else torch.zeros((hi - lo, n), dtype=torch.bool, device="cuda")
            if case["window"]:
                hidden = hidden | (j <= at - case["window"])
            empty = hidden.all(1)
            for h in range(H):
                (kq, kd), (vq, vd) = history(b, n, h, 0), history(b, n, h, 1)
                k, v = kq * kd[:, None], vq * vd[:, None]
                for x in range(h * group, h * group + group):
                    logits = (s["q"][lo:hi, x].to(f8) @ k.T) / D ** 0.5
                    w = torch.softmax(logits.masked_fill(hidden, -math.inf), 1)
                    out[lo:hi, x] = torch.where(empty[:, None], 0.0, w @ v)
        return out
    back = [torch.empty(s["k_back"].shape, dtype=f8, device="cuda") for _ in range(2)]
    cub, start = s["cu_back"].cpu().numpy(), s["start"].cpu().numpy()
    for half, x in enumerate((s["k"], s["v"])):
        for b in range(case["seqs"]):
            n, before, first = int(lens[b]), int(lens[b]) - int(cu[b + 1] - cu[b]), int(start[b])
            new = x[int(cu[b]):int(cu[b + 1])].to(f8)
            old = torch.empty((before - first, H, D), dtype=f8, device="cuda")
            d_old = torch.zeros(H, dtype=f8, device="cuda")
            for h in range(H if before > first else 0):
                q, d = history(b, before, h, half)
                old[:, h], d_old[h] = q[first:], d[first]
            rows = torch.cat([old * d_old[:, None], new])
            pad = -(-(n - first) // BLOCK) * BLOCK - (n - first)
            blocks = torch.cat([rows, torch.zeros((pad, H, D), dtype=f8, device="cuda")]).view(-1, BLOCK, H, D)
            kept = blocks.clone()
            kept[0, :before - first] = 0
            # a block's scale is one number in 32 bits
            d = (kept.abs().amax((1, 3)) / 127).float().to(f8)
            d[0] = torch.maximum(d[0], d_old)
            y = blocks / torch.where(d > 0, d, 1.0)[:, None, :, None]
            q = (torch.sign(y) * torch.floor(y.abs() + 0.5)).clamp(-127, 127)
            back[half][int(cub[b]):int(cub[b + 1])] = (q * d[:, None, :, None]).view(-1, H, D)[:n - first]
    return tuple(back)

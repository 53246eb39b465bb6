"""Measured cases of what a decoder layer does between its matrix products and the paged 8-bit cache, and of beam search at its end:
the residual's addition with RMSNorm and the Q8 plane, rotary positions (alone, and with the cache's append), the selection over beams
and vocabulary, and the reordering of the cached sequences that follows from it.

A Q8 plane holds blocks of 32 values of a row as codes of 8 bits with one f32 scale each; here it comes back as the values that the codes
stand for.  The cache is the paged one: a page holds ``page`` tokens of every layer, the slab of a layer is K codes [kv_heads][page][dim], V
codes, f32 scales [2][kv_heads][page / 32], padded to a multiple of 256 bytes; a code byte is q + 128.

Every case is a dict of plain values; lengths follow from the case alone (``lens`` seeds them), contents from the seed.  Hidden size 3584, 28
query heads and 4 KV heads of 128, 28 layers, the vocabulary of 152064 and the 3314-token prompt are the 7B shapes of this repository's inputs;
the other sizes are generic.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32
EPS = 1e-6


def _add(name, **kw):
    return {**{"name": name, "op": "add", "dtype": "f32", "rows": 1, "width": 3584, "use": "gemm"}, **kw}


def _rope(name, **kw):
    c = {"name": name, "op": "rope", "dtype": "f32", "tokens": 1, "heads": 28, "dim": 128, "rot": 128, "interleaved": False, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "original": 0, "first": 0}
    return {**c, **kw}


def _append(name, **kw):
    c = {"name": name, "op": "append", "dtype": "f32", "heads": 28, "kv_heads": 4, "dim": 128, "rot": 128, "interleaved": False, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "original": 0, "first": 0, "page": 64, "layers": 2, "seqs": 1, "len_lo": 0, "len_hi": 0, "q_lo": 1, "q_hi": 1,
         "lens": 1}
    return {**c, **kw}


def _select(name, **kw):
    return {**{"name": name, "op": "select", "dtype": "f32", "groups": 1, "beams": 4, "vocab": 152064, "pad": 0, "masked": 0.0, "dead": False}, **kw}


def _reorder(name, **kw):
    c = {"name": name, "op": "reorder", "kv_heads": 4, "dim": 128, "page": 64, "layers": 28, "groups": 1, "beams": 4, "len_lo": 1, "len_hi": 1,
         "new": 32, "ended": False, "lens": 1}
    return {**c, **kw}


def listed():
    return [
        # one decode token between attention and the FFN: latency is all
        _add("add_token", use="gemv"),
        # the 3314-token prompt of the 7B workload, f32 as the GEMMs write it
        _add("add_prompt", rows=3314),
        # a long ragged batch of prompts with a 16-bit residual stream
        _add("add_chunks", dtype="bf16", rows=9001, width=8192),
        # five drafted tokens' queries, part of each head rotated, pairs beside each other
        _rope("rope_drafted", tokens=5, rot=64, interleaved=True, first=4093),
        # queries of a long 16-bit prompt far into a stretched context
        _rope("rope_far", dtype="bf16", tokens=7001, heads=40, base=500000.0, scaling="turns", factor=8.0, original=8192, first=120_001),
        # a server's decode step: one token for each of 48 sequences, q rotated and k, v into the cache
        _append("append_decode", seqs=48, len_lo=33, len_hi=4097, lens=17),
        # ragged chunks of many prompts, 16-bit, eight KV heads, a stretched context
        _append("append_chunks", dtype="bf16", heads=32, kv_heads=8, page=128, seqs=16, len_lo=0, len_hi=3001, q_lo=700, q_hi=4095, scaling="index",
                factor=4.0, original=4096, base=1000000.0, lens=19),
        # one request with four beams over the whole vocabulary
        _select("select_one"),
        # a batch of them, the largest
        _select("select_batch", groups=32),
        # wide beams over an odd vocabulary in 16 bits, half of it forbidden, rows padded, some beams not alive yet
        _select("select_wide", dtype="bf16", groups=6, beams=16, vocab=50257, pad=7, masked=0.5, dead=True),
        # the cache of one request with four beams after a selection
        _reorder("reorder_one", len_lo=3314, len_hi=3314, lens=32),
        # a batch of them, some of whose beams have ended
        _reorder("reorder_batch", groups=24, len_lo=100, len_hi=2000, ended=True, lens=24),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _positions(rng, dim):
    """The arguments of a rotation that a draw may have."""
    scaling = rng.choice(["none", "none", "linear", "base", "turns", "index"])
    return {"rot": rng.choice([dim, dim, dim // 2, dim * 3 // 4]), "interleaved": rng.random() < 0.4, "base": rng.choice([10000.0, 500000.0, 1000000.0]),
            "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), "original": rng.choice([2048, 4096, 8192]),
            "first": 0 if rng.random() < 0.5 else _log_int(rng, 1, 1_000_000)}


def draw(rng):
    kind = rng.choice(["add", "add", "rope", "append", "append", "select", "select", "reorder"])
    lens = rng.randrange(1, 1 << 30)
    if kind == "add":
        width = 256 * _log_int(rng, 1, 64)
        c = _add("", dtype=rng.choice(list(TYPES)), rows=_log_int(rng, 1, 20000), width=width, use=rng.choice(["gemm", "gemv"]))
        shrink = [("rows", 1)]
    elif kind == "rope":
        dim = rng.choice([64, 80, 128, 256])
        c = _rope("", dtype=rng.choice(list(TYPES)), tokens=_log_int(rng, 1, 20000), heads=rng.choice([1, 5, 8, 28, 40, 64]), dim=dim, **_positions(rng, dim))
        c["rot"] = c["rot"] // 8 * 8
        shrink = [("tokens", 1)]
    elif kind == "append":
        heads, kv_heads, dim = rng.choice([(28, 4, 128), (32, 8, 128), (32, 8, 64), (16, 16, 64), (8, 1, 128), (40, 8, 128), (14, 2, 64), (9, 3, 128)])
        seqs = _log_int(rng, 1, 128)
        q_hi = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, 240_000 // (seqs * kv_heads)))
        hi = _log_int(rng, 1, 5000) - 1
        c = _append("", dtype=rng.choice(list(TYPES)), heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([32, 64, 128, 256]), seqs=seqs,
                    len_lo=rng.randint(0, hi), len_hi=hi, q_lo=_log_int(rng, 1, q_hi), q_hi=q_hi, lens=lens, **_positions(rng, dim))
        shrink = [("q_hi", 1), ("q_lo", 1), ("seqs", 1)]
    elif kind == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c = _select("", dtype=rng.choice(list(TYPES)), groups=_log_int(rng, 1, max(1, 64 // beams)), beams=beams, vocab=_log_int(rng, 1000, 200_000),
                    pad=rng.choice([0, 0, 3, 8]), masked=rng.choice([0.0, 0.0, 0.3, 0.95]), dead=rng.random() < 0.3)
        shrink = [("groups", 1), ("vocab", 1000)]
    else:
        kv_heads, dim = rng.choice([(4, 128), (8, 128), (8, 64), (1, 128), (2, 64)])
        beams = rng.choice([2, 3, 4, 5, 8])
        hi = _log_int(rng, 40, 4000)
        c = _reorder("", kv_heads=kv_heads, dim=dim, page=rng.choice([32, 64, 128, 256]), layers=rng.choice([1, 2, 12, 28]), groups=_log_int(rng, 1, 32),
                     beams=beams, len_lo=_log_int(rng, 1, hi), len_hi=hi, new=_log_int(rng, 1, 200), ended=rng.random() < 0.4, lens=lens)
        shrink = [("groups", 1), ("len_hi", 1)]
    del c["name"]
    top = [max(work(x)[k] for x in listed()) for k in ("bytes", "flops")]
    while any(work(c)[k] > t for k, t in zip(("bytes", "flops"), top)):  # no drawn case costs more than the largest listed one
        for name, least in shrink:
            c[name] = max(least, c[name] * 3 // 4)
        if "len_lo" in c:
            c["len_lo"] = min(c["len_lo"], c["len_hi"])
    return c


def _lengths(case):
    """append: (cached tokens with the new ones, new tokens) of every sequence; the ranges' ends both occur where there are two."""
    r = np.random.RandomState(case["lens"])
    n = case["seqs"]
    ln = np.rint(np.exp(r.uniform(math.log(case["len_lo"] + 1), math.log(case["len_hi"] + 1), n))).astype(np.int64) - 1
    q = r.randint(case["q_lo"], case["q_hi"] + 1, n).astype(np.int64)
    if n > 1:
        ln[0], ln[-1] = case["len_lo"], case["len_hi"]
    return ln + q, q


def _beams(case):
    """reorder: (prompt tokens, tokens since) of every group, and the row that every beam continues (-1: it has ended)."""
    r = np.random.RandomState(case["lens"])
    G, B = case["groups"], case["beams"]
    prompt = np.rint(np.exp(r.uniform(math.log(case["len_lo"]), math.log(case["len_hi"]), G))).astype(np.int64)
    since = r.randint(1, case["new"] + 1, G).astype(np.int64)
    parent = r.randint(0, B, (G, B))
    parent += np.arange(G)[:, None] * B
    parent = parent.reshape(-1)
    if case["ended"]:  # rows of beams that nobody continues stay empty
        parent[(r.rand(G * B) < 0.5) & ~np.isin(np.arange(G * B), parent)] = -1
    return prompt, since, parent


def _geometry(case):
    H, T, D = case["kv_heads"], case["page"], case["dim"]
    off_s = 2 * H * T * D
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


def _frequencies(case):
    """Radians per position of every pair of the rotated part, in 64 bits."""
    rot, base, s, original = case["rot"], case["base"], case["factor"], case["original"]
    if case["scaling"] == "base":
        base = base * s ** (rot / (rot - 2))
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        return f / s
    if case["scaling"] == "turns":  # pairs that turn often in the original length keep their speed
        keep = np.clip((original * f / (2 * np.pi) - 1.0) / (4.0 - 1.0), 0, 1)
        return f * (keep + (1 - keep) / s)
    if case["scaling"] == "index":  # the same, along the pairs' numbers
        lo, hi = (rot * np.log(original / (turns * 2 * np.pi)) / (2 * np.log(base)) for turns in (32.0, 1.0))
        lo, hi = max(np.floor(lo), 0), min(np.ceil(hi), rot - 1)
        keep = 1 - np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f * (keep + (1 - keep) / s)
    return f


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "index" else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    s = {"case": case}
    {"add": _prepare_add, "rope": _prepare_rope, "append": _prepare_append, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, g, s)
    return s


def _prepare_add(case, g, s):
    M, K, dtype = case["rows"], case["width"], TYPES[case["dtype"]]
    s["x"] = _normal(g, (M, K), dtype)
    res = _normal(g, (M, K))
    res[:, torch.randint(0, K, (max(1, K // 128),), generator=g, device="cuda")] *= 20  # a few channels of the stream are larger
    s["res"] = res.to(dtype)
    s["w"] = 1 + 0.1 * _normal(g, (K,))
    s["h"] = torch.empty_like(s["x"])
    s["back"] = torch.empty((M, K), dtype=torch.float16 if case["dtype"] == "f32" else dtype, device="cuda")  # what the codes stand for, in 16 bits


def _prepare_rope(case, g, s):
    s["x"] = _normal(g, (case["tokens"], case["heads"], case["dim"]), TYPES[case["dtype"]])
    s["pos"] = torch.arange(case["first"], case["first"] + case["tokens"], device="cuda", dtype=torch.int32)
    s["freq"] = torch.from_numpy(_frequencies(case)).cuda()
    s["out"] = torch.empty_like(s["x"])


def _prepare_append(case, g, s):
    ln, nq = _lengths(case)
    T, H, D, n, dtype = case["page"], case["kv_heads"], case["dim"], case["seqs"], TYPES[case["dtype"]]
    used = -(-ln // T)
    n_pages = int(used.sum()) + 3
    _, slab, page_bytes = _geometry(case)
    pool = torch.randint(0, 256, (n_pages, page_bytes), generator=g, device="cuda", dtype=torch.uint8)
    codes, scales = _codes(case, pool), _scales(case, pool)
    codes.clamp_(min=1)
    scales.copy_(torch.rand(scales.shape, generator=g, device="cuda") * 0.03 + 0.005)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)  # the pages of a sequence lie anywhere in the pool
    table = np.full((n, int(max(1, used.max()))), -1, np.int64)
    table[np.arange(table.shape[1])[None] < used[:, None]] = np.arange(used.sum())
    table = torch.from_numpy(table).cuda()
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
    s["lens"] = torch.from_numpy(ln).cuda().to(torch.int32)
    s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    s["refs"][s["table"][s["table"] >= 0].long()] = 1
    s["pool"], s["layer"] = pool, case["layers"] - 1
    cu = np.concatenate([[0], np.cumsum(nq)])
    s["cu"], s["tokens"] = torch.from_numpy(cu).cuda().to(torch.int32), int(cu[-1])
    # q, k and v beside each other, as one projection writes them; a few channels of the keys are larger
    qkv = _normal(g, (s["tokens"], case["heads"] + 2 * H, D))
    qkv[:, case["heads"]:case["heads"] + H, ::D // 4] *= 6
    s["q"], s["k"], s["v"] = qkv.to(dtype).split([case["heads"], H, H], 1)
    s["out"] = torch.empty((s["tokens"], case["heads"], D), dtype=dtype, device="cuda")
    s["freq"] = torch.from_numpy(_frequencies(case)).cuda()
    # positions of their own where the sequences go on from a text that the cache no longer holds
    b = np.repeat(np.arange(n), nq)
    at = np.arange(s["tokens"]) - cu[b] + (ln - nq)[b]
    s["pos"] = torch.from_numpy(at + case["first"]).cuda().to(torch.int32) if case["first"] else None
    start = (ln - nq) // BLOCK * BLOCK
    back = ln - start
    s["start"] = torch.from_numpy(start).cuda().to(torch.int32)
    s["cu_back"] = torch.from_numpy(np.concatenate([[0], np.cumsum(back)])).cuda().to(torch.int32)
    s["max_blocks"] = int((-(-back // BLOCK)).max())
    # what comes out of the cache is read in 16 bits
    s["k_back"] = torch.empty((int(back.sum()), H, D), dtype=torch.float16 if case["dtype"] == "f32" else dtype, device="cuda")
    s["v_back"] = torch.empty_like(s["k_back"])


def _prepare_select(case, g, s):
    G, B, V = case["groups"], case["beams"], case["vocab"]
    full = _normal(g, (G * B, V + case["pad"])) * 2.5
    full[:, :V].scatter_add_(1, torch.randint(0, V, (G * B, 24), generator=g, device="cuda"), 4 * torch.rand((G * B, 24), generator=g, device="cuda"))
    if case["masked"]:  # a grammar forbids part of the vocabulary
        full[torch.rand(full.shape, generator=g, device="cuda") < case["masked"]] = -math.inf
    s["logits"] = full.to(TYPES[case["dtype"]])[:, :V]
    s["scores"] = -4 * torch.rand((G, B), generator=g, device="cuda")
    if case["dead"]:  # a search's first step has one beam
        s["scores"][::2, 1:] = -math.inf
    s["stop"] = int(s["logits"][0].argmax())  # a token that does come out
    n = 2 * B
    s["cand"] = [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    s["next"] = [torch.empty((G, B), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]


def _prepare_reorder(case, g, s):
    prompt, since, parent = _beams(case)
    T, G, B = case["page"], case["groups"], case["beams"]
    total, full = prompt + since, prompt // T  # the prompt's full pages are shared by the beams
    mine = -(-total // T) - full
    at = np.cumsum(full + B * mine) - (full + B * mine)
    slot = np.arange(int((-(-total // T)).max()) + 1)[None, None]
    beam = np.arange(B)[None, :, None]
    table = np.where(slot < full[:, None, None], at[:, None, None] + slot, at[:, None, None] + full[:, None, None] + beam * mine[:, None, None] + slot - full[:, None, None])
    table = np.where(slot < (full + mine)[:, None, None], table, -1).reshape(G * B, -1)
    n_pages = int((full + B * mine).sum()) + G * B + 2
    _, slab, page_bytes = _geometry(case)
    s["pool"] = torch.randint(0, 256, (n_pages, page_bytes), generator=g, device="cuda", dtype=torch.uint8)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.from_numpy(table).cuda()
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0)], -1).to(torch.int32)
    s["lens"] = torch.from_numpy(np.repeat(total, B)).cuda().to(torch.int32)
    s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(), minlength=n_pages).to(torch.int32)
    s["parent"] = torch.from_numpy(parent).cuda().to(torch.int32)


def _kept(s):
    """What a user of the library keeps from call to call: descriptions, the rotation's plan, workspaces, a plane."""
    if "kept" not in s:
        from quantized_q8_activation_quantize_gb300 import binding, decoder, kv
        c = s["case"]
        s["kept"] = (binding, decoder, kv)
        if c["op"] == "add":
            s["plane"] = binding.alloc_plane(c["rows"], c["width"])
            s["sections"] = {"gemm": binding.PLANE_FOR_GEMM, "gemv": binding.PLANE_FOR_GEMV}[c["use"]]
        if c["op"] in ("rope", "append"):
            more = {"turns": {"low": 1.0, "high": 4.0}, "index": {"low": 1.0, "high": 32.0}}.get(c["scaling"], {})
            s["plan"] = decoder.rope_plan(c["rot"], c["base"], interleaved=c["interleaved"], scaling=c["scaling"], factor=c["factor"],
                                          original=c["original"], amplitude=_amplitude(c), **more)
        if c["op"] in ("append", "reorder"):
            s["cache"] = kv.cache(s["pool"], s["refs"], c["layers"], c["kv_heads"], c["dim"], c["page"])
            s["seqs"] = kv.sequences(s["table"], s["lens"])
        if c["op"] == "reorder":
            s["ws"] = kv.alloc_pages_workspace(s["cache"], s["seqs"])
        if c["op"] == "select":
            s["ws"] = decoder.alloc_beam_workspace(c["groups"], c["beams"], c["vocab"], 2 * c["beams"])
    return s["kept"]


def run(s):
    return {"add": _run_add, "rope": _run_rope, "append": _run_append, "select": _run_select, "reorder": _run_reorder}[s["case"]["op"]](s)


# ------------------------------------------------------- addition, norm, plane ---

def _run_add(s):
    """h = x + res and the Q8 plane of RMSNorm(h) w, as the values that its codes stand for."""
    if own:
        _, decoder, _ = _kept(s)
        decoder.mqd_add_quantize_q8(s["x"], s["res"], s["h"], s["w"], EPS, s["sections"], s["plane"])
        decoder.mqd_dequantize_q8(s["plane"], s["sections"], s["back"])
        return s["h"], s["back"]
    h = (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    y = h.float()
    # values next to a border between two codes: the factor in 64 bits, rounded once
    r = (1 / torch.sqrt(y.double().square().mean(1, keepdim=True) + np.float32(EPS).astype(np.float64))).float()
    y = ((y * r) * s["w"]).unflatten(1, (-1, BLOCK))
    d = y.abs().amax(2, keepdim=True) / torch.full((), 127.0, device="cuda")
    q = _away((y * torch.where(d > 0, 1 / d, 0.0)).double()).clamp(-127, 127).float()
    return h, (q * d).flatten(1).to(s["back"].dtype)


def _away(y):
    return torch.trunc(y + torch.copysign(torch.full_like(y, 0.5), y))


# ------------------------------------------------------------- rotary positions ---

def _rotated(case, x, pos, freq):
    """x [tokens, heads, dim] in 32 bits, rotated; the angles in 64."""
    angle = pos.double()[:, None, None] * freq
    a = _amplitude(case)
    c, s = (angle.cos() * a).float(), (angle.sin() * a).float()
    rot = case["rot"]
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = u * c - v * s, v * c + u * s
    y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _run_rope(s):
    if own:
        _, decoder, _ = _kept(s)
        decoder.mqd_rope(s["plan"], s["x"], s["out"], s["pos"])
        return s["out"]
    return _rotated(s["case"], s["x"].float(), s["pos"], s["freq"]).to(s["x"].dtype)


def _run_append(s):
    case = s["case"]
    if own:
        _, _, kv = _kept(s)
        kv.mqkv_append_rope(s["cache"], s["seqs"], s["layer"], s["plan"], s["q"], s["out"], s["k"], s["v"], s["cu"], s["pos"])
        kv.mqkv_read(s["cache"], s["seqs"], s["layer"], s["k_back"], s["v_back"], s["cu_back"], s["start"])
        return s["out"], s["k_back"], s["v_back"]
    T, n = case["page"], case["seqs"]
    lens, cu, start = s["lens"].long(), s["cu"].long(), s["start"].long()
    new = cu.diff()
    first = lens - new - start  # slots of the first block that hold earlier tokens
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b] + first[b]
    where = (lens - new)[b] + t - cu[b] if s["pos"] is None else s["pos"]
    q_out = _rotated(case, s["q"].float(), where, s["freq"]).to(s["q"].dtype)
    x = torch.zeros((n, s["max_blocks"] * BLOCK, 2, case["kv_heads"], case["dim"]), device="cuda")
    x[b, i] = torch.stack([_rotated(case, s["k"].float(), where, s["freq"]), s["v"].float()], 1)
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
    inv = torch.where(d > 0, 1.0 / d, 0.0)[:, :, None, :, :, None]
    shrink = torch.where(d > d0, d0 / d, 1.0)[:, :, None, :, :, None]
    q = torch.where(live[..., None, None, None], _away(x * inv).clamp(-127, 127), _away(q0 * shrink))
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
    kv = ((codes[page, :, :, slot].float() - 128.0) * scales[page, :, :, slot // BLOCK][..., None]).to(s["k_back"].dtype)
    return q_out, kv[:, 0], kv[:, 1]


# ------------------------------------------------------------------ beam search ---

def _run_select(s):
    """The 2 B best continuations of every group (score, row of the beam, token), and of those that do not end the best B."""
    case = s["case"]
    if own:
        _, decoder, _ = _kept(s)
        decoder.mqd_beam_select(s["logits"], s["scores"], s["cand"], s["next"], s["stop"], s["ws"])
        return *s["cand"], *s["next"]
    G, B, V = case["groups"], case["beams"], case["vocab"]
    x = s["logits"].double()  # scores of different beams may lie next to each other
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    logp = x - (m + torch.log(torch.exp(x - m).sum(1, keepdim=True)))
    total = torch.where(x == -math.inf, -math.inf, s["scores"].double().view(-1, 1) + logp).view(G, B * V)
    score, at = torch.sort(total, dim=1, descending=True, stable=True)  # of equals the lowest place
    score, at = score[:, :2 * B], at[:, :2 * B]
    none = score == -math.inf
    base = torch.arange(G, device="cuda")[:, None] * B
    row, token = torch.where(none, -1, at // V + base), torch.where(none, -1, at % V)
    keep = torch.argsort((none | (token == s["stop"])).int(), dim=1, stable=True)[:, :B]
    ends = (none | (token == s["stop"])).gather(1, keep)
    nxt = [torch.where(ends, e, v.gather(1, keep)) for v, e in ((score, -math.inf), (row, -1), (token, -1))]
    return score.float(), row.int(), token.int(), nxt[0].float(), nxt[1].int(), nxt[2].int()


def _run_reorder(s):
    """Every row's sequence becomes the one that its beam continues."""
    case = s["case"]
    if own:
        _, _, kv = _kept(s)
        kv.mqkv_reorder(s["cache"], s["seqs"], s["parent"], s["ws"])
    else:
        T = case["page"]
        table, lens, parent = s["table"].long(), s["lens"].long(), s["parent"].long()
        from_ = parent.clamp(min=0)
        ln = torch.where(parent >= 0, lens[from_], 0)
        order = torch.argsort(parent, stable=True)
        again = torch.zeros_like(parent, dtype=torch.bool)
        again[order[1:]] = parent[order[1:]] == parent[order[:-1]]  # the first row that continues a sequence keeps its last page
        slot = torch.arange(table.shape[1], device="cuda")[None]
        full, part = ln // T, ln % T > 0
        copy = again & part
        tail = (slot == full[:, None]) & copy[:, None]
        held = slot < ((lens + T - 1) // T)[:, None]
        share = (slot < ((ln + T - 1) // T)[:, None]) & ~tail
        old = table[from_]
        refs = s["refs"].index_add(0, table.clamp(min=0).flatten(), -held.int().flatten()).index_add(0, old.clamp(min=0).flatten(), share.int().flatten())
        free = torch.argsort((refs > 0).int(), stable=True)  # the free pages, the lowest first
        page = free[(copy.long().cumsum(0) - 1).clamp(min=0)]
        refs = refs.index_add(0, page, copy.int())
        s["table"].copy_(torch.where(share, old, torch.where(tail, page[:, None], -1)))
        s["lens"].copy_(ln), s["refs"].copy_(refs)
        # the used blocks of the last pages, and all of their scales; a row without a copy repeats the first one, or moves page 0 onto itself
        like = torch.where(copy, torch.arange(parent.numel(), device="cuda"), copy.int().argmax())
        src = old.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0][like]
        src, dst = torch.where(copy.any(), src, 0), torch.where(copy.any(), page[like], 0)
        blocks = torch.arange(T, device="cuda") // BLOCK * BLOCK < (ln % T)[like][:, None]
        codes, scales = _codes(case, s["pool"]), _scales(case, s["pool"])
        codes[dst] = torch.where(blocks[:, None, None, None, :, None], codes[src], codes[dst])
        scales[dst] = scales[src]
    # page memory as the 32-bit words that are copied
    return s["table"], s["lens"], s["refs"], s["pool"].view(torch.int32)


# ---------------------------------------------------------------------- work ---

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}.get(case.get("dtype"))
    if case["op"] == "add":
        n = case["rows"] * case["width"]
        # x and the residual in, h out; the plane's codes and block values out and in again, the values out
        plane = {"gemm": 2 + 16 / BLOCK, "gemv": 1 + 8 / BLOCK}[case["use"]]
        back = {"gemm": 2 + 4 / BLOCK, "gemv": 1 + 4 / BLOCK}[case["use"]]
        return {"bytes": n * (3 * size + plane + back + 2) + 4 * case["width"], "flops": 9 * n}
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"] + 20 * case["tokens"] * case["rot"]}
    if case["op"] == "append":
        ln, nq = _lengths(case)
        new, back = int(nq.sum()), int((ln - (ln - nq) // BLOCK * BLOCK).sum())
        per, n = 2 * case["kv_heads"] * case["dim"], int(nq.sum()) * case["heads"]
        # q in and out; the new values in, their codes out, and what earlier tokens share their block with in and out again; then all of it read back
        return {"bytes": 2 * n * case["dim"] * size + per * (new * (size + 1) + 2 * (back - new) + back * 3),
                "flops": 3 * (n + new * case["kv_heads"]) * case["rot"] + 20 * new * case["rot"] + per * (4 * new + back)}
    if case["op"] == "select":
        rows = case["groups"] * case["beams"]
        return {"bytes": rows * (case["vocab"] * size + 4 + 36), "flops": 4 * rows * case["vocab"]}
    prompt, since, parent = _beams(case)
    T, B = case["page"], case["beams"]
    ln = np.repeat(prompt + since, B)
    again = np.array([p >= 0 and p in parent[:i] for i, p in enumerate(parent)])
    part = ln[np.maximum(parent, 0)] % T
    blocks = (-(-part // BLOCK) * BLOCK)[again & (part > 0)]
    per = 2 * case["kv_heads"] * case["layers"]
    return {"bytes": float(2 * (blocks * per * case["dim"] + per * (T // BLOCK) * 4).sum() + 8 * (-(-ln // T)).sum()), "flops": 0}


# --------------------------------------------------------------------- exact ---

def exact(case, seed):
    """The definitions in 64 bits."""
    if case["op"] == "reorder":
        return None  # nothing is computed: bytes move
    s = prepare(case, seed)
    return {"add": _exact_add, "rope": _exact_rope, "append": _exact_append, "select": _exact_select}[case["op"]](case, s)


def _exact_add(case, s):
    h = s["x"].double() + s["res"].double()
    back = torch.empty_like(h)
    for lo in range(0, case["rows"], 1024):
        y = h[lo:lo + 1024].to(s["x"].dtype).double()  # the norm is of the stream as it is stored
        y = y * torch.rsqrt(torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / case["width"] + float(np.float32(EPS))) * s["w"].double()
        blocks = y.reshape(y.shape[0], -1, BLOCK)
        d = (blocks.abs().max(2, keepdim=True).values / 127).float().double()  # a block's scale is one number in 32 bits
        q = blocks / torch.where(d > 0, d, 1.0)
        back[lo:lo + 1024] = (torch.sign(q) * torch.floor(q.abs() + 0.5) * d).view(y.shape)
    return h, back


def _exact_rope(case, s, x=None, pos=None):
    """Pair by pair, as complex numbers."""
    x = (s["x"] if x is None else x).double()
    pos = (s["pos"] if pos is None else pos).double()
    freq, out, rot = _frequencies(case), x.clone(), case["rot"]
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        z = torch.complex(x[:, :, a], x[:, :, b]) * torch.polar(torch.full_like(pos, _amplitude(case)), pos * float(f))[:, None]
        out[:, :, a], out[:, :, b] = z.real, z.imag
    return out


def _exact_append(case, s):
    f8 = torch.float64
    H, D, T, layer = case["kv_heads"], case["dim"], case["page"], s["layer"]
    off_s, slab, _ = _geometry(case)
    table, lens, cu, cub, start = (s[k].cpu().numpy() for k in ("table", "lens", "cu", "cu_back", "start"))
    pos = s["pos"]
    if pos is None:
        pos = torch.cat([torch.arange(int(lens[b]) - int(cu[b + 1] - cu[b]), int(lens[b]), device="cuda") for b in range(case["seqs"])])

    def history(b, lo, n, h, half):
        """Tokens lo .. n of a sequence's K (half 0) or V (1) of one head, of one block of 32: codes and their scale."""
        base = s["pool"].view(-1, case["layers"], slab)[int(table[b, lo // T]), layer]
        at = lo % T
        q = base[(half * H + h) * T * D:][at * D:(at + n - lo) * D].reshape(-1, D).to(f8) - 128
        d = base[off_s + ((half * H + h) * (T // BLOCK) + at // BLOCK) * 4:][:4].contiguous().view(torch.float32)
        return q, d.to(f8)

    back = [torch.empty(s["k_back"].shape, dtype=f8, device="cuda") for _ in range(2)]
    for half, x in enumerate((_exact_rope(case, s, s["k"], pos), s["v"].double())):
        for b in range(case["seqs"]):
            n, before, first = int(lens[b]), int(lens[b]) - int(cu[b + 1] - cu[b]), int(start[b])
            new = x[int(cu[b]):int(cu[b + 1])]
            old = torch.empty((before - first, H, D), dtype=f8, device="cuda")
            d_old = torch.zeros(H, dtype=f8, device="cuda")
            for h in range(H if before > first else 0):
                q, d = history(b, first, before, h, half)
                old[:, h], d_old[h] = q * d, d[0]
            pad = -(-(n - first) // BLOCK) * BLOCK - (n - first)
            blocks = torch.cat([old, new, torch.zeros((pad, H, D), dtype=f8, device="cuda")]).view(-1, BLOCK, H, D)
            kept = blocks.clone()
            kept[0, :before - first] = 0
            d = (kept.abs().amax((1, 3)) / 127).float().to(f8)  # a block's scale is one number in 32 bits
            d[0] = torch.maximum(d[0], d_old)
            y = blocks / torch.where(d > 0, d, 1.0)[:, None, :, None]
            q = (torch.sign(y) * torch.floor(y.abs() + 0.5)).clamp(-127, 127)
            back[half][int(cub[b]):int(cub[b + 1])] = (q * d[:, None, :, None]).view(-1, H, D)[:n - first]
    return _exact_rope(case, s, s["q"], pos), *back


def _exact_select(case, s):
    """Group by group, the best of every beam first and then of those."""
    G, B, V = case["groups"], case["beams"], case["vocab"]
    cand = [torch.empty((G, 2 * B), dtype=t, device="cuda") for t in (torch.float64, torch.int32, torch.int32)]
    for a in range(G):
        best = []
        for b in range(a * B, a * B + B):
            x = s["logits"][b].double()
            logp = torch.log_softmax(x, 0)
            k = min(2 * B, V)
            edge = torch.topk(x, k).values[-1]
            at = torch.nonzero((x >= edge) & (x > -math.inf))[:, 0].tolist()
            base = float(s["scores"].view(-1)[b])
            best += [(-(base + p), b, t) for p, t in zip(logp[at].tolist(), at) if base > -math.inf]
        best = sorted(best)[:2 * B] + [(math.inf, -1, -1)] * 2 * B
        for out, col in zip(cand, zip(*best[:2 * B])):
            out[a] = torch.tensor(col, dtype=torch.float64, device="cuda").to(out.dtype)
    cand[0].neg_()
    go = [[(v, r, t) for v, r, t in zip(*rows) if r >= 0 and t != s["stop"]][:B] for rows in zip(*(c.tolist() for c in cand))]
    nxt = [torch.empty((G, B), dtype=c.dtype, device="cuda") for c in cand]
    for a, rows in enumerate(go):
        for out, col in zip(nxt, zip(*(rows + [(-math.inf, -1, -1)] * B)[:B])):
            out[a] = torch.tensor(col, dtype=torch.float64, device="cuda").to(out.dtype)
    return *cand, *nxt

"""GPU parity of include/mqd.h and of the cache's turned append and reordering: planes, codes, tables bit for bit; values and scores within bounds
that follow from the number formats, against the formulas in 64 bits."""
import numpy as np
import pytest

import oracle
from quantized_q8_activation_quantize_gb300 import binding as B
from quantized_q8_activation_quantize_gb300 import decoder as dec
from quantized_q8_activation_quantize_gb300 import kv
from tests import kv_util as U
from tests.test_gpu_kv import TYPES, Setup, cu_of, dev, i32, status, ttype

pytestmark = pytest.mark.gpu

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}          # half a step, relative


def bits(t):
    import torch
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


def same(a, b):
    import torch
    assert a.dtype == b.dtype and a.shape == b.shape
    assert torch.equal(bits(a), bits(b)), f"{int((bits(a) != bits(b)).sum())} of {a.numel()} differ, first at {(bits(a) != bits(b)).nonzero()[:3].tolist()}"


def sync():
    import torch
    torch.cuda.synchronize()
    B.mq_device_status()


# ------------------------------------------------------------------ residual, RMSNorm, Q8 plane ---

def stream_of(M, K, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda") * 0.7
    res = torch.randn((M, K), generator=g, device="cuda")
    res[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20
    w = 1 + 0.1 * torch.randn(K, generator=g, device="cuda")
    return x.to(ttype(dtype)), res.to(ttype(dtype)), w


# one warp to a whole block per row; few rows (a warp for every chunk), many, and rows past the registers
SHAPES = [(1, 256), (1, 3584), (5, 512), (7, 768), (304, 1280), (305, 1280), (333, 3584), (2, 8192), (400, 8192), (3, 8448), (37, 20480), (1, 18944), (613, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", SHAPES)
def test_add_quantize_equals_addition_then_quantize(M, K, dtype):
    import torch
    x, res, w = stream_of(M, K, dtype, M + K)
    x[0, :32], res[0, :32] = 0, 0                              # a block of zeros
    h, plane = torch.empty_like(x), B.alloc_plane(M, K)
    dec.mqd_add_quantize_q8(x, res, h, w, 1e-6, B.PLANE_ALL, plane)
    want_h = (x.float() + res.float()).to(x.dtype)
    want = B.alloc_plane(M, K)
    B.mq_quantize_q8(want_h.float().contiguous(), M, K, w, 1e-6, want)
    sync()
    same(h, want_h)
    for a, b in zip(B.plane_views(plane, M, K, with_ds=True), B.plane_views(want, M, K, with_ds=True)):
        same(a, b)


def test_add_quantize_matches_the_oracle():
    import torch
    x, res, w = stream_of(9, 1536, "f32", 3)
    h, plane = torch.empty_like(x), B.alloc_plane(9, 1536)
    dec.mqd_add_quantize_q8(x, res, h, w, 1e-5, B.PLANE_ALL, plane)
    sync()
    q, d, s = oracle.quantize_q8((x + res).cpu().numpy(), w.cpu().numpy(), 1e-5)
    _, q8, dg, sg = B.plane_views(plane, 9, 1536)
    assert np.array_equal(q8.cpu().numpy(), q) and np.array_equal(dg.t().cpu().numpy(), d) and np.array_equal(sg.t().cpu().numpy(), s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(3, 512), (320, 2048), (4, 9216)])
def test_add_quantize_in_place_strided_and_without_addition(M, K, dtype):
    import torch
    x, res, w = stream_of(M, K, dtype, 17)
    want_h = (x.float() + res.float()).to(x.dtype)

    def plane_of(t):
        p = B.alloc_plane(M, K)
        B.mq_quantize_q8(t.float().contiguous(), M, K, w, 1e-6, p)
        return B.plane_views(p, M, K)
    wide = [torch.full((M, K + 24), 7.0, device="cuda", dtype=x.dtype) for _ in range(3)]
    wide[0][:, 8:8 + K], wide[1][:, 16:16 + K] = x, res
    xs, rs, hs = wide[0][:, 8:8 + K], wide[1][:, 16:16 + K], wide[2][:, 8:8 + K]
    before = res.clone()
    for args, out in (((xs, rs, hs), hs), ((xs, rs, rs), rs), ((x, res, x), x)):
        plane = B.alloc_plane(M, K)
        dec.mqd_add_quantize_q8(*args, w, 1e-6, B.PLANE_ALL, plane)
        sync()
        same(out.contiguous(), want_h)
        for a, b in zip(B.plane_views(plane, M, K), plane_of(want_h)):
            same(a, b)
    assert (wide[2][:, :8] == 7).all() and (wide[2][:, 8 + K:] == 7).all() and (wide[1][:, :16] == 7).all() and (wide[1][:, 16 + K:] == 7).all()
    plane = B.alloc_plane(M, K)
    dec.mqd_add_quantize_q8(None, res, None, w, 1e-6, B.PLANE_ALL, plane)
    sync()
    same(res, before)
    for a, b in zip(B.plane_views(plane, M, K), plane_of(res)):
        same(a, b)


@pytest.mark.parametrize("sections", range(1, 8))
@pytest.mark.parametrize("M,K", [(2, 1024), (310, 512), (3, 8704)])
def test_add_quantize_writes_the_sections_it_is_asked_for(M, K, sections):
    import torch
    x, res, w = stream_of(M, K, "bf16", 5)
    h, full, part = torch.empty_like(x), B.alloc_plane(M, K), B.alloc_plane(M, K).fill_(0x5A)
    dec.mqd_add_quantize_q8(x, res, h, w, 1e-6, B.PLANE_ALL, full)
    dec.mqd_add_quantize_q8(x, res, h, w, 1e-6, sections, part)
    sync()
    for bit, a, b in zip((1, 2, 0, 0, 4), B.plane_views(part, M, K, with_ds=True), B.plane_views(full, M, K, with_ds=True)):
        same(a, b if bit == 0 or sections & bit else torch.full_like(bits(b).view(torch.uint8), 0x5A).view(b.dtype))


def test_add_quantize_of_rows_that_are_not_finite():
    import torch
    for M, K in ((6, 512), (400, 512), (6, 8448)):
        x, res, w = stream_of(M, K, "f32", 8)
        x[0, 5], x[1, 6], res[1, 6], x[2, 3], res[2, 3] = float("nan"), 3e38, 3e38, float("inf"), float("-inf")
        x[3], res[3] = 0, 0                                    # r = 1 / sqrt(eps)
        x[4], res[4] = 1e-30, 1e-30
        h, plane, want = torch.empty_like(x), B.alloc_plane(M, K), B.alloc_plane(M, K)
        dec.mqd_add_quantize_q8(x, res, h, w, 1e-6, B.PLANE_ALL, plane)
        B.mq_quantize_q8(x + res, M, K, w, 1e-6, want)
        sync()
        same(torch.nan_to_num(h, nan=1.0), torch.nan_to_num(x + res, nan=1.0))
        for a, b in zip(B.plane_views(plane, M, K), B.plane_views(want, M, K)):
            same(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 256), (9, 1280), (8, 4096), (70, 3584)])
def test_dequantize(M, K, dtype):
    import torch
    x = torch.randn((M, K), device="cuda") * torch.logspace(-6, 3, M, device="cuda")[:, None]
    plane = B.alloc_plane(M, K)
    B.mq_quantize_q8(x, M, K, None, 0.0, plane)
    _, q8, d, _ = B.plane_views(plane, M, K)
    want = (q8.float().unflatten(1, (-1, 32)) * d.t()[:, :, None]).flatten(1).to(ttype(dtype))      # one product in f32, one rounding
    for sections in (1, 2, 7):
        wide = torch.full((M, K + 16), 3.0, device="cuda", dtype=ttype(dtype))
        dec.mqd_dequantize_q8(plane, sections, wide[:, 8:8 + K])
        sync()
        same(wide[:, 8:8 + K].contiguous(), want)
        assert (wide[:, :8] == 3).all() and (wide[:, 8 + K:] == 3).all()


# ----------------------------------------------------------------------------- rotary positions ---

def turned(x, pos, turns, rot, interleaved, amplitude=1.0):
    """The rotation in 64 bits, x [tokens, heads, dim]; the angles from the turns, modulo a turn exactly.  Also |u| + |v| of every value's pair."""
    y, mass = x.astype(np.float64).copy(), np.zeros(x.shape)
    with np.errstate(over="ignore"):
        phase = pos.astype(np.int64).astype(np.uint64)[:, None] * np.array(turns, np.uint64)[None]
    angle = 2 * np.pi * phase.astype(np.float64) / 2.0 ** 64
    c, s = np.cos(angle)[:, None] * amplitude, np.sin(angle)[:, None] * amplitude
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., a].astype(np.float64), x[..., b].astype(np.float64)
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    mass[..., a] = mass[..., b] = (np.abs(u) + np.abs(v)) * abs(amplitude)
    return y, mass


def check_turned(got, x, pos, turns, rot, interleaved, amplitude, dtype):
    y, mass = turned(x.float().cpu().numpy(), pos, turns, rot, interleaved, amplitude)
    # cos and sin within 1.6e-7 (tests/test_decoder_host.py), times the amplitude, two products and a sum, each rounded to f32 (half a step: 2^-24 of
    # the terms); then the output's own rounding (f16 below 2^-14: 2^-25)
    tol = mass * (1.6e-7 + 4 * 2.0 ** -24) + UNIT[dtype] * np.abs(y) * 1.001 + (2.0 ** -25 if dtype == "f16" else 1e-38)
    tol[mass == 0] = 0                                         # past rot_dim: as they were
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - y)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 8, 8), (5, 28, 128, 128), (3, 7, 128, 64), (9, 3, 80, 32), (2, 4, 96, 72), (700, 5, 64, 64), (650, 2, 256, 256),
                                                  (4, 2, 1024, 1024), (611, 3, 128, 104), (640, 1, 24, 16)])
def test_rope(tokens, heads, dim, rot, interleaved, dtype):
    import torch
    r = np.random.default_rng(tokens + dim)
    x = torch.from_numpy(r.standard_normal((tokens, heads, dim)).astype(np.float32)).to(ttype(dtype)).cuda()
    pos = r.integers(-2 ** 31, 2 ** 31, tokens).astype(np.int32)
    pos[:4] = [0, 1, 2 ** 31 - 1, -2 ** 31][:min(4, tokens)]
    plan = dec.rope_plan(rot, 10000.0, interleaved=interleaved, amplitude=1.25)
    turns = dec.mqd_rope_turns(rot, 10000.0)
    out = torch.full_like(x, 5.0)
    dec.mqd_rope(plan, x, out, dev(pos))
    sync()
    check_turned(out, x, pos, turns, rot, interleaved, 1.25, dtype)
    # strided both ways (heads outermost on one side), then in place: the same bits
    buf = torch.full((heads, tokens, dim + 4), 9.0, device="cuda", dtype=x.dtype)
    xs = torch.zeros((tokens, heads + 3, dim + 4), device="cuda", dtype=x.dtype)
    xs[:, 1:1 + heads, :dim] = x
    dec.mqd_rope(plan, xs[:, 1:1 + heads, :dim], buf.transpose(0, 1)[:, :, :dim], dev(pos))
    y = x.clone()
    dec.mqd_rope(plan, y, y, dev(pos))
    sync()
    same(buf.transpose(0, 1)[:, :, :dim].contiguous(), out)
    same(y, out)
    assert (buf[:, :, dim:] == 9).all()


def test_rope_far_positions_and_back():
    import torch
    kw = dict(scaling="turns", factor=8.0, original=8192.0)
    plan, turns = dec.rope_plan(128, 500000.0, **kw), dec.mqd_rope_turns(128, 500000.0, **kw)
    x = torch.randn((64, 2, 128), device="cuda")
    pos = np.arange(64, dtype=np.int32) + 1_000_000
    out = torch.empty_like(x)
    dec.mqd_rope(plan, x, out, dev(pos))
    sync()
    check_turned(out, x, pos, turns, 128, False, 1.0, "f32")
    dec.mqd_rope(plan, out, out, dev(-pos))                    # turned back
    sync()
    # two rotations, each within the bound above of its pair (of at most |u| + |v| <= sqrt(2) of the pair's length)
    assert float((out - x).abs().max()) < 4 * (1.6e-7 + 4 * 2.0 ** -24) * float(x.abs().max())


# rows that begin past 2^31 elements from the first
def test_rope_of_heads_that_lie_far_apart():
    import torch
    x = torch.zeros((3, (1 << 30) + 64), device="cuda", dtype=torch.float16)
    view = x[:, (1 << 30):(1 << 30) + 64].unsqueeze(1)         # token stride 2^30 + 64
    view.copy_(torch.randn((3, 1, 64), device="cuda"))
    keep = view.clone()
    plan = dec.rope_plan(64)
    pos = np.array([3, 5, 9], np.int32)
    dec.mqd_rope(plan, view, view, dev(pos))
    sync()
    check_turned(view, keep, pos, dec.mqd_rope_turns(64), 64, False, 1.0, "f16")
    assert not x[:, :1 << 30].any()


# (cached before, new): fresh, inside a block, across blocks and pages, ending on boundaries, none at all
RAGGED = [(0, 1), (0, 33), (5, 1), (31, 2), (63, 70), (100, 0), (0, 0), (17, 300), (256, 1), (300, 5), (4096, 3)]


def check_append_rope(had, new, heads, kv_heads, dim, page, dtype, rot, interleaved, given, before=0, after=0, layers=2):
    """the fused call against mqd_rope and mqkv_append, bit for bit"""
    import torch
    r = np.random.default_rng(dim + page + rot)
    lens = [a + n for a, n in zip(had, new)]
    s, t = (Setup(lens, kv_heads, dim, page, layers=layers, seed=3) for _ in range(2))
    n = before + sum(new) + after
    qkv = torch.from_numpy(r.standard_normal((n, heads + 2 * kv_heads, dim)).astype(np.float32)).to(ttype(dtype)).cuda()
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    plan = dec.rope_plan(rot, 10000.0, interleaved=interleaved, amplitude=0.75)
    pos = np.zeros(n, np.int32)
    for at, (a, m) in zip(np.cumsum([0] + list(new)), zip(had, new)):
        pos[before + at:before + at + m] = np.arange(a, a + m)
    if given:
        pos = r.integers(-2 ** 31, 2 ** 31, n).astype(np.int32)
    cu = i32(before + np.concatenate([[0], np.cumsum(new)]))
    out = torch.full((n, heads, dim), 4.0, device="cuda", dtype=qkv.dtype)
    kv.mqkv_append_rope(s.cache, s.seqs, 1, plan, q, out, k, v, cu, dev(pos) if given else None)
    # as it should be: the keys in f32, appended from there
    kf = torch.empty((n, kv_heads, dim), device="cuda")
    dec.mqd_rope(plan, k.float(), kf, dev(pos))
    want = torch.full_like(out, 4.0)
    live = slice(before, before + sum(new))
    dec.mqd_rope(plan, q[live], want[live], dev(pos[live]))
    kv.mqkv_append(t.cache, t.seqs, 1, kf, v.float(), cu)
    status()
    same(out, want)
    same(s.pool, t.pool)
    # in place, in the projection's own buffer; without queries
    rest = torch.cat([q[:before], q[before + sum(new):]]).clone()
    t.pool.copy_(dev(t.m.bytes(fill=0xFF)))
    kv.mqkv_append_rope(t.cache, t.seqs, 1, plan, q, q, k, v, cu, dev(pos) if given else None)
    status()
    same(q[live].contiguous(), want[live].contiguous())
    same(torch.cat([q[:before], q[before + sum(new):]]), rest)
    same(s.pool, t.pool)
    t.pool.copy_(dev(t.m.bytes(fill=0xFF)))
    kv.mqkv_append_rope(t.cache, t.seqs, 1, plan, None, None, k, v, cu, dev(pos) if given else None)
    status()
    same(s.pool, t.pool)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim,page,rot,interleaved", [(28, 4, 128, 64, 128, False), (9, 3, 64, 32, 64, True), (8, 1, 128, 256, 96, False), (5, 5, 128, 64, 72, True),
                                                                     (3, 1, 64, 128, 24, False)])
@pytest.mark.parametrize("given", [False, True])
def test_append_rope(heads, kv_heads, dim, page, rot, interleaved, dtype, given):
    had, new = zip(*RAGGED)
    check_append_rope(had, new, heads, kv_heads, dim, page, dtype, rot, interleaved, given)


@pytest.mark.parametrize("dtype", TYPES)
def test_append_rope_of_many_tokens_and_rows_of_no_sequence(dtype):
    # enough for four blocks to a CTA and four tokens to a block of queries
    check_append_rope([5, 40, 7, 31, 0, 96, 64, 1001], [1700, 1, 0, 33, 128, 129, 2900, 500], 4, 16, 64, 64, dtype, 48, False, False, before=300, after=9, layers=2)


def test_append_rope_one_token_each_without_cu():
    import torch
    had = [0, 31, 32, 500, 63]
    s, t = (Setup([a + 1 for a in had], 2, 128, 32, seed=5) for _ in range(2))
    q, k, v = (torch.randn((5, h, 128), device="cuda") for h in (8, 2, 2))
    plan, out, want, kt = dec.rope_plan(128), torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    kv.mqkv_append_rope(s.cache, s.seqs, 0, plan, q, out, k, v)
    dec.mqd_rope(plan, q, want, i32(had))
    dec.mqd_rope(plan, k, kt, i32(had))
    kv.mqkv_append(t.cache, t.seqs, 0, kt, v)
    status()
    same(out, want)
    same(s.pool, t.pool)


def test_append_rope_bad_lengths_and_pages():
    import torch
    had, new = [40, 33, 70, 10], [3, 2, 4, 1]
    s = Setup([a + n for a, n in zip(had, new)], 2, 64, 32, seed=6)
    q, k, v = (torch.randn((10, h, 64), device="cuda") for h in (4, 2, 2))
    plan = dec.rope_plan(64)
    s.len[1] = 1                                               # fewer than the new tokens
    s.table[2, 2] = -5                                         # the page of the third's new tokens
    s.len[3] = 10 ** 6                                         # past the table row
    out = torch.full_like(q, 4.0)
    kv.mqkv_append_rope(s.cache, s.seqs, 0, plan, q, out, k, v, cu_of(new))
    status("length")
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(had, new)]).astype(np.int32)
    want = torch.empty_like(q)
    dec.mqd_rope(plan, q, want, dev(pos))
    sync()
    same(out[:3], want[:3])
    same(out[5:9], want[5:9])
    assert (out[3:5] == 0).all() and (out[9:] == 0).all()
    y = q.clone()                                              # in place just the same
    kv.mqkv_append_rope(s.cache, s.seqs, 0, plan, y, y, k, v, cu_of(new))
    status("pool")
    same(y, out)


def test_append_rope_keys_that_are_not_finite():
    import torch
    s, t = (Setup([40], 1, 64, 32, seed=7) for _ in range(2))
    q, k, v = (torch.randn((3, 1, 64), device="cuda") for _ in range(3))
    k[0, 0, 5], k[1, 0, 40] = float("nan"), float("inf")
    plan, kt, pos = dec.rope_plan(64), torch.empty_like(k), i32([37, 38, 39])
    kv.mqkv_append_rope(s.cache, s.seqs, 0, plan, q, torch.empty_like(q), k, v)
    dec.mqd_rope(plan, k, kt, pos)
    kv.mqkv_append(t.cache, t.seqs, 0, kt, v)
    status()
    same(s.pool, t.pool)


# -------------------------------------------------------------------------------- beam search ---

def select(logits, scores, n_cand, stop=-1, next=True):
    import torch
    G, Bm = scores.shape
    V = logits.shape[1]
    cand = [torch.full((G, n_cand), 77, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    nxt = [torch.full((G, Bm), 77, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)] if next else None
    dec.mqd_beam_select(logits, scores, cand, nxt, stop, dec.alloc_beam_workspace(G, Bm, V, n_cand))
    sync()
    return [c.cpu().numpy() for c in cand], [c.cpu().numpy() for c in nxt] if next else None


def check_select(logits, scores, n_cand, stop=-1):
    """Against the definition in 64 bits.

    A row's logarithm: every exponential is off by at most 2^-22 (ex2) and 2^-23 |x - max| in its argument (at most 2^-23 * 20 for what counts: less than e^-20 of
    the sum is beyond), sums of 16, 8 and 5 + 8 terms in f32 by 2^-24 each: less than 6e-6 in all.  Scores then have one rounding to f32.  The kernel's order may differ from the
    definition's only between rows, within that: each place's true score is the definition's of that place, and within a row the order is exact."""
    cand, nxt = select(logits, scores, n_cand, stop)
    G, Bm = scores.shape
    x = logits.float().cpu().numpy().astype(np.float64)
    x[np.isnan(x)] = -np.inf
    x = np.minimum(x, np.finfo(np.float32).max)
    cum = scores.cpu().numpy().astype(np.float64)
    for g in range(G):
        rows, V = x[g * Bm:(g + 1) * Bm], x.shape[1]
        m = rows.max(1, keepdims=True)
        m0 = np.where(np.isfinite(m), m, 0)
        with np.errstate(divide="ignore", invalid="ignore"):
            # the largest first: at 1e30 even 64 bits would lose the logarithm beside it
            base = cum[g][:, None] + ((rows - m0) - np.log(np.exp(rows - m0).sum(1, keepdims=True)))
        base = np.where(np.isneginf(rows) | ~(cum[g][:, None] > -np.inf), -np.inf, base)
        flat = base.reshape(-1)
        order = np.lexsort((np.arange(flat.size), -flat))[:n_cand]
        want = flat[order]
        want = np.concatenate([want, np.full(n_cand - len(want), -np.inf)])
        sc, row, tok = (c[g] for c in cand)
        none = np.isneginf(want)
        assert np.array_equal(row == -1, none) and np.array_equal(tok == -1, none) and np.isneginf(sc[none]).all()
        at = (row - g * Bm)[~none] * V + tok[~none]
        assert len(set(at.tolist())) == len(at) and (at >= 0).all() and (at < flat.size).all()
        true, top = flat[at], want[~none]
        tol = 6e-6 + 2.0 ** -24 * np.abs(top)
        assert (np.abs(true - top) <= 2 * tol).all() and (np.abs(sc[~none] - top) <= 2 * tol).all()
        for b in range(Bm):                                    # within a row: by logit, then by token, and none left out
            mine = tok[~none][(row - g * Bm)[~none] == b]
            best = np.lexsort((np.arange(V), -rows[b]))[:len(mine)]
            assert np.array_equal(mine, best)
        if np.diff(-top).size and np.diff(-top).min() > 2 * tol.max():
            assert np.array_equal(at, order[~none])
        go = [(s, r, t) for s, r, t in zip(sc, row, tok) if r >= 0 and t != stop][:Bm]
        go += [(-np.inf, -1, -1)] * (Bm - len(go))
        for got, col in zip(nxt, zip(*go)):
            assert np.array_equal(got[g], np.array(col, got.dtype))
    return cand, nxt


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,Bm,V,n_cand", [(1, 1, 1, 1), (1, 4, 3, 8), (3, 4, 1000, 8), (2, 5, 4097, 10), (1, 4, 152064, 8), (7, 3, 50257, 6), (1, 64, 9001, 64), (40, 2, 33333, 4),
                                          (2, 16, 20011, 32), (1, 1, 100003, 50), (300, 1, 4090, 2), (1, 1, 1 << 20, 64)])
def test_select(G, Bm, V, n_cand, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(G + V)
    pad = V % 5
    logits = (torch.randn((G * Bm, V + pad), generator=g, device="cuda") * 2.5).to(ttype(dtype))
    logits[:, V:] = 1000                                       # not the rows' own
    scores = -4 * torch.rand((G, Bm), generator=g, device="cuda")
    check_select(logits[:, :V], scores, n_cand, stop=int(logits[0, :V].argmax()))


def test_select_rows_at_every_alignment():
    import torch
    for dtype in TYPES:
        buf = torch.randn(9 * 5003 + 16, device="cuda").to(ttype(dtype))
        for off in range(9):
            logits = torch.as_strided(buf, (9, 5000), (5003, 1), off)
            check_select(logits, torch.zeros((3, 3), device="cuda") - torch.arange(3, device="cuda"), 6)


def test_select_ties_masks_and_beams_that_are_not_alive():
    import torch
    inf = float("inf")
    # every value the same: the lowest beam's lowest tokens
    cand, nxt = check_select(torch.zeros((4, 20000), device="cuda"), torch.zeros((1, 4), device="cuda"), 64)
    assert cand[2][0].tolist() == list(range(64)) and (cand[1][0] == 0).all() and nxt[2][0].tolist() == [0, 1, 2, 3]
    for value in (-0.0, 1e30, -1e30, 3e38, 1e-45):
        check_select(torch.full((2, 9000), value, device="cuda"), torch.zeros((1, 2), device="cuda"), 4)
    zeros = torch.zeros((1, 9000), device="cuda")
    zeros[0, ::3] = -0.0                                       # minus zero is zero
    cand, _ = check_select(zeros, torch.zeros((1, 1), device="cuda"), 9)
    assert cand[2][0].tolist() == list(range(9))
    # few values, each many times
    coarse = torch.randint(-3, 4, (6, 30011), device="cuda").float()
    check_select(coarse, torch.zeros((2, 3), device="cuda"), 40)
    check_select(coarse.bfloat16(), torch.zeros((2, 3), device="cuda"), 40)
    # sorted upward and downward: the best of a piece lie together
    ramp = torch.arange(70000, device="cuda").float() / 1000
    check_select(torch.stack([ramp, ramp.flip(0)]), torch.zeros((1, 2), device="cuda"), 64)
    # all of a row's best in one thread's, one warp's part
    spike = torch.randn((2, 50000), device="cuda")
    spike[0, 4096:4160] += 50
    spike[1, 1024 * 7:1024 * 7 + 4] += 50
    check_select(spike, torch.zeros((1, 2), device="cuda"), 32)
    # beams that are not alive, rows without a value, a group without a beam
    logits = torch.randn((8, 7000), device="cuda")
    logits[2] = -inf
    logits[5, 10:] = -inf
    scores = torch.tensor([[0.0, -inf, -1.0, float("nan")], [-inf, -0.5, -inf, -inf]], device="cuda")
    cand, _ = check_select(logits, scores, 16)
    assert (cand[1][1] >= 0).sum() == 10
    cand, nxt = check_select(logits, torch.full((2, 4), -inf, device="cuda"), 5)
    assert (cand[1] == -1).all() and (nxt[2] == -1).all()
    # masks of the type's lowest value are values; infinities and NaN
    for dtype in TYPES:
        low = torch.randn((4, 12345), device="cuda").to(ttype(dtype))
        low[:, 5:] = torch.finfo(low.dtype).min
        check_select(low, torch.zeros((1, 4), device="cuda"), 32)
        odd = torch.randn((4, 12345), device="cuda").to(ttype(dtype))
        odd[0, 77], odd[1, 99], odd[1, 12000], odd[2, :] = inf, float("nan"), -inf, float("nan")
        odd[3, ::2] = float("nan")
        check_select(odd, torch.zeros((1, 4), device="cuda"), 12)


def test_select_scores_that_lie_close():
    import torch
    # beams of the same logits, whose scores differ by less than a step of f32 at the sums' size: 64 bits tell them apart
    x = torch.randn(30000, device="cuda")
    logits = torch.stack([x, x, x])
    scores = torch.tensor([[-100.0, -100.0 + 2.0 ** -17, -100.0 - 2.0 ** -17]], device="cuda")
    cand, _ = check_select(logits, scores, 6)
    assert cand[1][0].tolist() == [1, 0, 2] * 2                # equal rows have equal logarithms, bit for bit


def test_select_is_the_same_every_time_and_in_a_graph():
    import torch
    G, Bm, V, n = 5, 4, 30001, 8
    logits = torch.randn((G * Bm, V), device="cuda") * 3
    scores = -torch.rand((G, Bm), device="cuda")
    first, _ = check_select(logits, scores, n, stop=3)
    for _ in range(5):
        for a, b in zip(select(logits, scores, n, stop=3)[0], first):
            assert np.array_equal(a, b)
    # next_score may be the scores themselves; two steps captured with one workspace, replayed with other logits, on another stream
    cand = [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    row, token = (torch.empty((G, Bm), dtype=torch.int32, device="cuda") for _ in range(2))
    ws, live = dec.alloc_beam_workspace(G, Bm, V, n), scores.clone()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(2):
            dec.mqd_beam_select(logits, live, cand, (live, row, token), 3, ws)
    for seed in (1, 2):
        logits.copy_(torch.randn((G * Bm, V), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        live.copy_(scores)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        _, one = select(logits, scores, n, stop=3)
        _, two = select(logits, dev(one[0]), n, stop=3)
        for a, b in zip((live, row, token), two):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("G, Bm, V, n_cand", [(1, 2, 50001, 64), (1, 1, 9000, 64), (3, 5, 4099, 33), (40, 4, 501, 32), (1, 64, 12289, 64), (2, 16, 20000, 17), (200, 3, 700, 43), (1, 1, 40, 64)])
def test_select_of_many_equal_logits(G, Bm, V, n_cand):
    import torch
    g = torch.Generator(device="cuda").manual_seed(V + n_cand)
    few = torch.randint(-3, 4, (G * Bm, V), generator=g, device="cuda").float()          # seven values
    scores = -torch.rand((G, Bm), generator=g, device="cuda")
    check_select(few.to(torch.bfloat16), scores, n_cand, stop=1)
    few[:] = 1.5                                                                          # and one: the first tokens of the best beam
    cand, _ = check_select(few.half(), scores, n_cand)
    n = min(n_cand, V)
    for i in range(G):
        best = int(scores[i].argmax())
        assert (cand[1][i][:n] == i * Bm + best).all() and np.array_equal(cand[2][i][:n], np.arange(n))
    scores[:] = -0.25                                                                     # equal beams: the lowest row, then the lowest token
    cand, _ = check_select(few.half(), scores, n_cand)
    n = min(n_cand, Bm * V)
    for i in range(G):
        assert np.array_equal(cand[1][i][:n], i * Bm + np.arange(n) // V) and np.array_equal(cand[2][i][:n], np.arange(n) % V)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n_cand", [2, 8, 61, 64])
def test_select_of_rows_that_rise(n_cand, dtype):
    import torch
    # pieces of several tiles, each better than all before it
    x = (torch.arange(60013, device="cuda") * 1e-4).repeat(240, 1)
    x[::3] += 0.3 * torch.rand((80, 60013), generator=torch.Generator(device="cuda").manual_seed(n_cand), device="cuda")
    x[5, ::7], x[6, 1000::1001], x[7, :50000] = float("nan"), float("inf"), -float("inf")
    check_select(x.to(ttype(dtype)), torch.zeros((60, 4), device="cuda") - torch.rand((60, 4), device="cuda"), n_cand, stop=60012)


@pytest.mark.parametrize("Bm,V,n_cand", [(3, 967, 64), (16, 4001, 32), (5, 2049, 33), (2, 200, 64)])
def test_select_of_neighbouring_logits(Bm, V, n_cand):
    # f32 logits one step apart near half a step of the row's logarithm, equal beams: the keys of a list are not in the order of its logits, and lists merge
    import torch
    for up in (2, 5, 9, 30):
        for half in (0.5, 1.0):
            x = np.float32(half * np.spacing(np.float32(np.log(V))))
            row = (np.array(x, np.float32).view(np.int32) + up - np.arange(V)).astype(np.int32).view(np.float32)
            cand, _ = check_select(dev(np.tile(row, (Bm, 1))), torch.full((1, Bm), -1.5, device="cuda"), n_cand)
            assert (cand[1][0] >= 0).all()


def test_select_scores_past_f32():
    import torch
    big, inf = torch.finfo(torch.float32).max, float("inf")
    logits = torch.full((2, 4000), -big, device="cuda")   # (one piece a row: equal scores in the order of their logits)
    logits[0, 7], logits[1, 3000:3003] = big, torch.tensor([1.0, 3.0, 2.0], device="cuda")
    for n_cand in (4, 64):                                     # (entries ranked, lists merged)
        # the second beam, of +inf, keeps it: its tokens in the order of their logits come before all of the first's
        cand, nxt = select(logits, torch.tensor([[0.0, inf]], device="cuda"), n_cand)
        assert (cand[0] == inf).all() and (cand[1] == 1).all() and cand[2][0][:4].tolist() == [3001, 3002, 3000, 0]
        assert (nxt[0] == inf).all() and nxt[2][0].tolist() == [3001, 3002]
        # and where its logits lie 2 FLT_MAX apart
        cand, _ = select(logits, torch.tensor([[inf, 0.0]], device="cuda"), n_cand)
        assert (cand[0] == inf).all() and (cand[1] == 0).all() and cand[2][0][:4].tolist() == [7, 0, 1, 2]


def log_bound(V):
    """What a row's logarithm may be off by.  A value's distance to the largest is passed in up to five steps (its thread's reference, a warp's, a block's, two among
    the pieces) and one for each time its thread's values rose by 4 after it, which is ceil(ln(V / 256) / 4) times at most for what still counts.  Each step's exponential is good to 2^-22 (ex2)
    and its factor rounds by 2^-24; the arguments together are the distance and at most twice 4 more, off by 2^-24 in the difference, 2^-24 in the product and 1.35e-8 in log2(e).
    What lies further than ln V + 1 from the largest has not the weight to count for more.  Sums of 16 in a tree 4 roundings, a warp's 6, a thread's running sum 2 (it keeps its
    roundings, but for tiles that are larger than all before them, each of which doubles it); the others are pairs."""
    steps = 5 + max(0, int(np.ceil(np.log(V / 256) / 4)))
    return (np.log(V) + 9) * (2 * 2.0 ** -24 + 1.35e-8) + steps * (2.0 ** -22 + 2.0 ** -24) + 12 * 2.0 ** -24


def log_error(logits):
    """of every row; the beams' scores are such that the result is near zero and its own rounding does not count"""
    import torch
    R, V = logits.shape
    top, lse = (torch.empty(R, dtype=torch.float64, device="cuda") for _ in range(2))
    for r in range(R):
        x = logits[r].double()
        top[r], lse[r] = x.max(), torch.logsumexp(x, 0)
    cum = (lse - top).float().view(R, 1)
    cand, _ = select(logits, cum, 1, next=False)
    return float(np.abs(cand[0].astype(np.float64).ravel() - (cum.double().view(R) + top - lse).cpu().numpy()).max())


@pytest.mark.parametrize("R,V", [(2, 5000), (4, 152064), (460, 30000), (460, 1 << 22)])       # (460 rows: one block each)
def test_select_logarithms(R, V):
    import torch
    x = torch.empty((R, V), device="cuda")
    for value in (-11.109375, -1.0, -0.3, -5.7, -8.3, -12.3, -16.1, -17.7):   # one peak over many equal logits, whose errors all go the same way
        x.fill_(value)
        x[:, V // 3] = 0
        assert log_error(x) <= log_bound(V), value
    ramp = torch.arange(V, device="cuda") / V
    for rise in (1e-3, 0.1, 1.0, 10.0, 60.0):                                  # every tile a little above the last one
        x.copy_(ramp * rise)
        assert log_error(x) <= log_bound(V), rise
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(V))
    assert log_error(x.mul_(3)) <= log_bound(V)
    assert log_error(x.bfloat16()) <= log_bound(V)


def test_select_rows_past_32_bits_and_heads_of_one_row():
    import torch
    # rows 2^31 + 40 elements apart
    buf = torch.full((2 ** 31 + 40 + 3001,), 7.0, dtype=torch.float16, device="cuda")
    logits = torch.as_strided(buf, (2, 3001), (2 ** 31 + 40, 1), 0)
    logits.copy_(torch.randn((2, 3001), device="cuda") * 2)
    check_select(logits, torch.tensor([[0.0, -0.5]], device="cuda"), 6)
    check_select(logits[:1].expand(3, -1).contiguous(), torch.tensor([[-1.0, -1.0, -1.0]], device="cuda"), 9)      # every score three times


def test_tensors_side_by_side_in_one_buffer():
    import torch
    M, H, D = 9, 3, 64
    K = 2 * 256
    both = torch.randn((M, 2 * K), device="cuda")
    x, h = both[:, :K], both[:, K:]
    res, w = torch.randn((M, K), device="cuda"), torch.ones(K, device="cuda")
    want, kept = x + res, x.clone()
    plane, plain = B.alloc_plane(M, K), B.alloc_plane(M, K)
    dec.mqd_add_quantize_q8(x, res, h, w, 1e-6, B.PLANE_ALL, plane)
    B.mq_quantize_q8(want, M, K, w, 1e-6, plain)
    sync()
    assert torch.equal(h, want) and torch.equal(x, kept)
    assert all(torch.equal(a, b) for a, b in zip(B.plane_views(plane, M, K), B.plane_views(plain, M, K)))
    rows = torch.randn((M, 2 * H, D), device="cuda")
    x, out = rows[:, :H], rows[:, H:]
    kept = x.clone()
    pos = np.arange(M, dtype=np.int32) * 77
    dec.mqd_rope(dec.rope_plan(D), x, out, dev(pos))
    sync()
    assert torch.equal(x, kept)
    check_turned(out, kept, pos, dec.mqd_rope_turns(D), D, False, 1.0, "f32")
    with pytest.raises(B.MQError):
        dec.mqd_add_quantize_q8(both[:, 8:K + 8], res, both[:, :K], w, 1e-6, B.PLANE_ALL, plane)
    with pytest.raises(B.MQError):
        dec.mqd_rope(dec.rope_plan(D), rows[:, :H + 1], rows[:, H - 1:], dev(pos))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, K", [(5, 9216), (2, 16384), (3, 24832), (7, 32768), (3, 33024), (1, 49408)])
def test_add_of_long_rows_in_place(M, K, dtype):
    import torch
    t = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    x, res, w = torch.randn((M, K), device="cuda").to(t), torch.randn((M, K), device="cuda").to(t), 1 + 0.1 * torch.randn(K, device="cuda")
    want = (x.float() + res.float()).to(t)
    plane, plain = B.alloc_plane(M, K), B.alloc_plane(M, K)
    dec.mqd_add_quantize_q8(x, res, x, w, 1e-5, B.PLANE_ALL, plane)
    B.mq_quantize_q8(want.float(), M, K, w, 1e-5, plain)
    sync()
    assert torch.equal(x, want)
    assert all(torch.equal(a, b) for a, b in zip(B.plane_views(plane, M, K), B.plane_views(plain, M, K)))


def test_rope_of_one_head_for_six():
    import torch
    x = torch.randn((5, 1, 64), device="cuda")
    out = torch.empty((5, 6, 64), device="cuda")
    pos = np.arange(5, dtype=np.int32) * 1000
    dec.mqd_rope(dec.rope_plan(64), x.expand(5, 6, 64), out, dev(pos))
    sync()
    check_turned(out, x.expand(5, 6, 64), pos, dec.mqd_rope_turns(64), 64, False, 1.0, "f32")


def test_select_without_next():
    import torch
    cand, nxt = select(torch.randn((6, 999), device="cuda"), torch.zeros((2, 3), device="cuda"), 5, next=False)
    assert nxt is None and (cand[1] >= 0).all()


# ----------------------------------------------------------------------------------- reordering ---

class Pages(U.Pages):
    def reorder(self, parent):
        """the copies made: (source page, page, used blocks); None if the pool is too full (nothing changes)"""
        old = [list(row) for row in self.table], list(self.len), list(self.refs)
        rows, lens, copies, kept = [], [], [], set()
        for row in self.table:
            for p in row:
                self.refs[p] -= 1
        for b, a in enumerate(parent):
            row = list(old[0][a]) if a >= 0 else []
            n = old[1][a] if a >= 0 else 0
            if n % self.T and a in kept:
                copies.append((b, row[-1], -(-(n % self.T) // U.BLOCK)))
                row[-1] = None
            kept.add(a)
            for p in row:
                if p is not None:
                    self.refs[p] += 1
            rows.append(row)
            lens.append(n)
        free = self.free()
        if len(copies) > len(free):
            self.table, self.len, self.refs = old
            return None
        done = []
        for (b, src, blocks), p in zip(copies, free):
            self.refs[p] = 1
            rows[b][-1] = p
            done.append((src, p, blocks))
        self.table, self.len = rows, lens
        return done


class Beams:
    """Rows that share a prompt's pages, as after forks; the device's state beside the model's."""

    def __init__(self, groups, beams, prompts, since, page, heads=2, dim=64, layers=2, spare=4, max_pages=None, seed=0, outside=0):
        r = np.random.default_rng(seed)
        n = groups * beams
        totals = [p + s for p, s in zip(prompts, since)]
        most = max(-(-t // page) for t in totals) + 1
        want = sum(p // page + beams * (-(-t // page) - p // page) for p, t in zip(prompts, totals))
        self.p = Pages(want + spare + outside, n, max_pages or most, page)
        ids = [int(x) for x in r.permutation(want + spare + outside)]
        for g, (p, t) in enumerate(zip(prompts, totals)):
            shared = [ids.pop() for _ in range(p // page)]
            for b in range(g * beams, (g + 1) * beams):
                row = shared + [ids.pop() for _ in range(-(-t // page) - len(shared))]
                self.p.table[b], self.p.len[b] = row, t
                for x in row:
                    self.p.refs[x] += 1
        for _ in range(outside):                               # pages of sequences that are not among the rows
            self.p.refs[ids.pop()] = 3
        self.m = U.Model(want + spare + outside, layers, heads, dim, page)
        self.m.codes[:] = r.integers(-127, 128, self.m.codes.shape)
        self.m.scales[:] = r.uniform(0.01, 1, self.m.scales.shape)
        self.pool = dev(self.m.bytes(fill=0xEE))
        self.refs, self.len = i32(self.p.refs), i32(self.p.len)
        self.table = dev(self.p.table_array())
        self.cache = kv.cache(self.pool, self.refs, layers, heads, dim, page)
        self.seqs = kv.sequences(self.table, self.len)
        self.ws = kv.alloc_pages_workspace(self.cache, self.seqs)

    def reorder(self, parent):
        kv.mqkv_reorder(self.cache, self.seqs, i32(parent), self.ws)
        copies = self.p.reorder(list(parent))
        for s, d, blocks in copies or ():
            self.m.codes[d, :, :, :, :blocks * 32] = self.m.codes[s, :, :, :, :blocks * 32]
            self.m.scales[d] = self.m.scales[s]
        return copies

    def check(self):
        assert self.len.cpu().tolist() == self.p.len
        assert self.refs.cpu().tolist() == self.p.refs
        assert np.array_equal(self.table.cpu().numpy(), self.p.table_array())
        assert np.array_equal(self.pool.cpu().numpy(), self.m.bytes(fill=0xEE))


@pytest.mark.parametrize("groups,beams,page,max_pages", [(1, 4, 64, None), (3, 5, 32, None), (2, 1, 128, None), (40, 4, 32, None), (6, 8, 64, 3000), (350, 4, 32, 40)])
def test_reorder_matches_the_model(groups, beams, page, max_pages):
    # the last two: a cluster of blocks; more rows than a block has threads, few columns at a time
    r = np.random.default_rng(groups + beams)
    hi = 300 if groups > 100 else 900
    prompts = r.integers(0, hi, groups)
    since = r.integers(1, 2 * page, groups)
    prompts[0], since[0] = page, page                          # lengths that end on a page: nothing to copy
    s = Beams(groups, beams, prompts.tolist(), since.tolist(), page, max_pages=max_pages, layers=1 if groups > 100 else 2, seed=7, outside=3)
    base = np.repeat(np.arange(groups) * beams, beams)
    for step in range(4):
        parent = base + r.integers(0, beams, groups * beams)
        if step == 1:
            parent[r.random(len(parent)) < 0.2] = -1
        if step == 2:
            parent = np.arange(groups * beams)                 # nothing moves
        if step == 3:
            parent = r.permutation(groups * beams)             # any map of the rows, across groups
        assert s.reorder(parent) is not None
        status()
        s.check()


def test_reorder_of_more_columns_than_a_block_holds():
    """4096 rows of up to 86 pages: each of the cluster's eight blocks takes 10 or 11 columns of the table and holds 8 at a time, so that every phase reads it in pieces."""
    groups, beams, page = 16, 256, 32
    r = np.random.default_rng(11)
    s = Beams(groups, beams, r.integers(2300, 2700, groups).tolist(), r.integers(1, 40, groups).tolist(), page, heads=1, layers=1, seed=5)
    most = max(-(-n // page) for n in s.p.len)
    assert groups * beams == 4096 and -(-most // 8) > 32768 // 4096
    base = np.repeat(np.arange(groups) * beams, beams)
    for step in range(4):
        parent = base + r.integers(0, beams, groups * beams)
        if step == 1:
            parent[r.random(len(parent)) < 0.2] = -1
        if step == 3:
            parent = r.permutation(groups * beams)             # any map of the rows, across groups
        assert s.reorder(parent) is not None
        status()
        s.check()
    # a bad entry in a column of the second piece of the last block: nothing changes
    keep = s.table.clone()
    b = int(np.argmax(s.p.len))
    s.table[b, -(-s.p.len[b] // page) - 1] = -7
    kv.mqkv_reorder(s.cache, s.seqs, i32(parent), s.ws)
    status("page table")
    s.table.copy_(keep)
    s.check()
    # too few pages: the counts of all columns go back.  One row ends whose own pages are named elsewhere too, another is continued twice, and no page is free
    parent = r.permutation(groups * beams)
    here, twice = [i for i in range(len(parent)) if s.p.len[parent[i]] % page][:2]
    ends, parent[here] = parent[here], parent[twice]
    own = [x for x in s.p.table[ends] if s.p.refs[x] == 1]
    for x in s.p.free():
        s.p.refs[x] = 1
    for x in own:
        s.p.refs[x] += 1
    s.refs.copy_(i32(s.p.refs))
    assert own and s.reorder(parent) is None
    status("too few free pages")
    s.check()
    s.p.refs[own[0]] -= 1                                      # this one comes free in the call, and takes the copy
    s.refs.copy_(i32(s.p.refs))
    assert [d for _, d, _ in s.reorder(parent)] == own[:1]
    status()
    s.check()


def test_reorder_takes_pages_that_end_in_the_same_call():
    # no page is free before: what row 1 leaves holds the copy of row 0's last page
    s = Beams(1, 2, [32], [40], 64, spare=0, seed=1)
    assert s.p.free() == [] and len(s.reorder([0, 0])) == 1
    status()
    s.check()
    assert len(s.reorder([1, 1])) == 1
    s.check()
    s.reorder([-1, -1])
    s.check()
    assert s.p.len == [0, 0]
    s.reorder([1, 0])                                          # of rows that are empty
    s.check()
    status()


def test_reorder_refuses_what_does_not_fit_and_bad_input():
    # an empty row each beside a row of its own: the copies need pages that are not there
    s = Beams(3, 2, [32, 64, 10], [40, 6, 1], 64, spare=0, seed=2)
    s.reorder([0, -1, 2, -1, 4, -1])
    free = len(s.p.free())
    s.check()
    hold = s.p.free()[:free - 1]                               # all but one are taken elsewhere
    for p in hold:
        s.p.refs[p] = 1
    s.refs.copy_(i32(s.p.refs))
    assert s.reorder([0, 0, 2, 2, 4, -1]) is None
    status("too few free pages")
    s.check()
    assert len(s.reorder([0, 0, 2, -1, 4, -1])) == 1
    status()
    s.check()
    for parent, word in (([0, 1, 2, 3, 4, 6], "sequence id"), ([0, -2, 2, 3, 4, 5], "sequence id"), ([2 ** 31 - 1] * 6, "sequence id")):
        kv.mqkv_reorder(s.cache, s.seqs, i32(parent), s.ws)
        status(word)
        s.check()
    keep = s.table.clone(), s.len.clone()
    for at, value, word in (((0, 0), 10 ** 6, "page table"), ((2, 0), -1, "page table")):
        s.table[at] = value
        kv.mqkv_reorder(s.cache, s.seqs, i32([2, 2, 0, 0, 4, 4]), s.ws)
        status(word)
        s.table.copy_(keep[0])
        s.check()
    for value in (-3, 10 ** 6, 2 ** 31 - 1):
        s.len[0] = value
        kv.mqkv_reorder(s.cache, s.seqs, i32([2, 2, 0, 0, 4, 4]), s.ws)
        status("length")
        s.len.copy_(keep[1])
        s.check()
    with pytest.raises(B.MQError):
        kv.mqkv_reorder(s.cache, s.seqs, i32([0, 1]), s.ws)


# ------------------------------------------------------------------------------- all of it, as it is used ---

@pytest.mark.parametrize("layers,heads,kv_heads,dim,prompt,beams,steps,page", [(2, 4, 2, 64, 45, 4, 40, 32), (1, 6, 1, 128, 7, 3, 9, 64), (3, 4, 4, 64, 96, 5, 33, 32)])
def test_beam_search_keeps_every_hypothesis_in_the_cache(layers, heads, kv_heads, dim, prompt, beams, steps, page):
    """Residuals, norms, planes, projections, rotations, appends, attention, head, selection and reordering in one captured step.  What the cache holds
    for each beam at the end is what its tokens give when they are run alone: but for the f32 sums of attention, which may move a code of the next plane by one
    (2e-2 of a state's size in all, as tests/test_gpu_kv.py has it), and for codes that then fall on the other side of a border (1 / 254 of a block's largest); rows
    that are not the beam's own would be off by their whole size."""
    import torch
    from examples import kv_decode
    ids = np.random.default_rng(9).integers(0, 300, prompt).tolist()

    def model():
        return kv_decode.Attention(layers, 512, heads, kv_heads, dim, beams, prompt + steps + 2, page)
    m = model()
    s = kv_decode.Search(m, beams, 300)
    paths, scores = s.run(ids, steps)
    assert all(len(p) == steps for p in paths) and len({tuple(p) for p in paths}) == beams
    assert scores == sorted(scores, reverse=True) and np.isfinite(scores).all()
    status()
    B.mq_device_status()
    assert m.len.tolist() == [prompt + steps - 1] * beams
    # every page is named as often as its count says
    names = torch.bincount(m.table[m.table >= 0].long(), minlength=len(m.refs))
    assert torch.equal(names.int(), m.refs)

    def cached(mm, seqs, layer, n, count):
        k, v = (torch.empty((count * n, kv_heads, dim), device="cuda") for _ in range(2))
        kv.mqkv_read(mm.cache, seqs, layer, k, v)
        return k.view(count, n, -1), v.view(count, n, -1)
    n = prompt + steps - 1
    alone = model()
    for b in range(beams):
        alone.step(s.table[torch.tensor(ids, device="cuda")], 1)
        for token in paths[b][:-1]:
            alone.step(s.table[token:token + 1].clone(), 1)
        for layer in range(layers):
            for got, want in zip(cached(m, m.seqs(beams), layer, n, beams), cached(alone, alone.seqs(1), layer, n, 1)):
                # per token: a single wrong row would show
                err = ((got[b] - want[0]).norm(dim=1) / want[0].norm(dim=1)).max().item()
                assert err < 0.05, (b, layer, err)
        kv.mqkv_release(alone.cache, alone.all, i32([0]))
    status()


def test_captured_search_step_equals_the_same_calls():
    import torch
    from examples import kv_decode
    got = []
    for captured in (False, True):
        m = kv_decode.Attention(2, 512, 4, 2, 64, 4, 120, 32)
        m.pool.zero_()                                         # (what no token has written)
        s = kv_decode.Search(m, 4, 500)
        x = s.table[:4].clone()
        m.step(x, 4)
        s.scores.copy_(torch.tensor([[-0.5, -0.25, -1.0, -2.0]]))
        if captured:
            stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            m.buffers(4, 4)
            with torch.cuda.graph(graph, stream=stream):
                s.step(x)
            with torch.cuda.stream(stream):
                for _ in range(40):
                    graph.replay()
        else:
            for _ in range(40):
                s.step(x)
        sync()
        status()
        got.append([t.clone() for t in (x, s.scores, s.row, s.token, m.table, m.len, m.refs, m.pool)])
    for a, b in zip(*got):
        same(a, b)


def test_a_search_serves_one_prompt_after_another():
    import torch
    from examples import kv_decode
    m = kv_decode.Attention(2, 512, 4, 2, 64, 3, 60, 32)
    s = kv_decode.Search(m, 3, 300)
    r = np.random.default_rng(4)
    prompts = [r.integers(0, 300, n).tolist() for n in (30, 7, 30)]
    prompts[2] = prompts[0]
    paths = [s.run(p, 12) for p in prompts]
    status()
    assert paths[0] == paths[2] and paths[0] != paths[1]      # (the same calls on the same pages: bit for bit)
    assert m.len.tolist() == [41] * 3
    other = kv_decode.Search(kv_decode.Attention(2, 512, 4, 2, 64, 3, 60, 32), 3, 300)
    assert other.run(prompts[1], 12) == paths[1]
    names = torch.bincount(m.table[m.table >= 0].long(), minlength=len(m.refs))
    assert torch.equal(names.int(), m.refs)

"""GPU parity of the paged 8-bit KV cache against the plain model of kv_util: codes, scales and page tables bit for bit,
attention within a bound that follows from the number formats."""
import numpy as np
import pytest

from quantized_q8_activation_quantize_gb300 import binding as B
from quantized_q8_activation_quantize_gb300 import kv
from tests import kv_util as U

pytestmark = pytest.mark.gpu

TYPES = ("f32", "f16", "bf16")


def ttype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


def status(expect=None):
    if expect is None:
        kv.mqkv_device_status()
        return
    with pytest.raises(B.MQError) as e:
        kv.mqkv_device_status()
    assert e.value.status == kv.MQKV_ERR_STATE and expect in str(e.value), str(e.value)
    kv.mqkv_device_status()                                  # and the word is clear again


class Setup:
    """A pool with a scattered page table for sequences of the given lengths; what no sequence uses is poison."""

    def __init__(self, lens, heads, dim, page, layers=2, seed=0, extra=3, max_pages=None, refs=True):
        r = np.random.default_rng(seed)
        self.lens = list(lens)
        used = [-(-n // page) for n in self.lens]
        n_pages = sum(used) + extra
        order = r.permutation(n_pages)
        self.rows, at = [], 0
        for u in used:
            self.rows.append(order[at:at + u])
            at += u
        self.m = U.Model(n_pages, layers, heads, dim, page)
        self.m.codes[:] = r.integers(-127, 128, self.m.codes.shape)
        self.m.scales[:] = np.float32(np.nan)
        for row, n in zip(self.rows, self.lens):
            for blk in range(-(-n // 32)):
                self.m.scales[row[blk * 32 // page], :, :, :, blk * 32 % page // 32] = r.uniform(0.002, 0.03, self.m.scales.shape[1:4])
        table = np.full((len(self.lens), max_pages or max(max(used, default=1), 1) + 1), 0x7FFFFFF0, np.int32)
        for b, row in enumerate(self.rows):
            table[b, :len(row)] = row
        ref = np.zeros(n_pages, np.int32)
        for row in self.rows:
            ref[row] += 1
        self.table, self.len, self.refs = dev(table), i32(self.lens), dev(ref)
        self.pool = dev(self.m.bytes(fill=0xFF))
        self.cache = kv.cache(self.pool, self.refs if refs else None, layers, heads, dim, page)
        self.seqs = kv.sequences(self.table, self.len)

    def check_pool(self):
        """the pool is the model's, byte for byte (padding and all)"""
        got, want = self.pool.cpu().numpy(), self.m.bytes(fill=0xFF)
        assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ, first at {np.argwhere(got != want)[:3]}"


def cu_of(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


# --------------------------------------------------------------------------------- append, read ---

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,heads", [(128, 64, 4), (64, 32, 3), (128, 256, 1), (64, 128, 2)])
def test_append_matches_the_model(dtype, dim, page, heads):
    import torch
    # (cached before, new): fresh, inside a block, across blocks and pages, ending on boundaries, none at all
    cases = [(0, 1), (0, 32), (0, 33), (5, 1), (31, 1), (32, 1), (31, 2), (63, 70), (64, 64), (100, 0), (0, 0), (17, 300), (256, 1), (300, 5)]
    s = Setup([a + n for a, n in cases], heads, dim, page, seed=dim + page)
    r = np.random.default_rng(3)
    new = [n for _, n in cases]
    x = r.standard_normal((2, sum(new), heads, dim)).astype(np.float32) * r.choice([1e-3, 0.3, 1.0, 30.0], (1, sum(new), 1, 1)).astype(np.float32)
    x[:, 3] = 0                                              # a token of zeros
    xt = torch.from_numpy(x).to(ttype(dtype)).cuda()
    kv.mqkv_append(s.cache, s.seqs, 1, xt[0], xt[1], cu_of(new))
    status()
    x = xt.float().cpu().numpy()
    at = 0
    for (a, n), row in zip(cases, s.rows):
        for half in range(2):
            if n:
                s.m.append(1, half, row, a + n, x[half, at:at + n])
        at += n
    s.check_pool()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("before", [0, 300])
def test_append_of_many_tokens(dtype, before):
    import torch
    # enough for four blocks to a CTA; sequences that begin and end anywhere in them, one of none, one inside a block
    new, had = [1700, 1, 0, 33, 128, 129, 2900, 500], [5, 40, 7, 31, 0, 96, 64, 1001]
    s = Setup([a + n for a, n in zip(had, new)], 16, 64, 64, layers=1, seed=41)
    x = np.random.default_rng(42).standard_normal((2, before + sum(new), 16, 64)).astype(np.float32)
    xt = torch.from_numpy(x).to(ttype(dtype)).cuda()
    kv.mqkv_append(s.cache, s.seqs, 0, xt[0], xt[1], i32(before + np.concatenate([[0], np.cumsum(new)])))
    status()
    x, at = xt.float().cpu().numpy(), before
    for b, n in enumerate(new):
        for half in range(2):
            if n:
                s.m.append(0, half, s.rows[b], s.lens[b], x[half, at:at + n])
        at += n
    s.check_pool()


def test_append_token_by_token_and_strided():
    import torch
    # one projection's output [tokens, q heads + 2 * kv heads, dim]: k and v are strided views; no cu, one token each
    s = Setup([40, 1, 64, 95], 2, 128, 32, seed=8)
    r = np.random.default_rng(9)
    lens = np.array(s.lens)
    for step in range(5):
        x = (r.standard_normal((4, 7, 128)) * 4.0 ** step).astype(np.float32)
        xt = dev(x)
        s.len.copy_(i32(lens))
        kv.mqkv_append(s.cache, s.seqs, 0, xt[:, 3:5], xt[:, 5:7])
        for b in range(4):
            s.m.append(0, 0, s.rows[b], lens[b], x[b:b + 1, 3:5])
            s.m.append(0, 1, s.rows[b], lens[b], x[b:b + 1, 5:7])
        lens = lens + (lens % 32 != 0)                       # stays inside the pages that are there
    status()
    s.check_pool()
    # the same with a head stride larger than the token's, [heads, tokens, dim]
    x = r.standard_normal((2, 4, 128)).astype(np.float32)
    xt = dev(x).transpose(0, 1)
    s.len.copy_(i32(s.lens))
    kv.mqkv_append(s.cache, s.seqs, 1, xt, xt)
    for b in range(4):
        for half in range(2):
            s.m.append(1, half, s.rows[b], s.lens[b], x[:, b][None])
    torch.cuda.synchronize()
    s.check_pool()


@pytest.mark.parametrize("before,after", [(300, 0), (130, 400), (1000, 7)])
def test_append_where_cu_does_not_begin_at_0(before, after):
    # rows before cu[0] and past cu[n] are no sequence's: nothing is read or written for them
    new = [3, 40, 0, 200]
    s = Setup([40, 45, 33, 210], 2, 64, 32, seed=12)
    r = np.random.default_rng(6)
    x = r.standard_normal((2, before + sum(new) + after, 2, 64)).astype(np.float32)
    xt = dev(x)
    kv.mqkv_append(s.cache, s.seqs, 1, xt[0], xt[1], i32(before + np.concatenate([[0], np.cumsum(new)])))
    status()
    at = before
    for b, n in enumerate(new):
        for half in range(2):
            if n:
                s.m.append(1, half, s.rows[b], s.lens[b], x[half, at:at + n])
        at += n
    s.check_pool()


def test_append_of_values_that_cannot_be_a_scale():
    s = Setup([70, 33, 40, 20], 1, 64, 64, seed=4)
    x = np.random.default_rng(5).standard_normal((70 + 1 + 8 + 20, 1, 64)).astype(np.float32)
    x[3, 0, 5], x[4, 0, :3], x[40] = np.nan, [np.inf, -np.inf, 2.0], np.nan
    x[70, 0, 1] = np.inf
    x[71:79] = 1e-40                                         # subnormal scale: stored as zeros (old codes of the block stay)
    x[79:] = 3e38
    new = [70, 1, 8, 20]
    xt = dev(x)
    kv.mqkv_append(s.cache, s.seqs, 0, xt, xt, cu_of(new))
    status()
    at = 0
    for b, n in enumerate(new):
        for half in range(2):
            s.m.append(0, half, s.rows[b], s.lens[b], x[at:at + n])
        at += n
    s.check_pool()
    assert np.isfinite(s.m.scales[s.rows[0], 0]).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,heads", [(128, 64, 4), (64, 32, 3)])
def test_read_gives_the_values(dtype, dim, page, heads):
    import torch
    lens, new, start = [1, 40, 200, 0, 97], [1, 7, 131, 0, 33], [0, 33, 11, 0, 64]
    s = Setup(lens, heads, dim, page, seed=2)
    n = sum(new)
    for st in (None, start):
        buf = torch.full((n, 2 * heads + 1, dim), 7.0, dtype=ttype(dtype), device="cuda")
        k, v = buf[:, :heads], buf[:, heads:2 * heads]
        kv.mqkv_read(s.cache, s.seqs, 1, k, v, cu_of(new), None if st is None else i32(st))
        status()
        for half, got in enumerate((k, v)):
            want = np.concatenate([s.m.values(1, half, s.rows[b], np.arange(new[b]) + (lens[b] - new[b] if st is None else st[b])) if new[b]
                                   else np.zeros((0, heads, dim)) for b in range(len(lens))])
            # f32: q * d rounded once; the narrower types round that once more
            assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(ttype(dtype)))
        assert (buf[:, 2 * heads] == 7).all()
    only = torch.zeros((n, heads, dim), dtype=ttype(dtype), device="cuda")
    kv.mqkv_read(s.cache, s.seqs, 1, None, only, cu_of(new), i32(start))
    assert torch.equal(only, v)
    status()


def test_bad_lengths_and_tables_are_reported_and_left_alone():
    import torch
    s = Setup([40, 70], 2, 64, 32, seed=6, max_pages=4)
    before = s.pool.clone()
    x = torch.randn((2, 2, 64), device="cuda")
    out = torch.ones((2, 2, 64), device="cuda")
    ws = kv.alloc_attention_workspace(s.cache, s.seqs, 2, 2, 1, 100, torch.float32)

    def each(expect):
        kv.mqkv_append(s.cache, s.seqs, 0, x[:1], x[:1], i32([0, 1, 1]))
        status(expect)
        out.fill_(1)
        kv.mqkv_read(s.cache, s.seqs, 0, out[:1], None, i32([0, 1, 1]))
        status(expect)
        assert (out[0] == 0).all()
    s.len.copy_(i32([0, 70]))                                # fewer cached tokens than new ones
    each("length")
    s.len.copy_(i32([32 * 4 + 1, 70]))                       # past the table row
    each("length")
    s.len.copy_(i32([-5, 70]))
    each("length")
    s.len.copy_(i32([40, 70]))
    good = s.table.clone()
    for bad in (-1, s.m.codes.shape[0], 2 ** 31 - 1):
        s.table[0, 1] = bad
        each("page table")
        kv.mqkv_attention(s.cache, s.seqs, 0, x, out, None, 1, 70, ws)
        status("page table")
        assert torch.isfinite(out[1]).all()
    s.table.copy_(good)
    s.refs[int(good[0, 1])] = 2                              # another sequence shares the page
    kv.mqkv_append(s.cache, s.seqs, 0, x[:1], x[:1], i32([0, 1, 1]))
    status("shared")
    assert torch.equal(s.pool, before)
    s.len.copy_(i32([-1, 70]))
    kv.mqkv_attention(s.cache, s.seqs, 0, x, out, None, 1, 70, ws)
    status("length")
    assert (out[0] == 0).all() and (out[1] != 0).any()
    s.len.copy_(i32([40, 70]))
    x4, o4 = torch.randn((4, 2, 64), device="cuda"), torch.zeros((4, 2, 64), device="cuda")
    kv.mqkv_attention(s.cache, s.seqs, 0, x4, o4, i32([0, 3, 4]), 2, 70, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    status("max_q")


# ------------------------------------------------------------------------------------ attention ---

def run_attention(s, q, new, dtype, layer=1, max_q=None, max_kv=None, stream=None, **kw):
    import torch
    qt = torch.from_numpy(q.astype(np.float32)).to(ttype(dtype)).cuda()
    out = torch.full_like(qt, 9.0)
    max_q, max_kv = max(new) if max_q is None else max_q, max(s.lens + [1]) if max_kv is None else max_kv
    ws = kv.alloc_attention_workspace(s.cache, s.seqs, q.shape[1], len(q), max_q, max_kv, qt.dtype)
    ws.fill_(0xFF)                                           # the workspace's contents are nothing to rely on
    kv.mqkv_attention(s.cache, s.seqs, layer, qt, out, cu_of(new), max_q, max_kv, ws, **kw)
    status()
    return out.float().cpu().numpy(), qt.double().cpu().numpy()


def check_attention(s, new, heads, dtype, layer=1, seed=1, qscale=1.0, rows=None, **kw):
    r = np.random.default_rng(seed)
    q = r.standard_normal((sum(new), heads, s.m.D)) * qscale
    got, q = run_attention(s, q, new, dtype, layer, **kw)
    kw.pop("max_q", None), kw.pop("max_kv", None)
    at = 0
    for b, n in enumerate(new):
        length = s.lens[b]
        k, v = (s.m.values(layer, half, s.rows[b], np.arange(length)) if length else np.zeros((0, s.m.H, s.m.D)) for half in range(2))
        out, mass, vmax = U.attention(q[at:at + n], k, v, length, **kw)
        tol = U.attention_tolerance(out, mass, vmax, length, dtype)
        off = np.abs(got[at:at + n] - out)
        assert np.isfinite(got[at:at + n]).all() and (off <= tol).all(), (b, n, length, float((off / tol).max()), np.argwhere(off > tol)[:3])
        at += n
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(28, 4, 128, 64), (8, 8, 64, 32), (5, 1, 128, 128), (40, 2, 64, 256), (9, 3, 128, 32)])
def test_decode(dtype, heads, kv_heads, dim, page):
    # one token each: lengths around a block's, a page's and a split's end, zero among them
    lens = [1, 2, 31, 32, 33, 0, 64, 65, 127, 257, 700, 1023, 1500]
    s = Setup(lens, kv_heads, dim, page, seed=heads)
    check_attention(s, [1] * len(lens), heads, dtype, qscale=2.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kw", [dict(), dict(window=1), dict(window=40), dict(causal=False), dict(causal=False, window=33),
                                dict(scale=0.5), dict(scale=-0.02), dict(scale=0.0), dict(max_kv=1), dict(max_q=300, max_kv=100000)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "causal")
def test_masks_and_ragged_rows(dtype, kw):
    # rows of every kind: none, one, a few, more than are cached (rows before the first token see nothing), many
    lens, new = [50, 300, 7, 0, 129, 64, 333, 20], [3, 1, 9, 2, 0, 64, 70, 20]
    s = Setup(lens, 2, 128, 64, seed=5)
    check_attention(s, new, 6, dtype, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(14, 2, 128, 64), (4, 4, 64, 32), (3, 1, 64, 256), (16, 1, 128, 128)])
def test_prefill(dtype, heads, kv_heads, dim, page):
    lens, new = [300, 131, 517, 40], [300, 129, 200, 1]
    s = Setup(lens, kv_heads, dim, page, seed=dim)
    check_attention(s, new, heads, dtype)
    check_attention(s, new, heads, dtype, window=100, seed=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=700), dict(window=3), dict(causal=False), dict(scale=0.0), dict(qscale=6.0), dict(max_kv=100000)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "causal")
def test_few_row_tiles(dtype, dim, kw):
    # too few row tiles for every SM: they are cut along the tokens, into more pieces than the short sequences have tiles for
    s = Setup([4100, 0, 37, 2500, 1], 2, dim, 64, seed=dim)
    check_attention(s, [40, 3, 37, 12, 0], 8, dtype, **kw)


@pytest.mark.parametrize("dtype,lens,new,heads,kv_heads", [("f32", [1500] * 40, [20] * 40, 16, 4), ("f16", [1500] * 40, [20] * 40, 16, 4),
                                                           ("f32", [2000], [640], 32, 8), ("bf16", [1500, 3000], [640, 645], 32, 8)])
def test_last_row_tiles_cut(dtype, lens, new, heads, kv_heads):
    # a wave of whole row tiles and more, the rest cut: some of many sequences, and the first of several per sequence
    s = Setup(lens, kv_heads, 64, 64, layers=1, seed=len(lens))
    check_attention(s, new, heads, dtype, layer=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31, 2 ** 40 + 1, 2 ** 63 - 1])
def test_windows_past_every_position(dtype, causal, window):
    # rows at positions far below the first token among them: without causality they see all of it
    for lens, new in (([2, 70], [7, 3]), ([10, 200], [200, 40])):
        s = Setup(lens, 2, 64, 32, seed=23)
        check_attention(s, new, 4, dtype, causal=causal, window=window)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,new,heads", [(128, 6, 14), (64, 20, 16), (128, 70, 4)])
def test_tiles_of_many_sequences_again_and_again(dtype, dim, new, heads):
    import torch
    # every SM with several row tiles after one another, whole ones and pieces: all waits end, and the results are the same each time
    s = Setup([1800 + 16 * b for b in range(48)], 2, dim, 64, layers=1, seed=dim)
    q = torch.randn((48 * new, heads, dim), device="cuda").to(ttype(dtype))
    ws = kv.alloc_attention_workspace(s.cache, s.seqs, heads, len(q), new, max(s.lens), q.dtype)
    out, first = torch.empty_like(q), None
    for i in range(40):
        out.fill_(9.0)
        kv.mqkv_attention(s.cache, s.seqs, 0, q, out, None, new, max(s.lens), ws)
        first = out.clone() if i == 0 else first
        assert torch.equal(out, first), i
    status()
    assert torch.isfinite(first).all()


@pytest.mark.parametrize("n,dtype", [(257, "f32"), (1500, "f16")])
def test_many_sequences(n, dtype):
    # more than the plan's shared memory holds, and more than one round of its scan; most of them short, some empty
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.choice([0, 1, 3, 17, 33, 70], n)]
    lens[5] = 900
    s = Setup(lens, 1, 64, 32, layers=1, seed=n)
    check_attention(s, [1] * n, 2, dtype, layer=0)
    new = [int(x) for x in r.integers(0, 3, n)]
    check_attention(s, new, 2, dtype, layer=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,new,heads", [([700, 90, 1500], [1, 1, 2], 4), ([70] * 90, [1] * 90, 8), ([20011, 300], [1, 1], 4),
                                            ([4100, 37, 2500], [40, 37, 12], 8), ([700] * 45, [70] * 45, 8)],
                         ids=["passes", "short", "joined", "cut", "whole"])
def test_rows_of_a_bad_page_entry_are_zero(dtype, lens, new, heads):
    import torch
    s = Setup(lens, 2, 64, 32, seed=21)
    q = torch.randn((sum(new), heads, 64), device="cuda").to(ttype(dtype))
    q[0, 1, 3] = float("nan")                                # zeros for a row that would be NaN, too
    at = np.concatenate([[0], np.cumsum(new)])
    ws = kv.alloc_attention_workspace(s.cache, s.seqs, heads, len(q), max(new), max(lens), q.dtype)
    good, out = torch.full_like(q, 9.0), torch.full_like(q, 9.0)
    kv.mqkv_attention(s.cache, s.seqs, 1, q, good, i32(at), max(new), max(lens), ws)
    status()
    entries = s.table.clone()
    # the last page (causal rows before it do not see it), one in the middle, the first one; of the first sequence and of others
    for b, page, entry in ((0, (lens[0] - 1) // 32, -1), (len(lens) - 1, lens[-1] // 64, len(s.refs)), (len(lens) // 2, 0, 2 ** 31 - 1)):
        s.table.copy_(entries)
        s.table[b, page] = entry
        out.fill_(9.0)
        kv.mqkv_attention(s.cache, s.seqs, 1, q, out, i32(at), max(new), max(lens), ws)
        status("page table")
        assert (out[at[b]:at[b + 1]] == 0).all()
        rest = torch.cat([torch.arange(0, at[b]), torch.arange(at[b + 1], at[-1])]).cuda()
        assert torch.equal(out[rest].nan_to_num(7.0), good[rest].nan_to_num(7.0))
    # an entry that no row's window reaches is not looked at
    far = [b for b, n in enumerate(lens) if n - new[b] > 200]
    if far:
        s.table.copy_(entries)
        kv.mqkv_attention(s.cache, s.seqs, 1, q, good, i32(at), max(new), max(lens), ws, window=100)
        status()
        s.table[far[0], 0] = -1
        kv.mqkv_attention(s.cache, s.seqs, 1, q, out, i32(at), max(new), max(lens), ws, window=100)
        status()
        assert torch.equal(out.nan_to_num(7.0), good.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_long_and_peaked(dtype):
    # long enough to be split many ways; scores far apart, so that one token carries a row
    s = Setup([20011, 4099], 1, 128, 128, seed=7)
    check_attention(s, [1, 2], 7, dtype, qscale=0.1)
    check_attention(s, [2, 1], 7, dtype, qscale=6.0)


@pytest.mark.parametrize("heads,dim", [(4, 128), (12, 128), (4, 64), (12, 64)])
def test_sums_over_long_shares(heads, dim):
    # four workers for 65536 tokens of values of one sign: sums that are cut instead of rounded drift (they did by 4e-5 of the result).
    # Of the terms of attention_tolerance the sums' is replaced: 1024 additions a worker (two per 32 tokens), each within 2^-24 of the sum and of
    # either sign, so four times their root in all; the rest as there.
    n = 65536
    s = Setup([n], 1, dim, 256, layers=1, seed=dim)
    s.m.codes[:, :, 1] = np.abs(s.m.codes[:, :, 1])
    s.pool.copy_(dev(s.m.bytes(fill=0xFF)))
    q = np.random.default_rng(1).standard_normal((1, heads, dim)) * 0.1
    got, q = run_attention(s, q, [1], "f32", layer=0, max_kv=1)
    k, v = (s.m.values(0, half, s.rows[0], np.arange(n)) for half in range(2))
    out, mass, vmax = U.attention(q, k, v, n)
    tol = (2 * (2 * (2.0 ** -21 + 2.0 ** -22) * mass + 2.0 ** -21) + 4 * 1024 ** 0.5 * 2.0 ** -24) * vmax
    off = np.abs(got - out).max(-1)
    assert (off <= tol).all(), (off / vmax, tol / vmax)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 200])
def test_scales_of_many_sizes(dtype, new):
    # V scales over twelve binary orders in one sequence, a block of zeros, K scales that make whole blocks vanish
    s = Setup([640], 2, 64, 64, seed=11)
    r = np.random.default_rng(12)
    for blk in range(20):
        p, sb = s.rows[0][blk * 32 // 64], blk % 2
        s.m.scales[p, :, 1, :, sb] = np.float32(0.02 * 2.0 ** -(blk % 13))
        s.m.scales[p, :, 0, :, sb] = np.float32(0.002 * r.uniform(0, 8))
    s.m.scales[s.rows[0][0], :, 1] = 0
    s.pool.copy_(dev(s.m.bytes()))
    check_attention(s, [new], 4, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,max_kv", [(5, None), (5, 1), (130, None), (130, 1)])
@pytest.mark.parametrize("kind,dim", [("later", 64), ("later", 128), ("window", 128), ("unweighted", 64), ("unweighted", 128)])
def test_large_values_take_no_bits_from_rows_that_do_not_weigh_them(dtype, new, max_kv, kind, dim):
    # a block of V up to 2^90 times the others': after a row, before its window, or where its weight vanishes; held to the row's own values.
    # (max_kv = 1: few workers with long shares, row tiles in one piece)
    n = 579
    r = np.random.default_rng(31)
    q = 1 + 0.2 * r.standard_normal((new, 4, dim))
    for ratio in (2.0 ** 12, 2.0 ** 28, 2.0 ** 90):
        s = Setup([n], 2, dim, 64, seed=32)
        # (positions 576 .. 578, 0 .. 95, 320 .. 351)
        for blk in {"later": [18], "window": [0, 1, 2], "unweighted": [10]}[kind]:
            p, sb = s.rows[0][blk // 2], blk % 2
            s.m.scales[p, :, 1, :, sb] *= np.float32(ratio)
            if kind == "unweighted":
                s.m.codes[p, :, 0, :, 32 * sb:32 * sb + 32] = -127
                s.m.scales[p, :, 0, :, sb] = 0.2
        s.pool.copy_(dev(s.m.bytes()))
        kw = {"window": 200} if kind == "window" else {}
        got, qq = run_attention(s, q, [new], dtype, max_kv=max_kv, **kw)
        pos = np.arange(n)
        k, v = (s.m.values(1, half, s.rows[0], pos) for half in range(2))
        d = s.m.scales[s.rows[0][pos // 64], 1, 1, :, pos % 64 // 32].astype(np.float64)
        out, tol = U.attention_own(qq, k, v, d, n, dtype, **kw)
        fits = np.abs(out) < (6e4 if dtype == "f16" else 1e37)
        assert fits[:new - 3].all()
        off = np.abs(got - out)
        assert (off <= tol)[fits].all(), (ratio, float((off / tol)[fits].max()), np.argwhere((off > tol) & fits)[:3])


@pytest.mark.parametrize("dtype", TYPES)
def test_queries_of_extreme_sizes_and_not_numbers(dtype):
    s = Setup([100, 90, 0], 2, 128, 32, seed=13)
    new = [3, 2, 1]
    big = {"f32": 1e30, "f16": 6e4, "bf16": 1e30}[dtype]
    q = np.random.default_rng(14).standard_normal((6, 4, 128))
    q[0] *= big / 4
    q[1] *= 1e-30 if dtype != "f16" else 6e-8
    q[2, 0, 5], q[2, 2, 7], q[4, 3, :] = np.nan, np.inf, -np.inf
    q[5, 0, 0] = np.nan                                      # a row that sees nothing: zero all the same
    got, q = run_attention(s, q, new, dtype, scale=1e-31 if dtype != "f16" else 1e-6)
    at = 0
    for b, n in enumerate(new):
        k, v = (s.m.values(1, half, s.rows[b], np.arange(s.lens[b])) if s.lens[b] else np.zeros((0, 2, 128)) for half in range(2))
        out, mass, vmax = U.attention(q[at:at + n], k, v, s.lens[b], scale=1e-31 if dtype != "f16" else 1e-6)
        assert np.array_equal(np.isnan(got[at:at + n]), np.isnan(out))
        fin = ~np.isnan(out)
        tol = U.attention_tolerance(out, mass, vmax, s.lens[b], dtype)
        assert (np.abs(got[at:at + n] - out)[fin] <= tol[fin]).all()
        at += n
    assert (got[5] == 0).all()


@pytest.mark.parametrize("new", [1, 150])
def test_strides_streams_and_repeats(new):
    import torch
    s = Setup([400, 333], 2, 128, 64, seed=15)
    n, heads = 2 * new, 6
    wide = torch.randn((n, heads + 4, 128), device="cuda")   # q inside a projection's output
    q = wide[:, :heads]
    out = torch.zeros((heads, n, 128), device="cuda").transpose(0, 1)
    ws = kv.alloc_attention_workspace(s.cache, s.seqs, heads, n, new, 400, torch.float32)
    dense = torch.zeros((n, heads, 128), device="cuda")
    torch.cuda.synchronize()
    kv.mqkv_attention(s.cache, s.seqs, 1, q.contiguous(), dense, None, new, 400, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.mqkv_attention(s.cache, s.seqs, 1, q, out, None, new, 400, ws, stream=side)
    side.synchronize()
    kv.mqkv_device_status(side)
    assert torch.equal(out, dense) and (dense != 0).any()
    for _ in range(3):                                       # no order of arrival in the results
        again = torch.zeros_like(dense)
        kv.mqkv_attention(s.cache, s.seqs, 1, q, again, None, new, 400, ws)
        assert torch.equal(again, dense)


def test_offsets_past_32_bits():
    import torch
    lay = kv.mqkv_page_layout(24, 8, 128, 256)
    n_pages = (1 << 32) // lay["page_bytes"] + 40            # the last pages lie past 4 GiB
    pool, refs = torch.empty((n_pages, lay["page_bytes"]), dtype=torch.uint8, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    c = kv.cache(pool, refs, 24, 8, 128, 256)
    table, length = i32([[n_pages - 1, n_pages - 3]]), i32([300])
    refs[n_pages - 1], refs[n_pages - 3] = 1, 1
    s = kv.sequences(table, length)
    x = torch.randn((2, 300, 8, 128), device="cuda")
    kv.mqkv_append(c, s, 23, x[0], x[1], i32([0, 300]))
    back = torch.empty_like(x)
    kv.mqkv_read(c, s, 23, back[0], back[1], i32([0, 300]))
    assert (back - x).abs().max() < 0.03 * x.abs().max()
    for n in (1, 200):
        q = torch.randn((n, 8, 128), device="cuda")
        out = torch.empty_like(q)
        kv.mqkv_attention(c, s, 23, q, out, i32([0, n]), n, 300, kv.alloc_attention_workspace(c, s, 8, n, n, 300, q.dtype))
        k, v = back.double()
        sc = torch.einsum("qhd,khd->hqk", q.double(), k) / 128 ** 0.5
        sc.masked_fill_(torch.arange(300, device="cuda")[None] > torch.arange(300 - n, 300, device="cuda")[:, None], -np.inf)
        assert torch.allclose(out.double(), torch.einsum("hqk,khd->qhd", sc.softmax(-1), v), atol=2e-5, rtol=0)
    status()
    src, dst = i32([n_pages - 1]), i32([n_pages - 7])
    kv.mqkv_copy_pages(c, src, dst)
    assert torch.equal(pool[n_pages - 7], pool[n_pages - 1])
    status()


# ---------------------------------------------------------------------------------------- pages ---

class PageSetup:
    def __init__(self, n_pages, n_seqs, max_pages, page=32, layers=2, heads=2, dim=64, seed=0):
        import torch
        self.p = U.Pages(n_pages, n_seqs, max_pages, page)
        self.m = U.Model(n_pages, layers, heads, dim, page)
        size = layers * self.m.slab
        self.pool = torch.randint(0, 256, (n_pages, size), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        self.want = self.pool.cpu().numpy()
        self.table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.len, self.refs = i32([0] * n_seqs), i32([0] * n_pages)
        self.cache, self.seqs = kv.cache(self.pool, self.refs, layers, heads, dim, page), kv.sequences(self.table, self.len)
        self.ws = kv.alloc_pages_workspace(self.cache, self.seqs)

    def moved(self, copies):
        """the model's copies of (source, page, used blocks) pages"""
        m, src = self.m, self.want.copy()
        n = len(src)
        a = self.want.reshape(n, m.L, m.slab)
        b = src.reshape(n, m.L, m.slab)
        for s, d, blocks in copies:
            codes = a[d, :, :m.off_s].reshape(m.L, 2 * m.H, m.T, m.D)
            codes[:, :, :32 * blocks] = b[s, :, :m.off_s].reshape(m.L, 2 * m.H, m.T, m.D)[:, :, :32 * blocks]
            e = m.off_s + 8 * m.H * (m.T // 32)
            a[d, :, m.off_s:e] = b[s, :, m.off_s:e]

    def check(self):
        assert self.len.tolist() == self.p.len
        assert self.refs.tolist() == self.p.refs
        t = self.table.cpu().numpy()
        for b, row in enumerate(self.p.table):
            assert t[b, :len(row)].tolist() == row, b
        assert np.array_equal(self.pool.cpu().numpy(), self.want)


@pytest.mark.parametrize("n_pages,n_seqs,page", [(40, 6, 32), (300, 17, 64), (5000, 1500, 32)])
def test_pages_random_walk(n_pages, n_seqs, page):
    s = PageSetup(n_pages, n_seqs, 12, page=page, layers=1, heads=1)
    r = np.random.default_rng(n_pages)
    for step in range(40):
        what = r.choice(["extend", "extend", "release", "fork", "compact"])
        if what == "extend":
            add = r.integers(0, 2 * page, n_seqs) * (r.random(n_seqs) < 0.5)
            ok = s.p.extend([int(x) for x in add])
            kv.mqkv_extend(s.cache, s.seqs, i32(add), s.ws)
            if ok:
                status()
            else:
                with pytest.raises(B.MQError):
                    kv.mqkv_device_status()
        elif what == "release":
            ids = r.permutation(n_seqs)[:r.integers(1, max(2, n_seqs // 2))]
            s.p.release(ids)
            kv.mqkv_release(s.cache, s.seqs, i32(ids))
            status()
        elif what == "fork":
            empty = [b for b in range(n_seqs) if s.p.len[b] == 0]
            n = min(len(empty), int(r.integers(1, 8)))
            if not n:
                continue
            pairs = list(zip(r.integers(0, n_seqs, n).tolist(), r.permutation(empty)[:n].tolist()))
            copies = s.p.fork(pairs)
            kv.mqkv_fork(s.cache, s.seqs, i32([a for a, _ in pairs]), i32([c for _, c in pairs]), s.ws)
            if copies is None:
                status("free pages")
            else:
                status()
                s.moved(copies)
        else:
            to = s.p.compact()
            old = s.want.copy()
            for a, b in to.items():
                s.want[b] = old[a]
            kv.mqkv_compact(s.cache, s.seqs, s.ws)
            status()
        s.check()


@pytest.mark.parametrize("page,layers,heads,dim", [(256, 3, 2, 128), (64, 28, 4, 128), (128, 1, 3, 64)])
def test_fork_copies_the_used_blocks(page, layers, heads, dim):
    s = PageSetup(30, 9, 4, page=page, layers=layers, heads=heads, dim=dim, seed=3)
    add = [page, page + 1, 2 * page - 1, 33, 0, 0, 0, 0, 0]
    assert s.p.extend(add)
    kv.mqkv_extend(s.cache, s.seqs, i32(add), s.ws)
    pairs = [(0, 4), (1, 5), (2, 6), (3, 7), (1, 8)]
    copies = s.p.fork(pairs)
    kv.mqkv_fork(s.cache, s.seqs, i32([a for a, _ in pairs]), i32([c for _, c in pairs]), s.ws)
    status()
    assert len(copies) == 4
    s.moved(copies)
    s.check()


def test_extend_defaults_and_refusals():
    s = PageSetup(6, 3, 3)
    kv.mqkv_extend(s.cache, s.seqs, None, s.ws)              # one token each
    assert s.p.extend([1, 1, 1])
    status()
    s.check()
    for add, word in (([-1, 0, 0], "length"), ([0, 100, 0], "length"), ([64, 64, 64], "free pages")):
        kv.mqkv_extend(s.cache, s.seqs, i32(add), s.ws)
        status(word)
        s.check()                                            # nothing has changed
    kv.mqkv_extend(s.cache, s.seqs, i32([63, 31, 32]), s.ws)  # to the very ends: all six pages but none more
    assert s.p.extend([63, 31, 32])
    status()
    s.check()


@pytest.mark.parametrize("n_seqs,max_pages", [(65536, 32768), (65536, 65536), (65537, 65536)])
def test_extend_by_more_pages_than_32_bits_count(n_seqs, max_pages):
    import torch
    # the pages that all sequences ask for are 2^31, 2^32 and 2^32 + 2^16: refused, and nothing changes
    pool, refs = kv.alloc_pool(70000, 1, 1, 64, 32)
    table = torch.empty((n_seqs, max_pages), dtype=torch.int32, device="cuda")
    table[:, :2] = -1
    length = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
    c, s = kv.cache(pool, refs, 1, 1, 64, 32), kv.sequences(table, length)
    kv.mqkv_extend(c, s, torch.full((n_seqs,), 32 * max_pages, dtype=torch.int32, device="cuda"), kv.alloc_pages_workspace(c, s))
    status("free pages")
    assert not length.any() and not refs.any() and (table[:, :2] == -1).all()


def test_fork_and_release_refusals():
    s = PageSetup(12, 5, 3)
    s.p.extend([40, 10, 0, 0, 0])
    kv.mqkv_extend(s.cache, s.seqs, i32([40, 10, 0, 0, 0]), s.ws)
    # a child that is not empty, one named twice, ids out of range: those pairs are left out, the others are made
    parent, child = [0, 0, 1, 9, 0], [1, 2, 2, 3, 4]
    kv.mqkv_fork(s.cache, s.seqs, i32(parent), i32(child), s.ws)
    status("sequence id")
    s.moved(s.p.fork([(0, 2), (0, 4)]))
    s.check()
    kv.mqkv_release(s.cache, s.seqs, i32([7, -1, 2, 2]))     # out of range; one twice counts once
    status("sequence id")
    s.p.release([2])
    s.check()


def test_copy_pages():
    s = PageSetup(50, 1, 1, layers=3, heads=4, dim=128, page=64)
    src, dst = [0, 3, 49, 7, 7], [10, 11, 12, 13, 14]
    kv.mqkv_copy_pages(s.cache, i32(src), i32(dst))
    status()
    s.want[dst] = s.want[src]
    s.check()
    kv.mqkv_copy_pages(s.cache, i32([5, 50, -1]), i32([6, 1, 2]))
    status("page table")
    s.want[6] = s.want[5]
    s.check()


# ------------------------------------------------------------------------------------- together ---

def test_steps_in_a_captured_graph():
    """Extend, append and attention of a decode step captured once and replayed: lengths and pages are read on the
    device, so a replay is the next step."""
    import torch
    H, D, T, G, n = 2, 64, 32, 3, 3
    pool, refs = kv.alloc_pool(20, 1, H, D, T)
    pool.zero_()
    table, length = torch.full((n, 6), -1, dtype=torch.int32, device="cuda"), i32([0] * n)
    c, s = kv.cache(pool, refs, 1, H, D, T), kv.sequences(table, length)
    ws, aws = kv.alloc_pages_workspace(c, s), kv.alloc_attention_workspace(c, s, H * G, n, 1, 128, torch.float32)
    k, v, q, out = (torch.zeros((n, h, D), device="cuda") for h in (H, H, H * G, H * G))

    def step():
        kv.mqkv_extend(c, s, None, ws)
        kv.mqkv_append(c, s, 0, k, v)
        kv.mqkv_attention(c, s, 0, q, out, None, 1, 128, aws)
    graph = torch.cuda.CUDAGraph()
    kv.lib()
    with torch.cuda.graph(graph):
        step()
    m, rows = U.Model(20, 1, H, D, T), U.Pages(20, n, 6, T)
    r = np.random.default_rng(1)
    for i in range(70):
        x = [r.standard_normal(t.shape).astype(np.float32) for t in (k, v, q)]
        for t, a in zip((k, v, q), x):
            t.copy_(dev(a))
        graph.replay()
        rows.extend([1] * n)
        for b in range(n):
            m.append(0, 0, rows.table[b], i + 1, x[0][b:b + 1])
            m.append(0, 1, rows.table[b], i + 1, x[1][b:b + 1])
        if i % 23 == 0 or i == 69:
            got = out.cpu().numpy()
            for b in range(n):
                kk, vv = (m.values(0, half, rows.table[b], np.arange(i + 1)) for half in range(2))
                want, mass, vmax = U.attention(x[2][b:b + 1].astype(np.float64), kk, vv, i + 1)
                assert (np.abs(got[b:b + 1] - want) <= U.attention_tolerance(want, mass, vmax, i + 1, "f32")).all()
    status()


@pytest.mark.parametrize("heads,kv_heads,dim,prompt", [(4, 2, 64, 70), (14, 2, 128, 200)])
def test_example_runs_the_operators_together(heads, kv_heads, dim, prompt):
    from examples import kv_decode
    tokens = 6
    got = kv_decode.run(layers=2, hidden=512, heads=heads, kv_heads=kv_heads, dim=dim, prompt=prompt, tokens=tokens, page=32,
                        say=lambda *a: None)
    # `tokens` decode steps alone, one as three, one more of the first; the second has ended
    assert got["len"] == [prompt + tokens + 2, 0, prompt + tokens + 1]
    # attention's f32 rounding may move a Q8 code of the o projection's input by one: 1 / 127 of a block's largest value, of which a
    # state sums `heads * dim` with random signs
    assert got["spread"] < 2e-2
    assert got["same_after_compact"] and np.isfinite(got["state"].cpu().numpy()).all()
    assert got["shared"] == (prompt + tokens) // 32

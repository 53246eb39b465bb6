"""A plain model of the paged 8-bit KV cache (include/mqkv.h) in numpy, for the parity tests: pages as Python
dictionaries of arrays, values and attention in 64 bits, every rule written out one token or page at a time."""
import numpy as np

BLOCK = 32


def f32(x):
    return np.float32(x)


def away(y):
    """round half away from zero, of f32 values"""
    return np.sign(y) * np.floor(np.abs(y).astype(np.float64) + 0.5)


class Model:
    """codes[page, layer, half, head, token, dim] as integers q, scales[page, layer, half, head, block] f32."""

    def __init__(self, n_pages, n_layers, heads, dim, page):
        self.T, self.H, self.D, self.L = page, heads, dim, n_layers
        self.codes = np.zeros((n_pages, n_layers, 2, heads, page, dim), np.int32)
        self.scales = np.zeros((n_pages, n_layers, 2, heads, page // BLOCK), np.float32)
        self.off_s = 2 * heads * page * dim
        self.slab = -(-(self.off_s + 8 * heads * (page // BLOCK)) // 256) * 256

    def bytes(self, fill=0):
        """the pool's bytes, uint8 [n_pages, page_bytes]; padding is `fill`"""
        n = len(self.codes)
        out = np.full((n, self.L, self.slab), fill, np.uint8)
        out[:, :, :self.off_s] = (self.codes + 128).astype(np.uint8).reshape(n, self.L, -1)
        s = np.ascontiguousarray(self.scales).view(np.uint8).reshape(n, self.L, -1)
        out[:, :, self.off_s:self.off_s + s.shape[2]] = s
        return out.reshape(n, -1)

    def take(self, pool):
        """the codes and scales of a pool's bytes"""
        p = pool.reshape(len(self.codes), self.L, self.slab)
        self.codes = p[:, :, :self.off_s].astype(np.int32).reshape(self.codes.shape) - 128
        n = 8 * self.H * (self.T // BLOCK)
        self.scales = np.ascontiguousarray(p[:, :, self.off_s:self.off_s + n]).view(np.float32).reshape(self.scales.shape).copy()

    def append(self, layer, half, table_row, length, x):
        """x f32 [n, H, D] are the last n of `length` tokens"""
        n = len(x)
        for h in range(self.H):
            t = length - n
            while t < length:
                blk = t // BLOCK
                end = min(length, (blk + 1) * BLOCK)
                page, slot = table_row[t // self.T], t % self.T
                sb = slot // BLOCK
                new = x[t - (length - n):end - (length - n), h].astype(np.float32)
                new = np.where(np.isnan(new), np.float32(0), new)
                fin = np.abs(new[np.isfinite(new)])
                amax = fin.max() if fin.size else np.float32(0)
                with np.errstate(under="ignore"):
                    d = f32(amax) * f32(f32(1) / f32(127))
                if d < np.finfo(np.float32).tiny:
                    d = f32(0)
                f = t % BLOCK
                old = self.scales[page, layer, half, h, sb] if f else f32(0)
                if f and old >= d:
                    d = old
                elif f:
                    r = f32(old) / f32(d)
                    q = self.codes[page, layer, half, h, sb * BLOCK:sb * BLOCK + f]
                    self.codes[page, layer, half, h, sb * BLOCK:sb * BLOCK + f] = away(q.astype(np.float32) * r)
                if d > 0:
                    with np.errstate(invalid="ignore", over="ignore"):
                        q = np.clip(away(np.clip(new * (f32(1) / d), -1e6, 1e6)), -127, 127)
                else:
                    q = np.zeros(new.shape)
                self.codes[page, layer, half, h, slot:slot + len(new)] = q
                self.scales[page, layer, half, h, sb] = d
                t = end

    def values(self, layer, half, table_row, pos):
        """q * d of the positions, in 64 bits [len(pos), H, D] (each product has at most 31 significant bits)"""
        pos = np.asarray(pos)
        page, slot = np.asarray(table_row)[pos // self.T], pos % self.T
        return self.codes[page, layer, half, :, slot].astype(np.float64) * self.scales[page, layer, half, :, slot // BLOCK].astype(np.float64)[..., None]


def attention(q, k, v, length, causal=True, window=0, scale=None):
    """q [n, Hq, D], k / v [length, H, D] in 64 bits; also returns, per row and head, the largest sum_d |q_d k_jd| scale
    and the largest |v| among what the row sees (for tolerances)."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1] if length else 1
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, mass, vmax = np.zeros((n, Hq, D)), np.zeros((n, Hq)), np.zeros((n, Hq))
    for i in range(n):
        p = length - n + i
        hi = min(p + 1, length) if causal else length
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        for x in range(Hq):
            h = x // G
            if not np.isfinite(q[i, x]).all():
                out[i, x] = np.nan
                continue
            s = (k[lo:hi, h] @ q[i, x]) * scale
            w = np.exp(s - s.max())
            out[i, x] = (w / w.sum()) @ v[lo:hi, h]
            mass[i, x] = (np.abs(k[lo:hi, h]) @ np.abs(q[i, x])).max() * abs(scale)
            vmax[i, x] = np.abs(v[lo:hi, h]).max()
    return out, mass, vmax


def attention_tolerance(out, mass, vmax, length, dtype):
    """How far a row may be from the 64-bit result, per element.

    Scores: q enters in two f16 parts (f32 rows; 2^-22 of each product) or exactly (16-bit rows), the f32 sums of the
    tensor cores and the scaling cost at most 2^-21 of sum |q k| scale; each is doubled for the maximum that is subtracted.
    A weight's relative error is that of its score, plus 2^-22 for exp2 and, in 16-bit rows, 2^-11 for rounding it to f16.
    A softmax average moves by at most twice the weights' relative error times the largest |v|; the sums over the tokens
    round at most once per 16 tokens, 2^-23 of the largest |v| each.  Then the output's own rounding."""
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    weight = 2 * (2.0 ** -21 + 2.0 ** -22) * mass + 2.0 ** -21 + (0 if dtype == "f32" else 2.0 ** -11)
    sums = (length / 16 + 8) * 2.0 ** -23
    # f16 outputs below 2^-14 are subnormal: 2^-25 absolute
    return (2 * weight + sums)[..., None] * vmax[..., None] + u * np.abs(out) + (2.0 ** -25 if dtype == "f16" else 1e-38)


def attention_own(q, k, v, d, length, dtype, causal=True, window=0):
    """attention() with a tolerance per element that knows only what the row sees and weighs: d [length, H] are the V scales.

    A weight's error (attention_tolerance; 2^-20 for exp2 and the factors between the two references) counts with its own token's
    w |v|, and in the sum of weights with the result; the sums with sum w |v|.  A weight times V scale below f16's subnormals is lost: 2^-30 of
    the row's largest, times at most 127, for each token."""
    n, Hq, D = q.shape
    G, scale = Hq // k.shape[1], 1 / np.sqrt(D)
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    out, tol = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for i in range(n):
        p = length - n + i
        hi, lo = min(p + 1, length) if causal else length, max(0, p - window + 1) if window else 0
        for x in range(Hq if hi > lo else 0):
            kk, vv, dd = k[lo:hi, x // G], v[lo:hi, x // G], d[lo:hi, x // G]
            s = kk @ q[i, x] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            e = 2 * (2.0 ** -21 + 2.0 ** -22) * (np.abs(kk) @ np.abs(q[i, x])) * scale + 2.0 ** -20 + (0 if dtype == "f32" else 2.0 ** -11)
            out[i, x] = w @ vv
            tol[i, x] = ((w * e) @ np.abs(vv) + np.abs(out[i, x]) * (w @ e) + (length / 16 + 8) * 2.0 ** -23 * (w @ np.abs(vv)) +
                         length * 2.0 ** -30 * 127 * (w * dd).max() + u * np.abs(out[i, x]) + (2.0 ** -25 if dtype == "f16" else 1e-38))
    return out, tol


# ----------------------------------------------------------------------------- pages ---

class Pages:
    """The page bookkeeping of include/mqkv.h on Python lists."""

    def __init__(self, n_pages, n_seqs, max_pages, T):
        self.T, self.max_pages = T, max_pages
        self.refs, self.len = [0] * n_pages, [0] * n_seqs
        self.table = [[] for _ in range(n_seqs)]

    def free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, add):
        need = [-(-(self.len[b] + a) // self.T) - len(self.table[b]) for b, a in enumerate(add)]
        if any(a < 0 for a in add) or any(len(self.table[b]) + k > self.max_pages for b, k in enumerate(need)):
            return False
        free = self.free()
        if sum(need) > len(free):
            return False
        for b, a in enumerate(add):
            for _ in range(need[b]):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[b].append(p)
            self.len[b] += a
        return True

    def release(self, ids):
        for b in ids:
            for p in self.table[b]:
                self.refs[p] -= 1
            self.table[b], self.len[b] = [], 0

    def fork(self, pairs):
        """the copies made: (source page, page, used blocks); None if the pool is too full (nothing changes)"""
        pairs = [(a, c) for i, (a, c) in enumerate(pairs) if self.len[c] == 0 and c not in [x for _, x in pairs[:i]]]
        free, copies = self.free(), []
        if sum(self.len[a] % self.T > 0 for a, _ in pairs) > len(free):
            return None
        for a, c in pairs:
            full, part = divmod(self.len[a], self.T)
            self.table[c] = self.table[a][:full]
            for p in self.table[c]:
                self.refs[p] += 1
            if part:
                p = free.pop(0)
                self.refs[p] = 1
                copies.append((self.table[a][full], p, -(-part // BLOCK)))
                self.table[c].append(p)
            self.len[c] = self.len[a]
        return copies

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return to

    def table_array(self, fill=-1):
        out = np.full((len(self.table), self.max_pages), fill, np.int32)
        for b, row in enumerate(self.table):
            out[b, :len(row)] = row
        return out

// mq_kv_append.cuh -- the append of new keys and values to the cache: what a block of threads does for some blocks of 32 slots
// and two vectors.  mq_kv_store.cu makes a kernel of it as it is, mq_kv_rope.cu one that turns the keys on their way (and the queries
// beside them).
#pragma once

#include <cfloat>
#include <type_traits>

#include "mq_kv.cuh"

namespace mq {

// the last sequence whose rows begin at or before row t (cu not falling): 32 ends at a time, one a lane
__device__ __forceinline__ int kv_find_seq(const KvRows &rows, int n_seqs, int64_t t, int step_per_seq, int shift) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;                                   // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int stride = (n + 31) / 32, at = min(lane * stride, n - 1);
        const int64_t begin = (rows.begin(lo + at) >> shift) + (int64_t)step_per_seq * (lo + at);
        const uint32_t yes = __ballot_sync(0xffffffffu, lane == 0 || begin <= t);
        // lanes past the end repeat the last sequence: the highest lane that says yes names its stride's beginning
        const int k = 31 - __clz(yes), from = min(k * stride, n - 1);
        lo += from;
        n = min(stride, n - from);
    }
    return lo;
}

// of a lane's values: the largest finite magnitude; whether all are finite
template <typename T, int IT>
__device__ __forceinline__ float amax_of(const Raw4<T> (&r)[IT], bool &finite) {
    float amax = 0.0f;
    if constexpr (sizeof(T) == 4) {
        uint64_t z = f2_pack(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < IT; ++i) scan4(r[i], amax, z);
        float a, b;
        f2_unpack(z, a, b);
        finite = a + b == 0.0f;
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const uint32_t none = 0;
        T2 m = *reinterpret_cast<const T2 *>(&none), z = m;
#pragma unroll
        for (int i = 0; i < IT; ++i) scan2(r[i].w.x, m, z), scan2(r[i].w.y, m, z);
        amax = fmaxf(to_f32(m.x), to_f32(m.y));
        finite = to_f32(z.x) + to_f32(z.y) == 0.0f;
    }
    if (!finite) {                                            // (rare) again, infinities aside
        amax = 0.0f;
#pragma unroll 1
        for (int i = 0; i < IT; ++i) {
            float x[4];
#pragma unroll
            for (int j = 0; j < IT; ++j)
                if (j == i) unpack4(r[j], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[e]) <= FLT_MAX ? fabsf(x[e]) : 0.0f);
        }
    }
    return amax;
}

constexpr int kAppendThreads = 256, kAppendVecs = 2, kAppendWarps = 8 / kAppendVecs;    // vectors per CTA, warps per vector

// A block of threads takes a group of `blocks` = 2^(shift - 5) consecutive blocks of 32 slots and two of the 2 H vectors (half, head), 2 y and 2 y + 1;
// four warps per vector, 8 slots each, all of a lane's values in registers between the maximum and the codes, the next block's asked for before this one's
// are worked on.  Unit u belongs to the last sequence b with U(b) <= u, U(b) = begin(b) / (32 blocks) + 2 b: a
// sequence of n tokens touches at most that many groups more, so the units of the sequences never overlap and need no prefix sum.
// ROPE::on: the keys are turned first, as f32.  rope.table (called by all threads, between barriers): the angles of the new slots [new0, new1)
// of the block that begins at position s0, position p being that of row p + row0.  rope.turn (by all lanes of a warp): a lane's
// four values 4 quad .. of new slot `slot` (whatever is not one of `slots` stays as it is).
struct NoRope {
    static constexpr bool on = false;
};
template <typename TIN, int D, typename ROPE>
__device__ __forceinline__ void kv_append_unit(const KvView &c, const KvRows &rows, int shift, int64_t u, int y, const TIN *k, int64_t kt,
                                               int64_t kh, const TIN *v, int64_t vt, int64_t vh, unsigned int *err, const ROPE &rope) {
    using V = typename std::conditional<ROPE::on, float, TIN>::type;
    constexpr int LPR = D / 4, RPW = 32 / LPR, IT = kKB / kAppendWarps / RPW;   // lanes per row, rows per warp and step, steps
    __shared__ float s_amax[2][8];
    const int blocks = 1 << (shift - 5);
    int b;
    int64_t u0;
    if (rows.cu == nullptr) {
        const int64_t per = (rows.each >> shift) + 2;
        b = (int)(u / per);
        u0 = b * per;
        if (b >= c.n_seqs) return;
    } else {
        b = kv_find_seq(rows, c.n_seqs, u, 2, shift);
        u0 = (rows.begin(b) >> shift) + 2 * (int64_t)b;
        if (u < u0) return;                                                     // (cu does not begin at 0: rows of no sequence)
    }
    int64_t lo, hi;
    rows.of(b, lo, hi);
    const int64_t n = hi - lo;
    if (n == 0) return;
    const int64_t len = c.len[b];
    if (len < n || ((len - 1) >> c.tshift) >= c.max_pages) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_LEN);
        return;
    }
    const int64_t p0 = len - n, first = p0 / kKB + (u - u0) * blocks;
    if (first * kKB >= len) return;
    const int count = (int)min((int64_t)blocks, (len + kKB - 1) / kKB - first);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane % LPR;
    const int vec = y * kAppendVecs + warp / kAppendWarps, half = vec >= c.H, h = vec - half * c.H;
    const bool in = vec < 2 * c.H;
    const TIN *src = (half ? v + h * vh : k + h * kh) + 4 * quad;
    const int64_t st = half ? vt : kt, step = st * RPW;
    const int r0 = kKB / kAppendWarps * (warp % kAppendWarps) + lane / LPR;     // this lane's first slot
    const int32_t *table = c.table + (int64_t)b * c.max_pages;

    Raw4<TIN> raw[IT];
    int page;
    auto ask = [&](int64_t blk) {                                               // a block's new values and its page
        page = table[blk >> (c.tshift - 5)];
        const int n0 = (int)max(p0 - blk * kKB, (int64_t)0), n1 = in ? (int)min(len - blk * kKB, (int64_t)kKB) : 0;
        const TIN *row = src + (lo + blk * kKB + r0 - p0) * st;
        if (n0 == 0 && n1 == kKB) {
#pragma unroll
            for (int i = 0; i < IT; ++i) raw[i] = *reinterpret_cast<const Raw4<TIN> *>(row + i * step);
        } else {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                raw[i].w = {};
                if (r0 + i * RPW >= n0 && r0 + i * RPW < n1) raw[i] = *reinterpret_cast<const Raw4<TIN> *>(row + i * step);
            }
        }
    };
    ask(first);
#pragma unroll 1
    for (int z = 0; z < count; ++z) {
        const int64_t s0 = (first + z) * kKB;
        const int new0 = (int)max(p0 - s0, (int64_t)0), new1 = (int)min(len - s0, (int64_t)kKB);   // slots of new tokens
        if constexpr (ROPE::on) rope.table(c, s0, new0, new1, lo - p0, y);
        Raw4<V> now[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if constexpr (ROPE::on) {
                float x[4];
                unpack4(raw[i], x);
                if (!half) rope.turn(x, r0 + i * RPW - new0, new1 - new0, quad, lane - quad);
                now[i].w = make_float4(x[0], x[1], x[2], x[3]);
            } else {
                now[i] = raw[i];
            }
        }
        const int pg = page;
        const bool there = pg >= 0 && pg < c.n_pages, ours = there && (c.refs == nullptr || c.refs[pg] == 1);
        const int slot0 = (int)(s0 & (c.T - 1));
        uint8_t *slab = c.pool + (ours ? pg : 0) * c.page_bytes;
        uint8_t *codes = slab + (half ? c.off_v : 0) + ((int64_t)h * c.T + slot0) * D + 4 * quad;
        float *scale = reinterpret_cast<float *>(slab + c.off_s) + vec * (c.T / kKB) + slot0 / kKB;
        float d_old = ours && in && new0 > 0 ? *scale : 0.0f;                   // slots of earlier tokens share the block
        if (!(d_old >= 0.0f && d_old <= FLT_MAX)) d_old = 0.0f;
        if (z + 1 < count) ask(first + z + 1);
        bool finite;
        float amax = amax_of(now, finite);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) s_amax[z & 1][warp] = amax;
        __syncthreads();
        if (!ours) {
            if (threadIdx.x == 0) kv_error(err, there ? KV_ERR_SHARED : KV_ERR_PAGE);
            continue;
        }
        if (!in) continue;
        const float *others = s_amax[z & 1] + warp / kAppendWarps * kAppendWarps;
        float d = __fmul_rn(fmaxf(fmaxf(others[0], others[1]), fmaxf(others[2], others[3])), 1.0f / 127.0f);
        if (d < FLT_MIN) d = 0.0f;
        d = fmaxf(d, d_old);
        const float id = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        const bool whole = new0 == 0 && new1 == kKB;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int r = r0 + i * RPW;
            if (whole || (r >= new0 && r < new1)) {
                float x[4];
                unpack4(now[i], x);
                if (!finite) {                                                  // NaN is zero, an infinity the end of the range
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = x[e] == x[e] ? fminf(fmaxf(x[e], -127.0f * d), 127.0f * d) : 0.0f;
                }
                const uint64_t f = f2_pack(id, id);
                *reinterpret_cast<uint32_t *>(codes + r * D) = pack_codes(f2_mul(f2_pack(x[0], x[1]), f), f2_mul(f2_pack(x[2], x[3]), f));
            }
        }
        if (new0 > 0 && d > d_old) {                                            // earlier codes under a larger scale
            const float shrink = __fdiv_rn(d_old, d);
#pragma unroll 4
            for (int i = 0; i < IT; ++i) {
                const int r = r0 + i * RPW;
                if (r < new0) {
                    uint32_t *dst = reinterpret_cast<uint32_t *>(codes + r * D);
                    const uint32_t old = *dst;
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = __fmul_rn(code_value(old, e), shrink);
                    *dst = pack_codes(f2_pack(y[0], y[1]), f2_pack(y[2], y[3]));
                }
            }
        }
        if (warp % kAppendWarps == 0 && lane == 0) *scale = d;
    }
}

struct AppendShape {
    int gy, shift;              // pairs of vectors; log2 of a unit's slots
    int64_t units;
};
inline AppendShape append_shape(const KvView &c, const KvRows &r) {
    // Four blocks to a CTA where that leaves a few CTAs per SM, one where it would not.  One / four, from f32 and from bf16: 512 tokens of 4 heads
    // of 128 3.4 / 7.2, 3.4 / 7.9 us, 3314 of them 5.8 / 8.6, 4.4 / 9.1; 10k of 8 heads 30 / 25, 23 / 24, 32k 86 / 63, 64 / 58 (two: 70, 59).
    const int gy = (2 * c.H + kAppendVecs - 1) / kAppendVecs;
    const int shift = (r.n_tokens >> 7) * gy >= 4 * sm_count() ? 7 : 5;
    const int64_t units = r.cu == nullptr ? c.n_seqs * ((r.each >> shift) + 2) : (r.n_tokens >> shift) + 2 * (int64_t)c.n_seqs;
    return {gy, shift, units};
}

}  // namespace mq

// mq_kv_store.cu -- the cache's writes and reads of values: quantizing new keys and values into their pages, and the
// values back out of them.  Both move each byte once; the arithmetic is a few instructions a value.
#include <cfloat>
#include <type_traits>

#include "mqd.cuh"

namespace mq {
namespace {

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

// One CTA per (group of `blocks` consecutive blocks of 32 slots, two of the 2 H vectors (half, head)); four warps per vector, 8 slots
// each, all of a lane's values in registers between the maximum and the codes, the next block's asked for before this one's
// are worked on.  Unit u of the grid's x belongs to the last sequence b with U(b) <= u, U(b) = begin(b) / (32 blocks) + 2 b: a
// sequence of n tokens touches at most that many groups more, so the units of the sequences never overlap and need no prefix sum.
// Moves 5 (f32) or 3 bytes a value: 32k tokens of 8 heads of 128 in 63 us from f32 (5.2 TB/s), 46 from f16 (4.3), 58 from bf16 (3.4; its
// kernel spills 88 bytes at three CTAs per SM).
template <typename TIN, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(TIN) == 4 ? 2 : 3) kv_append_kernel(KvView c, KvRows rows, int shift, const TIN *k, int64_t kt, int64_t kh,
                                                                      const TIN *v, int64_t vt, int64_t vh, unsigned int *err) {
    constexpr int LPR = D / 4, RPW = 32 / LPR, IT = kKB / kAppendWarps / RPW;   // lanes per row, rows per warp and step, steps
    __shared__ float s_amax[2][8];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t u = blockIdx.x;
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
    const int vec = blockIdx.y * kAppendVecs + warp / kAppendWarps, half = vec >= c.H, h = vec - half * c.H;
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
        Raw4<TIN> now[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) now[i] = raw[i];
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

constexpr int kReadTokens = 16, kReadThreads = 256;

// One CTA per 16 rows of the output, a warp per row and some of its 2 H vectors (half, head) at a time: their loads fly together.  Moves 5
// (f32) or 3 bytes a value: 40960 tokens of 8 heads of 128 at 6.3 and 6.1 TB/s (66 and 41 us).  A lane takes CPL codes: 4, or where 16-byte stores of 16-bit values
// fit 8.  32 rows a CTA: 67 and 41, and 64 tokens 5.2 for 3.6.
template <typename TOUT, int D, int CPL>
__global__ void __launch_bounds__(kReadThreads, 3) kv_read_kernel(KvView c, KvRows rows, TOUT *k, int64_t kt, int64_t kh, TOUT *v,
                                                               int64_t vt, int64_t vh, const int32_t *start, unsigned int *err) {
    constexpr int LPR = D / CPL, RPW = 32 / LPR, B = 2 * CPL / RPW, VECS = RPW * B;    // lanes per vector, vectors per load, loads in flight
    __shared__ const uint8_t *s_slab[kReadTokens];
    __shared__ int s_slot[kReadTokens];
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane % LPR;
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    const int nt = (int)min((int64_t)kReadTokens, rows.n_tokens - t0);
    const int heads = 2 * c.H;
    if (warp == 0) {
        // the sequence of the CTA's first row; the others' follow within a few
        int b = rows.cu == nullptr ? (int)(t0 / rows.each) : kv_find_seq(rows, c.n_seqs, t0, 0, 0);
        if (lane < nt) {
            const int64_t t = t0 + lane;
            if (rows.cu == nullptr) b = (int)(t / rows.each);
            else
                while (b + 1 < c.n_seqs && rows.begin(b + 1) <= t) ++b;
            int64_t lo, hi;
            rows.of(b, lo, hi);
            const int64_t len = c.len[b], n = hi - lo;
            const int64_t pos = (start != nullptr ? (int64_t)start[b] : len - n) + (t - lo);
            const uint8_t *slab = nullptr;
            if (t < lo || t >= hi || pos < 0 || pos >= len || (pos >> c.tshift) >= c.max_pages) {
                kv_error(err, KV_ERR_LEN);
            } else {
                const int page = c.table[(int64_t)b * c.max_pages + (pos >> c.tshift)];
                if (page < 0 || page >= c.n_pages) kv_error(err, KV_ERR_PAGE);
                else slab = c.pool + page * c.page_bytes;
            }
            s_slab[lane] = slab;
            s_slot[lane] = (int)(pos & (c.T - 1));
        }
    }
    __syncthreads();
    const int spp = c.T / kKB, step = RPW * c.T * D;
    for (int t = warp; t < nt; t += kReadThreads / 32) {
        const uint8_t *slab = s_slab[t];
        const int slot = s_slot[t], sub = lane / LPR;
        const uint8_t *src = slab + ((int64_t)sub * c.T + slot) * D + CPL * quad;
        const float *scale = reinterpret_cast<const float *>(slab + c.off_s) + sub * spp + slot / kKB;
        TOUT *to_k = k + (t0 + t) * kt + sub * kh + CPL * quad, *to_v = v + (t0 + t) * vt + (sub - c.H) * vh + CPL * quad;
        for (int v0 = 0; v0 < heads; v0 += VECS) {
            uint32_t w[B][CPL / 4];
            float d[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                d[i] = 0.0f;
#pragma unroll
                for (int q = 0; q < CPL / 4; ++q) w[i][q] = 0x80808080u;
                if (slab != nullptr && v0 + i * RPW + sub < heads) {
                    // K of every head, then V of every head: one run of vectors
                    if constexpr (CPL == 8) {
                        const uint2 two = *reinterpret_cast<const uint2 *>(src);
                        w[i][0] = two.x, w[i][1] = two.y;
                    } else {
                        w[i][0] = *reinterpret_cast<const uint32_t *>(src);
                    }
                    d[i] = *scale;
                }
                src += step, scale += RPW * spp;
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int vec = v0 + i * RPW + sub;
                const bool half = vec >= c.H;
                TOUT *dst = half ? to_v : to_k;
                to_k += RPW * kh, to_v += RPW * vh;
                if (vec >= heads || (half ? v : k) == nullptr) continue;
                float x[CPL];
#pragma unroll
                for (int e = 0; e < CPL; e += 2) f2_unpack(f2_mul(code_values(w[i][e / 4], e % 4), f2_pack(d[i], d[i])), x[e], x[e + 1]);
                if constexpr (CPL == 8) store8(dst, pack8(x, TOUT()));
                else store4(dst, x);
            }
        }
    }
}

template <typename T>
int append_t(const KvView &c, const KvRows &r, const void *k, int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh,
             unsigned int *err, cudaStream_t s) {
    // Four blocks to a CTA where that leaves a few CTAs per SM, one where it would not.  One / four, from f32 and from bf16: 512 tokens of 4 heads
    // of 128 3.4 / 7.2, 3.4 / 7.9 us, 3314 of them 5.8 / 8.6, 4.4 / 9.1; 10k of 8 heads 30 / 25, 23 / 24, 32k 86 / 63, 64 / 58 (two: 70, 59).
    const int gy = (2 * c.H + kAppendVecs - 1) / kAppendVecs;
    const int shift = (r.n_tokens >> 7) * gy >= 4 * sm_count() ? 7 : 5;
    const int64_t units = r.cu == nullptr ? c.n_seqs * ((r.each >> shift) + 2) : (r.n_tokens >> shift) + 2 * (int64_t)c.n_seqs;
    const dim3 grid((unsigned)units, gy);
    auto fn = c.D == 128 ? kv_append_kernel<T, 128> : kv_append_kernel<T, 64>;
    return cuda_error(launch_pdl(fn, grid, dim3(kAppendThreads), 0, s, c, r, shift, static_cast<const T *>(k), kt, kh,
                                 static_cast<const T *>(v), vt, vh, err),
                      "mqkv_append launch");
}

template <typename T>
int read_t(const KvView &c, const KvRows &r, void *k, int64_t kt, int64_t kh, void *v, int64_t vt, int64_t vh,
           const int32_t *start, unsigned int *err, cudaStream_t s) {
    const dim3 grid((unsigned)((r.n_tokens + kReadTokens - 1) / kReadTokens));
    auto fn = c.D == 128 ? kv_read_kernel<T, 128, 4> : kv_read_kernel<T, 64, 4>;
    if constexpr (sizeof(T) == 2) {
        // 40960 tokens of 8 heads of 128 to bf16: 8 codes a lane 41 us, 4 50; 64 tokens 3.6 and 4.3
        if (aligned(k, 16) && aligned(v, 16) && (kt % 8 | kh % 8 | vt % 8 | vh % 8) == 0) fn = c.D == 128 ? kv_read_kernel<T, 128, 8> : kv_read_kernel<T, 64, 8>;
    }
    return cuda_error(launch_pdl(fn, grid, dim3(kReadThreads), 0, s, c, r, static_cast<T *>(k), kt, kh, static_cast<T *>(v), vt,
                                 vh, start, err),
                      "mqkv_read launch");
}

}  // namespace

int kv_launch_append(const KvView &c, const KvRows &r, int dtype, const void *k, int64_t kt, int64_t kh, const void *v,
                     int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s) {
    return dtype == MQKV_F32   ? append_t<float>(c, r, k, kt, kh, v, vt, vh, err, s)
           : dtype == MQKV_F16 ? append_t<__half>(c, r, k, kt, kh, v, vt, vh, err, s)
                               : append_t<__nv_bfloat16>(c, r, k, kt, kh, v, vt, vh, err, s);
}

int kv_launch_read(const KvView &c, const KvRows &r, int dtype, void *k, int64_t kt, int64_t kh, void *v, int64_t vt,
                   int64_t vh, const int32_t *start, unsigned int *err, cudaStream_t s) {
    return dtype == MQKV_F32   ? read_t<float>(c, r, k, kt, kh, v, vt, vh, start, err, s)
           : dtype == MQKV_F16 ? read_t<__half>(c, r, k, kt, kh, v, vt, vh, start, err, s)
                               : read_t<__nv_bfloat16>(c, r, k, kt, kh, v, vt, vh, start, err, s);
}

}  // namespace mq

// mq_kv_prefill.cu -- attention over the paged 8-bit cache for many rows per KV head (prompts and chunks of them) on
// tcgen05: the products bound it, so everything else is arranged to keep the tensor core fed.
//
// Mathematics: that of mq_kv_attn.cu, in tiles of 128 rows x 128 tokens.  K and V codes are exact in f16, so
// S = Q K^T accumulates exact products; a tile's score is S times (row scale) (K scale of the token's block), the
// weights enter the second product as p' = 2^(s - m + shift) dv / g in f16.  f32 rows use two f16 parts of q and
// of p' (twice the MMAs, f32 accuracy).  The reference m of a row moves only when its maximum grows by more than
// kTau (powers of two, so the result does not depend on it beyond rounding), and g only when a V scale exceeds it, then to
// twice that: O is rescaled a few times per row instead of at every tile.
//
// CTA = 16 warps, two row tiles that share every K / V tile: warps 0-3 and 4-7 softmax of tile 0 and 1 (a thread
// per row, the whole row of S in registers), 8-11 widen codes (raw bytes -> f16 operand tiles, 128-byte swizzle),
// 12 TMA of the raw pages and the scales, 13 MMA issuer.  Order on the tensor core: PV0(j) S0(j+1) PV1(j) S1(j+1), so
// the softmax of one tile runs under the products of the other.  P replaces S in TMEM (f16, A operand from TMEM);
// V is the MN-major B operand, so it needs no transposition.
#include <cuda.h>

#include <climits>
#include <type_traits>

#include "mq_kv_attn.cuh"

namespace mq {
namespace {

constexpr int kPfThreads = 512;
constexpr int kPfRows = 256, kPfN = 128;       // rows of a CTA, tokens of a tile
constexpr float kTau = 8.0f, kPfShift = 6.0f;   // p' <= 2^(6 + 8) in f16

struct PfArgs {
    KvView c;
    KvRows r;
    const void *q;
    void *out;
    int64_t qt, qh, ot, oh;
    int32_t group, causal, tiles, layer;
    int64_t max_q, window;
    float c_log2;               // |scale| * log2(e)
    float sign;                 // of scale: folded into q, so that the score factors are not negative
};

template <int D, bool TWO>
struct PfCfg {
    static constexpr int PARTS = TWO ? 2 : 1;
    static constexpr int NS = TWO ? 2 : 4;                     // f16 operand tiles in flight (K0 V0 K1 V1 ...)
    static constexpr int OPT = kPfN * D * 2, RAWT = kPfN * D;
    static constexpr int QT = 128 * D * 2;                     // one part of one row tile
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_OP = OFF_Q + PARTS * 2 * QT;
    static constexpr int OFF_RAW = OFF_OP + NS * OPT;
    static constexpr int OFF_RS = OFF_RAW + 2 * RAWT;          // row scales [256]
    static constexpr int OFF_INFO = OFF_RS + kPfRows * 4;      // [4 tiles][dk[4], dv[4]]
    static constexpr int OFF_BAR = OFF_INFO + 4 * 8 * 4;
    static constexpr int NBAR = 2 + 2 + 2 * NS + 4 + 2 + 2 + 2 + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA exceeds the per-CTA limit");
    static constexpr uint32_t COL_S = 0, COL_O = 256;
};

__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16: A holds two f16 per 32-bit column
__device__ __forceinline__ void mma_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Descriptor of an MN-major operand tile with the 128-byte swizzle: K rows (tokens) of 64 f16 = 128 B, 8-row atoms of
// 1024 B; `mn_stride` bytes from 64 columns to the next 64
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t addr, uint32_t mn_stride) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((mn_stride >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// a wait whose outcome is the same for the whole warp (a warp gives up together)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned int *err, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait_prompt(bar, parity, err, KV_ERR_WAIT, abort));
}

template <typename T, int D>
__global__ void __launch_bounds__(kPfThreads, 1) kv_prefill_kernel(const __grid_constant__ CUtensorMap tm, PfArgs a, unsigned int *err) {
    constexpr bool TWO = sizeof(T) == 4;
    using C = PfCfg<D, TWO>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *s_rs = reinterpret_cast<float *>(sm + C::OFF_RS);
    float *s_info = reinterpret_cast<float *>(sm + C::OFF_INFO);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    uint64_t *raw_full = bar, *raw_empty = bar + 2, *op_full = bar + 4, *op_empty = op_full + NS, *info_full = op_empty + NS,
             *s_full = info_full + 4, *p_full = s_full + 2, *o_done = p_full + 2, *drain = o_done + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sm + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_dep_launch();
    grid_dep_wait();
    // the CTA's rows: KV head fastest, then the sequence, the latest (longest) row tiles first
    int64_t u = blockIdx.x;
    const int h = (int)(u % a.c.H);
    u /= a.c.H;
    const int b = (int)(u % a.c.n_seqs), tile = a.tiles - 1 - (int)(u / a.c.n_seqs);
    int64_t lo, hi;
    a.r.of(b, lo, hi);
    int64_t n = hi - lo;
    if (n > a.max_q) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_ROWS);
        n = a.max_q;
    }
    const int64_t len = a.c.len[b], first = len - (hi - lo);
    const int G = a.group;
    const int64_t rows = n * G, r0 = (int64_t)tile * kPfRows;
    if (r0 >= rows) return;
    const bool bad = len < 0 || (len > 0 && ((len - 1) >> a.c.tshift) >= a.c.max_pages);
    if (bad && threadIdx.x == 0) kv_error(err, KV_ERR_LEN);
    const int nrow = (int)min((int64_t)kPfRows, rows - r0);
    const int nt = nrow > 128 ? 2 : 1;                         // row tiles
    // what the rows see: the ranges' ends do not fall from row to row
    int64_t t_lo = 0, t_hi = 0, all_lo = 0, all_hi = 0;
    if (!bad) {
        int64_t x0, y0, x1, y1;
        row_range(first + r0 / G, len, a.causal, a.window, x0, y0);
        row_range(first + (r0 + nrow - 1) / G, len, a.causal, a.window, x1, y1);
        all_lo = max(x0, x1), all_hi = y0 > x0 ? min(y0, y1) : 0;
        // the first row that sees anything starts no later than any other
        t_hi = y1;
        t_lo = y0 > x0 ? x0 : 0;
        if (y1 <= x1) {                                        // the last row sees nothing: nor does any other
            t_hi = 0;
            if (y0 > x0) t_hi = y0, t_lo = x0;                   // (a window past the cache's end, without causality)
        }
    }
    const int64_t b_lo = t_lo / kKB, b_hi = (t_hi + kKB - 1) / kKB;
    const int nj = (int)((b_hi - b_lo + 3) / 4);               // token tiles
    const int64_t base = b_lo * kKB;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(raw_full + i, 1);
            mbar_init(raw_empty + i, 128);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 128);
            mbar_init(o_done + i, 1);
        }
        for (int i = 0; i < NS; ++i) mbar_init(op_full + i, 128), mbar_init(op_empty + i, 1);
        for (int i = 0; i < 4; ++i) mbar_init(info_full + i, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 13) tmem_alloc(tmem_holder, 512);
    // q of the rows as f16 parts in the K-major swizzled layout, a warp per row; rows that are not there are zeros
#pragma unroll 1
    for (int r = warp; r < nt * 128; r += kPfThreads / 32) {
        float x[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = 0.0f;
        if (r < nrow) {
            const int64_t rr = r0 + r, i = rr / G;
            const T *p = static_cast<const T *>(a.q) + (lo + i) * a.qt + (int64_t)(h * G + (int)(rr - i * G)) * a.qh + lane * (D / 32);
            if constexpr (D == 128) {
                load4(p, x);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) x[e] = static_cast<float>(p[e]);
            }
        }
        float amax = 0.0f;
        bool fin = true;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            amax = fmaxf(amax, fabsf(x[e]));
            fin = fin && fabsf(x[e]) <= 3.402823466e38f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        fin = __all_sync(0xffffffffu, fin);
        const int ex = fin ? row_exponent(amax) : 0;
        const float down = fin ? pow2i(-ex) * a.sign : __int_as_float(0x7fc00000);   // a row with a NaN or an infinity becomes NaN
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = fin ? x[e] * down : down;
        const int t = r >> 7, rt = r & 127, col = lane * (D / 32);
        // 16-byte unit (col / 8) % 8 of row rt in the 64-column half col / 64
        uint8_t *dst = sm + C::OFF_Q + t * C::QT + (col >> 6) * 16384 + rt * 128 + ((((col >> 3) & 7) ^ (rt & 7)) << 4) + (col & 7) * 2;
#pragma unroll
        for (int e = 0; e < D / 32; e += 2) {
            const uint32_t p0 = pack_f16(x[e], x[e + 1]);
            *reinterpret_cast<uint32_t *>(dst + 2 * e) = p0;
            if constexpr (TWO) {
                const float2 f = unpack_f16(p0);
                *reinterpret_cast<uint32_t *>(dst + 2 * C::QT + 2 * e) = pack_f16(x[e] - f.x, x[e + 1] - f.y);
            }
        }
        if (lane == 0) s_rs[r] = pow2i(ex) * a.c_log2;
    }
    fence_proxy_async_smem();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 12) {
            // ---------------------------------------------------------------- raw pages and scales
            int pg = -1;
            float dk = 0.0f, dv = 0.0f;
            auto fetch = [&](int64_t blk0) {                   // one block a lane, from blk0 on
                pg = -1, dk = dv = 0.0f;
                const int64_t blk = blk0 + lane;
                if (blk < b_hi) {
                    pg = a.c.table[(int64_t)b * a.c.max_pages + ((blk * kKB) >> a.c.tshift)];
                    if (pg < 0 || pg >= a.c.n_pages) {
                        kv_error(err, KV_ERR_PAGE);
                        pg = -1;
                    } else {
                        const float *sc = reinterpret_cast<const float *>(a.c.pool + pg * a.c.page_bytes + a.c.off_s);
                        const int sb = (int)((blk * kKB) & (a.c.T - 1)) / kKB, spp = a.c.T / kKB;
                        dk = sc[h * spp + sb];
                        dv = sc[(a.c.H + h) * spp + sb];
                    }
                }
            };
            int issued = 0;
            for (int i = 0; i < 2 * nj; ++i) {
                const int j = i >> 1, half = i & 1, slot = i & 1;
                if (half == 0 && (j & 7) == 0) fetch(b_lo + 4 * (int64_t)j);
                const int l0 = 4 * (j & 7);
                const int nb = (int)min((int64_t)4, b_hi - (b_lo + 4 * (int64_t)j));
                if (i >= 2 && !warp_wait(raw_empty + slot, ((i >> 1) - 1) & 1, err, abort_flag)) break;
                if (half == 0) {
                    const int e = lane - l0;
                    if (e >= 0 && e < 4) s_info[(j & 3) * 8 + e] = dk, s_info[(j & 3) * 8 + 4 + e] = dv;
                    __threadfence_block();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(info_full + (j & 3));
                }
                if (lane == 0) mbar_arrive_expect_tx(raw_full + slot, nb * kKB * D);
                __syncwarp();
                const int e = lane - l0;
                if (e >= 0 && e < nb) {
                    const int64_t blk = b_lo + 4 * (int64_t)j + e;
                    tma_load_5d(sm + C::OFF_RAW + slot * C::RAWT + e * kKB * D, &tm, 0, (int)((blk * kKB) & (a.c.T - 1)), half * a.c.H + h, a.layer,
                                pg, raw_full + slot);
                }
                issued = i + 1;
            }
            if (*abort_flag)                                   // copies in flight land before the CTA ends
                for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i) mbar_wait(raw_full + (i & 1), (i >> 1) & 1, err, KV_ERR_WAIT, nullptr);
        } else if (warp == 13) {
            // ---------------------------------------------------------------- MMA issuer
            constexpr uint32_t id_s = idesc_f16_f32(128, kPfN);
            constexpr uint32_t id_o = idesc_f16_f32(128, D) | (1u << 16);       // B (V) MN-major
            const uint32_t q0 = smem_u32(sm + C::OFF_Q), op0 = smem_u32(sm + C::OFF_OP);
            auto scores = [&](int t, int slot) {
#pragma unroll
                for (int part = 0; part < C::PARTS; ++part)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
                        mma_f16_warp(tmem + C::COL_S + t * 128, sw128_kmajor_desc(q0 + (part * 2 + t) * C::QT + off),
                                     sw128_kmajor_desc(op0 + slot * C::OPT + off), id_s, part + ks > 0);
                    }
                mma_commit_warp(s_full + t);
            };
            auto output = [&](int t, int slot, int j) {
#pragma unroll
                for (int part = 0; part < C::PARTS; ++part)
#pragma unroll
                    for (int ks = 0; ks < kPfN / 16; ++ks)
                        mma_f16_ts_warp(tmem + C::COL_O + t * D, tmem + C::COL_S + t * 128 + part * 64 + ks * 8,
                                        sw128_mnmajor_desc(op0 + slot * C::OPT + ks * 2048, 16384), id_o, j + part + ks > 0);
                mma_commit_warp(o_done + t);
            };
            bool ok = nj > 0;
            if (ok) {
                ok = warp_wait(op_full, 0, err, abort_flag);
                tc_fence_after();
                if (ok) {
                    for (int t = 0; t < nt; ++t) scores(t, 0);
                    mma_commit_warp(op_empty);
                }
            }
            for (int j = 0; ok && j < nj; ++j) {
                const int iv = 2 * j + 1, ik = 2 * j + 2;
                if (!(ok = warp_wait(op_full + iv % NS, (iv / NS) & 1, err, abort_flag))) break;
                for (int t = 0; t < nt; ++t) {
                    if (!(ok = warp_wait(p_full + t, j & 1, err, abort_flag))) break;
                    tc_fence_after();
                    output(t, iv % NS, j);
                    if (t == nt - 1) mma_commit_warp(op_empty + iv % NS);
                    if (j + 1 < nj) {
                        if (t == 0) {
                            if (!(ok = warp_wait(op_full + ik % NS, (ik / NS) & 1, err, abort_flag))) break;
                            tc_fence_after();
                        }
                        scores(t, ik % NS);
                        if (t == nt - 1) mma_commit_warp(op_empty + ik % NS);
                    }
                }
            }
            if (*abort_flag) {                                 // products in flight end before the TMEM is freed
                mma_commit_warp(drain);
                mbar_wait(drain, 0, err, KV_ERR_WAIT, nullptr);
            }
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // -------------------------------------------------------------------- widen codes: a thread per token
        const int row = threadIdx.x - 256;
        for (int i = 0; i < 2 * nj; ++i) {
            const int rs = i & 1, slot = i % NS;
            if (!mbar_wait_prompt(raw_full + rs, (i >> 1) & 1, err, KV_ERR_WAIT, abort_flag)) break;
            if (i >= NS && !mbar_wait_prompt(op_empty + slot, (i / NS - 1) & 1, err, KV_ERR_WAIT, abort_flag)) break;
            const uint8_t *src = sm + C::OFF_RAW + rs * C::RAWT + row * D;
            uint8_t *dst = sm + C::OFF_OP + slot * C::OPT + row * 128;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const int pc = D == 128 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));
                const uint4 w = *reinterpret_cast<const uint4 *>(src + pc * 16);
                uint4 x, y;
                codes_f16(w.x, x.x, x.y);
                codes_f16(w.y, x.z, x.w);
                codes_f16(w.z, y.x, y.y);
                codes_f16(w.w, y.z, y.w);
                uint8_t *d = dst + (c >> 2) * 16384;
                const int unit = 2 * (c & 3);
                *reinterpret_cast<uint4 *>(d + ((unit ^ (row & 7)) << 4)) = x;
                *reinterpret_cast<uint4 *>(d + (((unit + 1) ^ (row & 7)) << 4)) = y;
            }
            fence_proxy_async_smem();
            mbar_arrive(op_full + slot);
            mbar_arrive(raw_empty + rs);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // -------------------------------------------------------------------- softmax: a thread per row
        const int t = warp >> 2, r = threadIdx.x;
        if (t < nt) {
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t ts = tmem + C::COL_S + t * 128 + lanes, to = tmem + C::COL_O + t * D + lanes;
            int v0 = 0, v1 = 0;                                 // what the row sees, from the first tile's start
            if (r < nrow && !bad) {
                int64_t x, y;
                row_range(first + (r0 + r) / G, len, a.causal, a.window, x, y);
                v0 = (int)max(x - base, (int64_t)0), v1 = (int)max(y - base, (int64_t)0);
            }
            const int i_lo = (int)max(all_lo - base, (int64_t)INT_MIN), i_hi = (int)max(all_hi - base, (int64_t)INT_MIN);
            const float rs = s_rs[r];
            float m = -INFINITY, g = 0.0f;
            uint64_t l2 = f2_pack(0.0f, 0.0f);
            bool ok = true;
            for (int j = 0; j < nj; ++j) {
                if (!(ok = warp_wait(info_full + (j & 3), (j >> 2) & 1, err, abort_flag))) break;
                float kb[4], dv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // at least 2^-120, so that a masked score stays minus infinity under a scale of zero
                    kb[e] = fmaxf(rs * s_info[(j & 3) * 8 + e], 0x1p-120f);
                    dv[e] = s_info[(j & 3) * 8 + 4 + e];
                }
                const float dmax = fmaxf(fmaxf(dv[0], dv[1]), fmaxf(dv[2], dv[3]));
                float gf = 1.0f;
                if (dmax > g) {
                    gf = g / (2.0f * dmax);
                    g = 2.0f * dmax;
                }
                const float ig = g > 0.0f ? 1.0f / g : 0.0f;
                if (!(ok = warp_wait(s_full + t, j & 1, err, abort_flag))) break;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int e = 0; e < 4; ++e) tmem_ld32(ts + 32 * e, s[e]);
                tmem_ld_wait();
                const int t0 = j * kPfN;
                if (!(t0 >= i_lo && t0 + kPfN <= i_hi)) {
                    const int x0 = v0 - t0, x1 = v1 - t0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * e + k < x0 || 32 * e + k >= x1) s[e][k] = 0xff800000u;
                }
                float mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y = __uint_as_float(s[e][0]);
#pragma unroll
                    for (int k = 1; k < 32; ++k) y = fmaxf(y, __uint_as_float(s[e][k]));
                    mx = fmaxf(mx, y * kb[e]);
                }
                const bool grow = mx > m + kTau || (m == -INFINITY && mx > m);
                if (__any_sync(0xffffffffu, grow || gf != 1.0f)) {
                    const float mn = grow ? mx : m;
                    const float f = mn == -INFINITY ? 1.0f : exp2_approx(m - mn);
                    m = mn;
                    l2 = f2_mul(l2, f2_pack(f, f));
                    if (j > 0) {
                        if (!(ok = warp_wait(o_done + t, (j - 1) & 1, err, abort_flag))) break;
                        tc_fence_after();
                        const uint64_t ff = f2_pack(f * gf, f * gf);
#pragma unroll
                        for (int e = 0; e < D / 16; ++e) {
                            uint32_t o[16];
                            tmem_ld16(to + 16 * e, o, 0);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                float x, y;
                                f2_unpack(f2_mul(f2_pack(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), ff), x, y);
                                o[k] = __float_as_uint(x), o[k + 1] = __float_as_uint(y);
                            }
                            tmem_st16(to + 16 * e, o);
                        }
                    }
                }
                const float off = kPfShift - (m == -INFINITY ? 0.0f : m);
                const uint64_t off2 = f2_pack(off, off);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t kk = f2_pack(kb[e], kb[e]);
                    const float pv = dv[e] * ig;
                    const uint64_t pp = f2_pack(pv, pv);
                    uint64_t acc = f2_pack(0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float x, y;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e][k]), __uint_as_float(s[e][k + 1])), kk, off2), x, y);
                        const uint64_t p = f2_pack(exp2_approx(x), exp2_approx(y));
                        acc = f2_add(acc, p);
                        f2_unpack(f2_mul(p, pp), x, y);
                        const uint32_t w = pack_f16(x, y);
                        s[e][k] = w;                           // the parts take the places of the two scores
                        if constexpr (TWO) {
                            const float2 z = unpack_f16(w);
                            s[e][k + 1] = pack_f16(x - z.x, y - z.y);
                        }
                    }
                    l2 = f2_add(l2, acc);
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = s[e][2 * k], w[16 + k] = s[e + 1][2 * k];
                    tmem_st32(ts + 16 * e, w);
                    if constexpr (TWO) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[k] = s[e][2 * k + 1], w[16 + k] = s[e + 1][2 * k + 1];
                        tmem_st32(ts + 64 + 16 * e, w);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_full + t);
            }
            // ---------------------------------------------------------------- the rows' outputs
            if (nj > 0 && ok) ok = warp_wait(o_done + t, (nj - 1) & 1, err, abort_flag);
            tc_fence_after();
            float l, l1;
            f2_unpack(l2, l, l1);
            l += l1;
            const float inv = l == 0.0f ? 0.0f : g / l;
            const int64_t i = (r0 + r) / G;
            const int gq = (int)(r0 + r - i * G);
            T *dst = static_cast<T *>(a.out) + (lo + i) * a.ot + (int64_t)(h * G + gq) * a.oh;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                uint32_t o[32];
                if (nj > 0) {
                    tmem_ld32(to + 32 * e, o);
                    tmem_ld_wait();
                }
                if (r < nrow) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float x[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) x[z] = nj > 0 && l != 0.0f ? __uint_as_float(o[k + z]) * inv : 0.0f;
                        store4(dst + 32 * e + k, x);
                    }
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

template <typename T, int D>
int kv_prefill_t(const CUtensorMap &tm, const PfArgs &a, unsigned int *err, cudaStream_t s) {
    using C = PfCfg<D, sizeof(T) == 4>;
    const int slot = kAttrSlotKv + 8 + 2 * (sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 1 : 2) + (D == 128);
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(&kv_prefill_kernel<T, D>), C::SMEM, slot);
    if (rc != MQ_OK) return rc;
    return cuda_error(launch_pdl(kv_prefill_kernel<T, D>, dim3((unsigned)((int64_t)a.c.H * a.c.n_seqs * a.tiles)), dim3(kPfThreads), C::SMEM, s, tm,
                                 a, err),
                      "mqkv_attention (tiles) launch");
}

int kv_launch_prefill(const CUtensorMap &tm, int layer, const KvView &c, const KvRows &r, const KvAttn &p, unsigned int *err,
                      cudaStream_t s) {
    PfArgs a;
    a.c = c, a.r = r, a.q = p.q, a.out = p.out, a.qt = p.qt, a.qh = p.qh, a.ot = p.ot, a.oh = p.oh;
    a.group = p.group, a.causal = p.causal, a.layer = layer, a.max_q = p.max_q, a.window = p.window;
    a.tiles = (int)((p.max_q * p.group + kPfRows - 1) / kPfRows);
    a.c_log2 = fabsf(p.scale) * kLog2e;
    a.sign = p.scale < 0.0f ? -1.0f : 1.0f;
    if (c.D == 128)
        return p.dtype == MQKV_F32   ? kv_prefill_t<float, 128>(tm, a, err, s)
               : p.dtype == MQKV_F16 ? kv_prefill_t<__half, 128>(tm, a, err, s)
                                     : kv_prefill_t<__nv_bfloat16, 128>(tm, a, err, s);
    return p.dtype == MQKV_F32   ? kv_prefill_t<float, 64>(tm, a, err, s)
           : p.dtype == MQKV_F16 ? kv_prefill_t<__half, 64>(tm, a, err, s)
                                 : kv_prefill_t<__nv_bfloat16, 64>(tm, a, err, s);
}

}  // namespace mq

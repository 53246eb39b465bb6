// mq_kv_prefill.cu -- attention over the paged 8-bit cache for many rows per KV head (prompts and chunks of them) on
// tcgen05: the products bound it, so everything else is arranged to keep the tensor core fed.
//
// Mathematics: that of mq_kv_attn.cu, in tiles of 128 rows x 128 tokens.  K and V codes are exact in f16, so
// S = Q K^T accumulates exact products; a tile's score is S times (row scale) (K scale of the token's block).
//
// Both kernels: 16 warps; 8-11 widen codes (global memory -> registers -> f16 operand tiles with the 128-byte swizzle, a
// ring of five, of four for f32 rows), 12 looks up pages and scales ahead of everyone, 13 issues the MMAs, 14 looks over the
// sequence's table entries; a softmax thread owns a row and reads its scores from TMEM, 32 or 64 at a time.  P replaces S in
// TMEM (f16, the A operand comes from TMEM); V is the MN-major B operand, so nothing is transposed.
//
// 16-bit rows (kv_tiles_kernel): two row tiles (256 rows) share every K / V tile, warps 0-3 and 4-7 their softmax; the
// tensor core runs PV0(j) S0(j+1) PV1(j) S1(j+1), the softmax of one tile under the products of the other.  A row's
// references move only when the maximum grows by more than kTau (a factor that cancels in o / l), so O in TMEM is rescaled a
// few times per row instead of at every tile.  (V as f16(code * f16(256 dv / g)) took the factor off the weights and 3% off the time, but its two
// roundings showed in f16 outputs.)
//
// Their weights are one f16 part: the worst of 320 f16 rows over 2048, 8192 and 16384 tokens of either sign is 4.0e-4 to 4.3e-4 off, with the
// rounding of the outputs alone 2.5e-4; of one sign 2.7e-4 for 2.7e-4.  O stays in TMEM over a row tile's whole length, where the tensor
// core cuts its sums toward zero (f32 rows, below, do not let it): of one sign 3.2e-4 at 32768 tokens and 4.8e-4 at 65536, for 2.5e-4 and
// 1.8e-4.  bf16 outputs show neither (2.0e-3 with and without).
//
// Many rows of long sequences are 636 jobs of 40 to 64 tiles in the largest case measured: 434 us, 1060 TFLOP/s (of 1864 that cuBLAS
// reaches; issue 49%); what is left is the chain MMA - commit - softmax - arrival - MMA of each tile and a CTA's beginning
// and end (8 tiles' time).
//
// f32 rows (kv_tiles_f32_kernel): q and the weights enter as two f16 parts each (twice the MMAs), V as its exact codes.
// The tensor core's f32 accumulation truncates; over a long row of tiles that grew to 4e-6 of the result (3314 tokens), so
// each tile's P V goes to a fresh accumulator and is added to the row's sum in registers, rounding to nearest, under the
// products of the next tiles: one row tile per CTA, S and O double-buffered, warps 0-3 and 4-7 the softmax of the tiles in turn.  A prompt
// of 3314 tokens, 28 query heads on 4 of 128: 183 us (157 GFLOP in two parts: 858 TFLOP/s); the tiles' chain bounds it
// (tensor pipe 36%, issue 48%).
//
// q is staged by the softmax warps while the others look up and widen the first tiles: with all warps and before everything else, a CTA's
// beginning took 5 us more (the prompt 187 us, the 16-bit chunks 478).
#include <cuda.h>

#include <climits>
#include <type_traits>

#include "mq_kv_attn.cuh"

namespace mq {
namespace {

constexpr int kPfThreads = 512;
constexpr int kPfN = 128;                      // tokens of a tile
constexpr int kPfSlots = 5;                    // f16 operand tiles in flight at most
constexpr int kPfInfo = 4;                     // tiles that the lookup runs ahead
// What a wave of pieces costs beside its tiles, the join, and each piece for the join, in tiles of 128 tokens (0.9 to 1.5 us each)
constexpr double kPfPieceSteps = 8, kPfJoinSteps = 4, kPfPartSteps = 0.5;

struct PfArgs {
    KvView c;
    KvRows r;
    const void *q;
    void *out;
    int64_t qt, qh, ot, oh;
    int32_t group, causal, tiles;
    int32_t cut, pieces;        // the last `cut` row tiles (in the grid's order) are done in `pieces` pieces
    float *part;                // [piece][row][D + 4]: the mean, m, l
    int64_t max_q, window;
    float c_log2;               // |scale| * log2(e)
    float sign;                 // of scale: folded into q, so that the score factors are not negative
};

// what the lookup leaves for a tile of four blocks
struct PfInfo {
    float dk[4], dv[4], lv[4];  // K scales; V scales and their binary logarithms
    int page[4];                // -1: no such block (codes of zero)
};

template <int D, bool TWO>
struct PfCfg {
    static constexpr int PARTS = TWO ? 2 : 1, TILES = TWO ? 1 : 2, ROWS = 128 * TILES;
    static constexpr int SLOTS = TWO ? 4 : 5;                  // f16 operand tiles in flight
    static constexpr int OPT = kPfN * D * 2;
    static constexpr int QT = 128 * D * 2;                     // one part of one row tile
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_OP = OFF_Q + PARTS * TILES * QT;
    static constexpr int OFF_RS = OFF_OP + SLOTS * OPT;     // row scales [ROWS]; f32 rows: then factors, references A [4][128] each, maxima and sums [2][2][128]
    static constexpr int OFF_INFO = OFF_RS + ROWS * 4 + (TWO ? 3 * 512 * 4 : 0);
    static constexpr int OFF_BAR = OFF_INFO + kPfInfo * (int)sizeof(PfInfo);
    static constexpr int NBAR = 2 * kPfSlots + 2 * kPfInfo + 5 * 2 + 4;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1008;
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA exceeds the per-CTA limit");
    static constexpr uint32_t COL_S = 0, COL_O = 256;
};

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

// The instruction cache is a resource here: four roles run their own straight-line code, and a fully unrolled version stalled on
// instruction fetch more than on anything but memory.  So loops are unrolled only as far as the latencies ask.

// A bounded wait whose outcome is the same for the whole warp (a warp gives up together).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned int *err, volatile int *abort) {
    const uint32_t at = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait(at, parity)); ++i) {
        if ((i & 255u) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            const bool late = now - t0 > kWaitTimeoutNs;
            if (__any_sync(0xffffffffu, late || *abort)) {
                if (late) kv_error(err, KV_ERR_WAIT);
                *abort = 1;
                return false;
            }
        }
    }
    return true;
}
// two barriers at once: each probe costs 130 to 150 clocks, side by side they cost one
__device__ __forceinline__ bool warp_wait2(uint64_t *bar, uint64_t *bar2, uint32_t parity, uint32_t parity2, unsigned int *err, volatile int *abort) {
    const bool one = mbar_try_wait(smem_u32(bar), parity), two = mbar_try_wait(smem_u32(bar2), parity2);
    if (__all_sync(0xffffffffu, one && two)) return true;
    return warp_wait(bar, parity, err, abort) && warp_wait(bar2, parity2, err, abort);
}
__device__ __forceinline__ bool warp_wait2(uint64_t *bar, uint64_t *bar2, uint32_t parity, unsigned int *err, volatile int *abort) {
    return warp_wait2(bar, bar2, parity, parity, err, abort);
}
__device__ __forceinline__ bool warp_wait3(uint64_t *bar, uint64_t *bar2, uint64_t *bar3, uint32_t parity, uint32_t parity2, uint32_t parity3,
                                           unsigned int *err, volatile int *abort) {
    const bool one = mbar_test_wait(smem_u32(bar), parity), two = mbar_test_wait(smem_u32(bar2), parity2);
    const bool three = mbar_try_wait(smem_u32(bar3), parity3);
    if (__all_sync(0xffffffffu, one && two && three)) return true;
    return warp_wait(bar, parity, err, abort) && warp_wait(bar2, parity2, err, abort) && warp_wait(bar3, parity3, err, abort);
}
// one arrival for the warp, after what its lanes did
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// A wait looks at a phase's parity only, so a barrier must not complete a phase while a warp that waits for the one before it has not
// looked.  Why none does (tests/test_kv_tiles_model.py walks the waits and arrivals of both kernels through schedules):
//   op_full, op_empty    the ring: a place is filled after its products were committed, which came after both fillers' arrivals
//   info_full, info_empty  the lookup's ring: refilled after every reader has arrived
//   s_full[b]            the next scores of a buffer are issued after p_full of its last ones, to which every reader of s_full arrives
//   p_full[b]            only the MMA warp waits; the next weights need scores that it issues after that wait
//   o_done[b]            f32 rows: the next products wait for o_free, to which all eight warps arrive.  16-bit rows: they wait for p_full of
//                        the same row tile, to which its four warps arrive
//   o_free[b]            only the MMA warp waits; the warps' next arrivals need products that it issues after that wait
//   m_full[b]            the warpgroup that arrives waits, before its next arrival, for the other one's, sent after that one's wait; the wait after the
//                        last tile is for an arrival that has no successor
//   q_full, l_full, pages, drain  one phase
// (The sums of f32 rows may not wait for p_full: its owner can arrive for tile j + 2 before the other warpgroup looks for tile j.)
struct PfBars {
    uint64_t *op_full, *op_empty, *info_full, *info_empty, *s_full, *p_full, *o_done, *o_free, *m_full, *drain, *l_full, *q_full, *pages;
    __device__ __forceinline__ explicit PfBars(uint64_t *b) {
        op_full = b, op_empty = op_full + kPfSlots, info_full = op_empty + kPfSlots, info_empty = info_full + kPfInfo;
        s_full = info_empty + kPfInfo, p_full = s_full + 2, o_done = p_full + 2, o_free = o_done + 2, m_full = o_free + 2, drain = m_full + 2;
        l_full = drain + 1, q_full = l_full + 1, pages = q_full + 1;
    }
    // info_readers: warps that read a tile's lookup
    __device__ __forceinline__ void init(int info_readers) {
        for (int i = 0; i < kPfSlots; ++i) mbar_init(op_full + i, 2), mbar_init(op_empty + i, 1);
        for (int i = 0; i < kPfInfo; ++i) mbar_init(info_full + i, 1), mbar_init(info_empty + i, info_readers);
        for (int i = 0; i < 2; ++i) mbar_init(s_full + i, 1), mbar_init(p_full + i, 4), mbar_init(o_done + i, 1), mbar_init(o_free + i, 8), mbar_init(m_full + i, 4);
        mbar_init(drain, 1);
        mbar_init(l_full, 8);
        mbar_init(q_full, 8);
        mbar_init(pages, 1);
        mbar_init_fence();
    }
};

// how a row tile of nj tiles of tokens is cut: `each` per piece, the last ones may have nothing
__device__ __forceinline__ int pf_each(int nj, int pieces) { return (nj + pieces - 1) / pieces; }

// the rows of a CTA and what they see; false if there are none
struct PfTile {
    int64_t lo, first, len;          // the sequence's first new token: its row, its position; the sequence's tokens
    int i0, g0;                      // row 0's new token and the head in the group
    int64_t base, b_lo, b_hi;        // first tile's first token; blocks that are read
    int64_t all_lo, all_hi;          // positions that every row sees
    int b, h, nrow, nj;
    int slot;                        // of the piece's partial; -1: the rows are done here
    bool bad;
    __device__ __forceinline__ int token(int r, int G) const { return i0 + (int)((uint32_t)(g0 + r) / (uint32_t)G); }
    __device__ __forceinline__ int head(int r, int G) const { return h * G + (int)((uint32_t)(g0 + r) % (uint32_t)G); }
    // the row tile `job`, or piece `piece` of it: KV head fastest, then the sequence, the latest (longest) row tiles first
    __device__ __forceinline__ bool init(const PfArgs &a, int per, uint32_t job, int piece, unsigned int *err) {
        const uint32_t of = job / a.c.H, up = of / a.c.n_seqs;
        h = (int)(job - of * a.c.H), b = (int)(of - up * a.c.n_seqs);
        const int tile = a.tiles - 1 - (int)up;
        int64_t hi;
        a.r.of(b, lo, hi);
        int64_t n = hi - lo;
        if (n > a.max_q) {
            if (threadIdx.x == 0 && err != nullptr) kv_error(err, KV_ERR_ROWS);
            n = a.max_q;
        }
        len = a.c.len[b], first = len - (hi - lo);
        const int G = a.group;
        const int64_t rows = n * G;
        const int64_t r0 = (int64_t)tile * per;
        if (r0 >= rows) return false;
        i0 = (int)(r0 / G), g0 = (int)(r0 - (int64_t)i0 * G);
        bad = len < 0 || (len > 0 && ((len - 1) >> a.c.tshift) >= a.c.max_pages);
        if (bad && threadIdx.x == 0 && err != nullptr) kv_error(err, KV_ERR_LEN);
        nrow = (int)min((int64_t)per, rows - r0);
        // the ends of what the rows see do not fall from row to row (rows that see nothing come first)
        int64_t t_lo = 0, t_hi = 0;
        all_lo = all_hi = 0;
        if (!bad) {
            int64_t x0, y0, x1, y1;
            row_range(first + token(0, G), len, a.causal, a.window, x0, y0);
            row_range(first + token(nrow - 1, G), len, a.causal, a.window, x1, y1);
            t_lo = x0, t_hi = max(y0, y1);
            if (y0 > x0) all_lo = x1, all_hi = y0;
        }
        b_lo = t_lo / kKB, b_hi = (t_hi + kKB - 1) / kKB;
        nj = (int)((b_hi - b_lo + 3) / 4);
        slot = -1;
        if (piece >= 0) {
            const int each = pf_each(nj, a.pieces), j0 = piece * each;
            if (piece > 0 && j0 >= nj) return false;
            if (each < nj) slot = 0;
            b_lo += 4 * (int64_t)j0;
            nj = min(each, nj - j0);
            b_hi = min(b_hi, b_lo + 4 * (int64_t)nj);
        }
        base = b_lo * kKB;
        return true;
    }
};

// a CTA's work: whole row tiles first, then the pieces of the others
__device__ __forceinline__ bool pf_work(PfTile &w, const PfArgs &a, int per, unsigned int *err) {
    const uint32_t whole = (uint32_t)(a.tiles * a.c.n_seqs * a.c.H - a.cut);
    const bool cut = blockIdx.x >= whole;
    const uint32_t v = blockIdx.x - whole, up = cut ? v / (uint32_t)a.pieces : 0;
    if (!w.init(a, per, cut ? whole + up : blockIdx.x, cut ? (int)(v - up * a.pieces) : -1, err)) return false;
    if (w.slot >= 0) w.slot = (int)v;
    return true;
}

// the bits of the largest magnitude, as f32 (an infinity's or more if there is one or a NaN)
template <int N>
__device__ __forceinline__ uint32_t pf_amax(const Raw4<float> (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float4 w = x[e].w;
        m = max(max(m, __float_as_uint(w.x) & 0x7fffffffu), max(__float_as_uint(w.y) & 0x7fffffffu, __float_as_uint(w.z) & 0x7fffffffu));
        m = max(m, __float_as_uint(w.w) & 0x7fffffffu);
    }
    return m;
}
template <typename T, int N>
__device__ __forceinline__ uint32_t pf_amax(const Raw4<T> (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) m = __vmaxu2(m, __vmaxu2(x[e].w.x & 0x7fff7fffu, x[e].w.y & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    return m << 16;
}

// q of the rows as f16 parts in the K-major swizzled layout, by warps 0-7: 16 bytes a lane, eight loads in flight; rows that are not
// there are zeros
template <typename T, int D>
__device__ __forceinline__ void pf_stage_q(const PfArgs &a, const PfTile &w, uint8_t *sm, float *s_rs, int count) {
    constexpr bool TWO = sizeof(T) == 4;
    using C = PfCfg<D, TWO>;
    constexpr int N = TWO ? 1 : 2, LPR = D / (4 * N), RPW = 32 / LPR, FLY = 8;       // fours of elements per lane, lanes per row, rows per load
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.group, col = (lane % LPR) * 4 * N;
#pragma unroll 1
    for (int r0 = warp * RPW + lane / LPR; r0 < count; r0 += 8 * RPW * FLY) {
        Raw4<T> x[FLY][N];
#pragma unroll
        for (int z = 0; z < FLY; ++z) {
            const int r = r0 + 8 * RPW * z;
#pragma unroll
            for (int e = 0; e < N; ++e) x[z][e] = Raw4<T>{};
            if (r < w.nrow) {
                const T *p = static_cast<const T *>(a.q) + (w.lo + w.token(r, G)) * a.qt + (int64_t)w.head(r, G) * a.qh + col;
#pragma unroll
                for (int e = 0; e < N; ++e) x[z][e] = *reinterpret_cast<const Raw4<T> *>(p + 4 * e);
            }
        }
#pragma unroll
        for (int z = 0; z < FLY; ++z) {
            const int r = r0 + 8 * RPW * z;
            uint32_t amax = pf_amax(x[z]);
            if constexpr (LPR == 32) {
                amax = __reduce_max_sync(0xffffffffu, amax);
            } else {
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            }
            const bool fin = amax < 0x7f800000u;
            const int ex = fin ? row_exponent(__uint_as_float(amax)) : 0;
            const float down = fin ? pow2i(-ex) * a.sign : __int_as_float(0x7fc00000);   // a row with a NaN or an infinity becomes NaN
            uint32_t hi[2 * N], lo[2 * N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float y[4];
                unpack4(x[z][e], y);
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float y0 = fin ? y[k] * down : down, y1 = fin ? y[k + 1] * down : down;
                    hi[2 * e + (k >> 1)] = pack_f16(y0, y1);
                    const float2 f = unpack_f16(hi[2 * e + (k >> 1)]);
                    lo[2 * e + (k >> 1)] = pack_f16(y0 - f.x, y1 - f.y);
                }
            }
            // 16-byte unit (col / 8) % 8 of row r % 128 in the 64-column half col / 64
            uint8_t *dst = sm + C::OFF_Q + (r >> 7) * C::QT + (col >> 6) * 16384 + (r & 127) * 128 + ((((col >> 3) & 7) ^ (r & 7)) << 4) + (col & 7) * 2;
            if (r < count) {
                if constexpr (TWO) {
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2 *>(dst + C::TILES * C::QT) = make_uint2(lo[0], lo[1]);
                } else {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                }
                if (lane % LPR == 0) s_rs[r] = pow2i(ex) * a.c_log2;
            }
        }
    }
}
// ... then the tensor core and the other softmax warps have it
__device__ __forceinline__ void pf_q_staged(const PfBars &bar, int lane) {
    fence_proxy_async_smem();
    warp_arrive(bar.q_full, lane);
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

// warp 14: whether every page that rows of the CTA's sequence read is there.  If one is not, all of the sequence's rows are zeros, those
// too that do not see it: every CTA looks at all of them (a pool of pages of 32 tokens: 4 bytes for the 8 KB that a head of 128 reads).
__device__ __forceinline__ void pf_check_pages(const PfArgs &a, const PfTile &w, const PfBars &bar, unsigned int *err, volatile int *lost) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if (!w.bad) {
        int64_t lo, hi, x0, y0, x1, y1;
        a.r.of(w.b, lo, hi);
        row_range(w.first, w.len, a.causal, a.window, x0, y0);
        row_range(w.first + min(hi - lo, a.max_q) - 1, w.len, a.causal, a.window, x1, y1);
        const int32_t *table = a.c.table + (int64_t)w.b * a.c.max_pages;
        const int64_t end = (max(y0, y1) + a.c.T - 1) >> a.c.tshift;
#pragma unroll 4
        for (int64_t p = (x0 >> a.c.tshift) + lane; p < end; p += 32) {
            const int page = table[p];
            bad = bad || page < 0 || page >= a.c.n_pages;
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) {
        kv_error(err, KV_ERR_PAGE);
        *lost = 1;
    }
    warp_arrive(bar.pages, lane);
}

// warp 12: pages and scales of the tiles, 32 blocks at a time, one a lane
__device__ __forceinline__ void pf_lookup(const PfArgs &a, const PfTile &w, PfInfo *info, const PfBars &bar, unsigned int *err, volatile int *abort) {
    const int lane = threadIdx.x & 31;
    int pg = -1, pg_n = -1;
    float dk = 0.0f, dv = 0.0f, dk_n = 0.0f, dv_n = 0.0f;
    auto fetch = [&](int64_t blk) {                            // into the next batch
        pg_n = -1, dk_n = dv_n = 0.0f;
        if (blk < w.b_hi) {
            pg_n = a.c.table[(int64_t)w.b * a.c.max_pages + ((blk * kKB) >> a.c.tshift)];
            if (pg_n < 0 || pg_n >= a.c.n_pages) {
                kv_error(err, KV_ERR_PAGE);
                pg_n = -1;
            } else {
                const float *sc = reinterpret_cast<const float *>(a.c.pool + pg_n * a.c.page_bytes + a.c.off_s);
                const int sb = (int)((blk * kKB) & (a.c.T - 1)) / kKB, spp = a.c.T / kKB;
                dk_n = sc[w.h * spp + sb];
                dv_n = sc[(a.c.H + w.h) * spp + sb];
            }
        }
    };
    fetch(w.b_lo + lane);
    for (int j = 0; j < w.nj; ++j) {
        if ((j & 7) == 0) {
            pg = pg_n, dk = dk_n, dv = dv_n;
            fetch(w.b_lo + 4 * (int64_t)(j + 8) + lane);
        }
        const int e = lane - 4 * (j & 7);
        if (j >= kPfInfo && !warp_wait(bar.info_empty + j % kPfInfo, (j / kPfInfo - 1) & 1, err, abort)) break;
        PfInfo &o = info[j % kPfInfo];
        if (e >= 0 && e < 4) {
            o.dk[e] = dk;
            o.dv[e] = dv;
            o.lv[e] = log2_approx(dv);
            o.page[e] = pg;
        }
        __threadfence_block();
        warp_arrive(bar.info_full + j % kPfInfo, lane);
    }
}

// Place of an operand tile in the ring's order K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1)
__device__ __forceinline__ int pf_order(int j, int half, int nj) { return half ? (j == nj - 1 ? 2 * nj - 1 : 2 * j + 2) : (j == 0 ? 0 : 2 * j - 1); }

// warps 8-11: codes widened into the operand ring, two warps for K, two for V, two blocks of 32 tokens each per tile.  A lane turns 8
// bytes into one 16-byte unit, eight lanes the eight units of a 128-byte line; the next tile's bytes are in flight meanwhile.
template <int D, bool TWO>
__device__ __forceinline__ void pf_widen(const PfArgs &a, const PfTile &w, uint8_t *ops, const PfInfo *info, const PfBars &bar, unsigned int *err,
                                         volatile int *abort) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, IT = kKB / RPI, NV = 8 / RPI, OPT = PfCfg<D, TWO>::OPT, SLOTS = PfCfg<D, TWO>::SLOTS;   // lanes per row, rows per load, loads
    const int wi = (threadIdx.x >> 5) - 8, lane = threadIdx.x & 31, half = wi >> 1, blk0 = 2 * (wi & 1), u = lane % LPR;
    uint32_t off[NV];                                          // this lane's unit in rows 0 .. 7 of its first block
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int row = v * RPI + lane / LPR;
        off[v] = smem_u32(ops) + (u >> 3) * 16384 + (32 * blk0 + row) * 128 + (((u & 7) ^ row) << 4);
    }
    const int64_t in0 = (half ? a.c.off_v : 0) + (int64_t)w.h * a.c.T * D + lane * 8;
    const int tmask = a.c.T - 1, tok0 = (int)((w.base + 32 * blk0) & tmask);
    uint2 raw[2][IT];
    const uint8_t *src[2];
    auto locate = [&](int j) -> bool {
        if (!warp_wait(bar.info_full + j % kPfInfo, (j / kPfInfo) & 1, err, abort)) return false;
        const PfInfo &o = info[j % kPfInfo];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int page = o.page[blk0 + z];
            src[z] = page >= 0 ? a.c.pool + page * a.c.page_bytes + in0 + ((tok0 + (4 * j + z) * kKB) & tmask) * D : nullptr;
        }
        warp_arrive(bar.info_empty + j % kPfInfo, lane);
        return true;
    };
    auto load = [&](int z, int k) { return src[z] != nullptr ? __ldg(reinterpret_cast<const uint2 *>(src[z] + k * 256)) : make_uint2(0x80808080u, 0x80808080u); };
    if (w.nj == 0 || !locate(0)) return;
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int k = 0; k < IT; ++k) raw[z][k] = load(z, k);
    for (int j = 0; j < w.nj; ++j) {
        const bool more = j + 1 < w.nj;
        if (more) {
            if (!locate(j + 1)) break;
        }
        const int n = pf_order(j, half, w.nj), slot = n % SLOTS;
        if (n >= SLOTS && !warp_wait(bar.op_empty + slot, (n / SLOTS - 1) & 1, err, abort)) break;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                uint4 x;
                codes_f16(raw[z][k].x, x.x, x.y);
                codes_f16(raw[z][k].y, x.z, x.w);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(off[k % NV] + slot * OPT + z * 4096 + (k / NV) * 1024), "r"(x.x),
                             "r"(x.y), "r"(x.z), "r"(x.w)
                             : "memory");
            }
        }
        fence_proxy_async_smem();
        warp_arrive(bar.op_full + slot, lane);
        // all loads at once: issued one by one between the conversions, each conversion waited for the loads just issued
        if (more) {
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int k = 0; k < IT; ++k) raw[z][k] = load(z, k);
        }
    }
}

// MMAs of one tile: scores (A = q from shared memory) and outputs (A = the weights from TMEM).  Descriptors are made once; a
// step adds to their address fields (16-byte units).
template <int D, bool TWO>
struct PfMma {
    using C = PfCfg<D, TWO>;
    static constexpr uint32_t ID_S = idesc_f16_f32(128, kPfN), ID_O = idesc_f16_f32(128, D) | (1u << 16);     // B of O is MN-major
    static constexpr uint32_t HI = (1024 >> 4) | (1u << 14) | (2u << 29);        // the upper words of both descriptors: stride, version, swizzle
    uint32_t dq, dk, dv;                                       // the lower words: address and leading stride
    __device__ __forceinline__ explicit PfMma(uint8_t *sm) {
        dq = (uint32_t)sw128_kmajor_desc(smem_u32(sm + C::OFF_Q)), dk = (uint32_t)sw128_kmajor_desc(smem_u32(sm + C::OFF_OP));
        dv = (uint32_t)sw128_mnmajor_desc(smem_u32(sm + C::OFF_OP), 16384);
    }
    static __device__ __forceinline__ uint64_t desc(uint32_t lo) {
        uint64_t d;
        asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "n"(HI));
        return d;
    }
    __device__ __forceinline__ void scores(uint32_t d, int t, uint32_t slot) const {
        const uint32_t q = dq + t * (C::QT >> 4), k = dk + slot * (C::OPT >> 4);
        uint32_t acc = 0;
#pragma unroll 1
        for (int i = 0; i < C::PARTS * (D / 64); ++i) {        // 64 columns of one part; the smaller part first
            const uint32_t part = i < D / 64 ? C::PARTS - 1 : 0, hc = i & (D / 64 - 1);
            const uint32_t qi = q + part * C::TILES * (C::QT >> 4) + hc * 1024, ki = k + hc * 1024;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mma_f16_warp(d, desc(qi + 2 * e), desc(ki + 2 * e), ID_S, acc);
                acc = 1;
            }
        }
    }
    __device__ __forceinline__ void output(uint32_t d, uint32_t p, uint32_t slot, uint32_t more) const {
        const uint32_t v = dv + slot * (C::OPT >> 4);
#pragma unroll 1
        for (int i = 0; i < 2 * C::PARTS; ++i) {               // 64 tokens of one part; the smaller part first
            const uint32_t part = i < 2 ? C::PARTS - 1 : 0, ht = i & 1;
            const uint32_t pi = p + (TWO ? ht * 64 + part * 16 : ht * 32), vi = v + ht * 512;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mma_f16_ts_warp(d, pi + (TWO ? 32 * (e >> 1) + 8 * (e & 1) : 8 * e), desc(vi + 128 * e), ID_O, more);
                more = 1;
            }
        }
    }
};

// minus infinity over the row's scores outside positions x0 <= k < x1 (tiles that are not seen whole)
__device__ __forceinline__ void pf_mask(uint32_t ts, int x0, int x1) {
#pragma unroll 1
    for (int e = 0; e < kPfN; e += 16) {
        uint32_t s[16];
        tmem_ld16(ts + e, s, 0);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (e + k < x0 || e + k >= x1) s[k] = 0xff800000u;
        tmem_st16(ts + e, s);
    }
    tmem_st_wait();
}
// 64 scores of the row as they lie in TMEM
__device__ __forceinline__ void pf_load_scores(uint32_t ts, uint32_t (&s)[2][32]) {
    tmem_ld32(ts, s[0]);
    tmem_ld32(ts + 32, s[1]);
    tmem_ld_wait();
}
__device__ __forceinline__ float pf_max32(const uint32_t (&s)[32]) {
    float y[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        y[z] = max3(__uint_as_float(s[8 * z]), __uint_as_float(s[8 * z + 1]), __uint_as_float(s[8 * z + 2]));
        y[z] = max3(y[z], __uint_as_float(s[8 * z + 3]), __uint_as_float(s[8 * z + 4]));
        y[z] = max3(y[z], __uint_as_float(s[8 * z + 5]), __uint_as_float(s[8 * z + 6]));
        y[z] = fmaxf(y[z], __uint_as_float(s[8 * z + 7]));
    }
    return fmaxf(max3(y[0], y[1], y[2]), y[3]);
}

// the largest of 32 consecutive columns of the lane's row, found by the load itself (the values are not used)
__device__ __forceinline__ float pf_load_max32(uint32_t taddr) {
    uint32_t s[32];
    float m;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
        : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7]), "=r"(s[8]), "=r"(s[9]), "=r"(s[10]),
          "=r"(s[11]), "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15]), "=r"(s[16]), "=r"(s[17]), "=r"(s[18]), "=r"(s[19]), "=r"(s[20]),
          "=r"(s[21]), "=r"(s[22]), "=r"(s[23]), "=r"(s[24]), "=r"(s[25]), "=r"(s[26]), "=r"(s[27]), "=r"(s[28]), "=r"(s[29]), "=r"(s[30]),
          "=r"(s[31]), "=f"(m)
        : "r"(taddr)
        : "memory");
    return m;
}
// The softmax reads a tile's scores twice from TMEM: once for the maximum, once, 64 or 32 at a time, for the weights.  Holding all 128
// in registers left the compiler none to overlap the elements' chains with (3600 clocks a tile for f32 rows).
// ... and `top`: the largest of a block's maximum times its V scale (binary logarithms)
__device__ __forceinline__ float pf_tile_max(uint32_t ts, const float (&kb)[4], const float4 &lv, float &top) {
    float mx = -INFINITY;
    top = -INFINITY;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        float m0 = pf_load_max32(ts + 64 * e), m1 = pf_load_max32(ts + 64 * e + 32);
        tmem_ld_wait();
        m0 *= e ? kb[2] : kb[0], m1 *= e ? kb[3] : kb[1];
        mx = max3(mx, m0, m1);
        top = max3(top, m0 + (e ? lv.z : lv.x), m1 + (e ? lv.w : lv.y));
    }
    return mx;
}
// the weights of 32 scores: 2^(s kb + off) summed into l2 and, times pv (f32 rows), packed to f16: leading parts w, the rest v
template <bool TWO>
__device__ __forceinline__ void pf_weights(const uint32_t (&s)[32], float kb, uint64_t off2, float pv, uint64_t &l2, uint32_t (&w)[16],
                                           uint32_t (&v)[16]) {
    const uint64_t kk = f2_pack(kb, kb), pp = f2_pack(pv, pv);
    uint64_t acc[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        float x, y;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), kk, off2), x, y);
        x = exp2_approx(x), y = exp2_approx(y);
        const uint64_t p = f2_pack(x, y);
        acc[(k >> 1) & 1] = f2_add(acc[(k >> 1) & 1], p);
        f2_unpack(f2_mul(p, pp), x, y);
        if constexpr (TWO) {
            w[k >> 1] = pack_f16(x, y);
            const float2 z = unpack_f16(w[k >> 1]);
            f2_unpack(f2_fma(f2_pack(z.x, z.y), f2_pack(-1.0f, -1.0f), f2_pack(x, y)), x, y);
            v[k >> 1] = pack_f16(x, y);
        } else {
            w[k >> 1] = pack_f16(x, y);
        }
    }
    l2 = f2_add(l2, f2_add(acc[0], acc[1]));
}
// the weights of the tile, written over the scores that have been read.  16-bit rows: 32 columns per 64 scores, from the front
__device__ __forceinline__ void pf_tile_weights(uint32_t ts, const float (&kb)[4], const float (&pb)[4], float off, uint64_t &l2) {
    const uint64_t off2 = f2_pack(off, off);
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        uint32_t s[2][32], w[16], v[16];
        pf_load_scores(ts + 64 * e, s);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            pf_weights<false>(s[z], e ? kb[2 + z] : kb[z], off2, e ? pb[2 + z] : pb[z], l2, w, v);
            tmem_st16(ts + 32 * e + 16 * z, w);
        }
    }
}
// f32 rows, a block of 32 tokens at a time: its 16 columns of leading parts and 16 of the rest in the scores' place
__device__ __forceinline__ float pf_score_factor(float rs, float dk) { return fmaxf(rs * dk, 0x1p-120f); }
__device__ __forceinline__ float pf_tile_max_f32(uint32_t ts, float rs, const PfInfo &o, float &top) {
    float mx = -INFINITY;
    top = -INFINITY;
#pragma unroll 1
    for (int e = 0; e < 4; e += 2) {
        uint32_t s[2][32];
        pf_load_scores(ts + 32 * e, s);
        const float m0 = pf_max32(s[0]) * pf_score_factor(rs, o.dk[e]), m1 = pf_max32(s[1]) * pf_score_factor(rs, o.dk[e + 1]);
        mx = max3(mx, m0, m1);
        top = max3(top, m0 + o.lv[e], m1 + o.lv[e + 1]);
    }
    return mx;
}
__device__ __forceinline__ void pf_tile_weights_f32(uint32_t ts, float rs, const PfInfo &o, float off, float m_over_a, uint64_t &l2) {
    const uint64_t off2 = f2_pack(off, off);
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
        uint32_t s[32], w[16], v[16];
        tmem_ld32(ts + 32 * e, s);
        const float kb = pf_score_factor(rs, o.dk[e]), pv = v_factor(o.dv[e], m_over_a);
        tmem_ld_wait();
        pf_weights<true>(s, kb, off2, pv, l2, w, v);
        tmem_st16(ts + 32 * e, w);
        tmem_st16(ts + 32 * e + 16, v);
    }
}

#define PF_PROLOGUE(T, D, INFO_READERS)                                                                                       \
    using C = PfCfg<D, sizeof(T) == 4>;                                                                                       \
    extern __shared__ uint8_t smem_raw[];                                                                                     \
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));             \
    float *s_rs = reinterpret_cast<float *>(sm + C::OFF_RS);                                                                  \
    PfInfo *info = reinterpret_cast<PfInfo *>(sm + C::OFF_INFO);                                                              \
    const PfBars bar(reinterpret_cast<uint64_t *>(sm + C::OFF_BAR));                                                          \
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(sm + C::OFF_MISC);                                                   \
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 4);                                        \
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;                                                               \
    grid_dep_launch();                                                                                                        \
    grid_dep_wait();                                                                                                          \
    PfTile w;                                                                                                                 \
    if (!pf_work(w, a, C::ROWS, err)) return;                                                                                 \
    const int nt = w.nrow > 128 ? 2 : 1, nj = w.nj;                                                                           \
    if (threadIdx.x == 0) {                                                                                                   \
        *abort_flag = 0;                                                                                                      \
        abort_flag[1] = w.slot;                                                                                               \
        abort_flag[2] = 0;                                                                                                    \
        const_cast<PfBars &>(bar).init(INFO_READERS);                                                                         \
    }                                                                                                                         \
    if (warp == 13) tmem_alloc(tmem_holder, 512);                                                                             \
    tc_fence_before();                                                                                                        \
    __syncthreads();                                                                                                          \
    tc_fence_after();                                                                                                         \
    const uint32_t tmem = *tmem_holder

// 16-bit rows: two row tiles per CTA
template <typename T, int D>
__global__ void __launch_bounds__(kPfThreads, 1) kv_tiles_kernel(PfArgs a, unsigned int *err) {
    PF_PROLOGUE(T, D, 4 * nt + 4);
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == 12) {
            pf_lookup(a, w, info, bar, err, abort_flag);
        } else if (warp == 13) {
            const PfMma<D, false> mma(sm);
            const uint32_t s0 = tmem + C::COL_S, o0 = tmem + C::COL_O;
            uint32_t slot = 0, ph = 0;
            auto next = [&]() {
                if (++slot == C::SLOTS) slot = 0, ph ^= 1;
            };
            bool ok = nj > 0 && warp_wait2(bar.q_full, bar.op_full, 0, err, abort_flag);
            if (ok) {
                tc_fence_after();
                mma.scores(s0, 0, 0);
                mma_commit_warp(bar.s_full);
                if (nt == 2) {
                    mma.scores(s0 + 128, 1, 0);
                    mma_commit_warp(bar.s_full + 1);
                }
                mma_commit_warp(bar.op_empty);
                next();
            }
            for (int j = 0; ok && j < nj; ++j) {
                const bool more = j + 1 < nj;
                const uint32_t sk = slot, pk = ph;
                if (more) next();
                const uint32_t sv = slot, pv = ph;
                next();
                if (!(ok = warp_wait3(bar.op_full + sk, bar.op_full + sv, bar.p_full, pk, pv, j & 1, err, abort_flag))) break;
                tc_fence_after();
                mma.output(o0, s0, sv, j > 0);
                mma_commit_warp(bar.o_done);
                if (more) {
                    mma.scores(s0, 0, sk);
                    mma_commit_warp(bar.s_full);
                }
                if (nt == 2) {
                    if (!(ok = warp_wait(bar.p_full + 1, j & 1, err, abort_flag))) break;
                    tc_fence_after();
                    mma.output(o0 + D, s0 + 128, sv, j > 0);
                    mma_commit_warp(bar.o_done + 1);
                    mma_commit_warp(bar.op_empty + sv);
                    if (more) {
                        mma.scores(s0 + 128, 1, sk);
                        mma_commit_warp(bar.s_full + 1);
                    }
                } else {
                    mma_commit_warp(bar.op_empty + sv);
                }
                if (more) mma_commit_warp(bar.op_empty + sk);
            }
            // products and arrivals in flight end before the TMEM and the barriers go
            mma_commit_warp(bar.drain);
            mbar_wait(bar.drain, 0, err, KV_ERR_WAIT, nullptr);
        } else if (warp == 14) {
            pf_check_pages(a, w, bar, err, abort_flag + 2);
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        pf_widen<D, false>(a, w, sm + C::OFF_OP, info, bar, err, abort_flag);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        pf_stage_q<T, D>(a, w, sm, s_rs, nt * 128);
        pf_q_staged(bar, lane);
        const int t = warp >> 2, r = threadIdx.x;
        if (t < nt) {
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t ts = tmem + C::COL_S + t * 128 + lanes, to = tmem + C::COL_O + t * D + lanes;
            int v0 = 0, v1 = 0;                                 // what the row sees, from the first tile's start
            if (r < w.nrow && !w.bad) {
                int64_t x, y;
                row_range(w.first + w.token(r, a.group), w.len, a.causal, a.window, x, y);
                v0 = (int)max(x - w.base, (int64_t)0), v1 = (int)max(y - w.base, (int64_t)0);
            }
            const int i_lo = (int)max(w.all_lo - w.base, (int64_t)INT_MIN), i_hi = (int)max(w.all_hi - w.base, (int64_t)INT_MIN);
            const float rs = s_rs[r];
            float m = -INFINITY, ra = -INFINITY;                // the references m and A
            uint64_t l2 = f2_pack(0.0f, 0.0f);
            bool ok = true;
            for (int j = 0; j < nj; ++j) {
                if (!(ok = warp_wait(bar.info_full + j % kPfInfo, (j / kPfInfo) & 1, err, abort_flag))) break;      // under the products
                const PfInfo &o = info[j % kPfInfo];
                const float4 dk = *reinterpret_cast<const float4 *>(o.dk), dv = *reinterpret_cast<const float4 *>(o.dv),
                             lv = *reinterpret_cast<const float4 *>(o.lv);
                // at least 2^-120, so that a masked score stays minus infinity under a scale of zero
                const float kb[4] = {fmaxf(rs * dk.x, 0x1p-120f), fmaxf(rs * dk.y, 0x1p-120f), fmaxf(rs * dk.z, 0x1p-120f), fmaxf(rs * dk.w, 0x1p-120f)};
                warp_arrive(bar.info_empty + j % kPfInfo, lane);
                if (!(ok = warp_wait(bar.s_full + t, j & 1, err, abort_flag))) break;
                tc_fence_after();
                const int t0 = j * kPfN;
                if (!(t0 >= i_lo && t0 + kPfN <= i_hi)) pf_mask(ts, v0 - t0, v1 - t0);
                float top;
                const float mx = pf_tile_max(ts, kb, lv, top);
                if (__any_sync(0xffffffffu, mx > m + kTau || top > ra + kTau || (m == -INFINITY && mx > m))) {
                    const float mn = fmaxf(m, mx), ref = max3(ra, top, mn - kRefSpan);
                    const float f = mn == -INFINITY ? 1.0f : exp2_approx(m - mn), fo = ref == -INFINITY ? 1.0f : exp2_approx(ra - ref);
                    m = mn, ra = ref;
                    l2 = f2_mul(l2, f2_pack(f, f));
                    if (j > 0 && __any_sync(0xffffffffu, fo != 1.0f)) {
                        if (!(ok = warp_wait(bar.o_done + t, (j - 1) & 1, err, abort_flag))) break;
                        tc_fence_after();
                        const uint64_t ff = f2_pack(fo, fo);
#pragma unroll 1
                        for (int e = 0; e < D / 16; ++e) {
                            uint32_t x[16];
                            tmem_ld16(to + 16 * e, x, 0);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                float y, z;
                                f2_unpack(f2_mul(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), ff), y, z);
                                x[k] = __float_as_uint(y), x[k + 1] = __float_as_uint(z);
                            }
                            tmem_st16(to + 16 * e, x);
                        }
                    }
                }
                const float over = ref_factor(m, ra);
                const float pb[4] = {v_factor(dv.x, over), v_factor(dv.y, over), v_factor(dv.z, over), v_factor(dv.w, over)};
                pf_tile_weights(ts, kb, pb, kLazyShift - (m == -INFINITY ? 0.0f : m), l2);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(bar.p_full + t, lane);
            }
            // ---------------------------------------------------------------- the rows' outputs
            if (nj > 0 && ok) ok = warp_wait(bar.o_done + t, (nj - 1) & 1, err, abort_flag);
            warp_wait(bar.pages, 0, err, abort_flag);
            tc_fence_after();
            float l, l1;
            f2_unpack(l2, l, l1);
            l += l1;
            const int piece = abort_flag[1];
            const bool lost = abort_flag[2] != 0;              // zeros leave, with a sum of weights below zero for the join
            if (lost) l = piece >= 0 ? -1.0f : 0.0f;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l * ref_factor(ra, m);
            float *pd = a.part + ((int64_t)piece * C::ROWS + r) * (D + 4);
            if (piece >= 0 && r < w.nrow) *reinterpret_cast<float2 *>(pd + D) = make_float2(m, l);
            T *dst = static_cast<T *>(a.out) + (w.lo + w.token(r, a.group)) * a.ot + (int64_t)w.head(r, a.group) * a.oh;
#pragma unroll 1
            for (int e = 0; e < D / 32; ++e) {
                uint32_t x[32];
                if (nj > 0) {
                    tmem_ld32(to + 32 * e, x);
                    tmem_ld_wait();
                }
                if (r < w.nrow) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float y[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) y[z] = nj > 0 && l != 0.0f && !lost ? __uint_as_float(x[k + z]) * inv : 0.0f;
                        if (piece >= 0) store4(pd + 32 * e + k, y);
                        else store4(dst + 32 * e + k, y);
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

// f32 rows: one row tile per CTA, every tile's P V summed in registers.  The MMAs (2048 clocks per 128 tokens) leave one softmax
// warpgroup no time (it took 4250, with a second one for the sums: 204 us for the 3314-token prompt), so two share the work.
template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) kv_tiles_f32_kernel(PfArgs a, unsigned int *err) {
    PF_PROLOGUE(float, D, 4 + 4);
    float *s_f = s_rs + 128, *s_a = s_f + 512;                 // [4 tiles][128] factors of what was summed before, references A
    float *s_l = s_a + 512;                                    // [warpgroup][2][128] maxima and sums of weights
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 12) {
            pf_lookup(a, w, info, bar, err, abort_flag);
        } else if (warp == 13) {
            const PfMma<D, true> mma(sm);
            const uint32_t s0 = tmem + C::COL_S, o0 = tmem + C::COL_O;
            uint32_t slot = 0, ph = 0;
            auto next = [&]() {
                if (++slot == C::SLOTS) slot = 0, ph ^= 1;
            };
            bool ok = nj > 0 && warp_wait2(bar.q_full, bar.op_full, 0, err, abort_flag);
            if (ok) {
                tc_fence_after();
                mma.scores(s0, 0, 0);
                mma_commit_warp(bar.s_full);
                mma_commit_warp(bar.op_empty);
                next();
            }
            for (int j = 0; ok && j < nj; ++j) {
                const uint32_t at = j & 1, nx = at ^ 1;
                if (j + 1 < nj) {                              // P(j - 1) in this buffer was read by products issued before
                    if (!(ok = warp_wait(bar.op_full + slot, ph, err, abort_flag))) break;
                    tc_fence_after();
                    mma.scores(s0 + nx * 128, 0, slot);
                    mma_commit_warp(bar.s_full + nx);
                    mma_commit_warp(bar.op_empty + slot);
                    next();
                }
                if (!(ok = warp_wait(bar.op_full + slot, ph, err, abort_flag))) break;
                if (j >= 2 && !(ok = warp_wait(bar.o_free + at, ((j >> 1) - 1) & 1, err, abort_flag))) break;
                if (!(ok = warp_wait(bar.p_full + at, (j >> 1) & 1, err, abort_flag))) break;
                tc_fence_after();
                mma.output(o0 + at * D, s0 + at * 128, slot, 0);
                mma_commit_warp(bar.o_done + at);
                mma_commit_warp(bar.op_empty + slot);
                next();
            }
            // products and arrivals in flight end before the TMEM and the barriers go
            mma_commit_warp(bar.drain);
            mbar_wait(bar.drain, 0, err, KV_ERR_WAIT, nullptr);
        } else if (warp == 14) {
            pf_check_pages(a, w, bar, err, abort_flag + 2);
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        pf_widen<D, true>(a, w, sm + C::OFF_OP, info, bar, err, abort_flag);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        pf_stage_q<float, D>(a, w, sm, s_rs, 128);
        pf_q_staged(bar, lane);
        // Two warpgroups take the tiles' softmax in turn, and each sums half of the columns of every tile's P V.
        const int a2 = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, ts = tmem + C::COL_S + lanes, to = tmem + C::COL_O + a2 * (D / 2) + lanes;
        int v0 = 0, v1 = 0;                                    // what the row sees, from the first tile's start
        if (r < w.nrow && !w.bad) {
            int64_t x, y;
            row_range(w.first + w.token(r, a.group), w.len, a.causal, a.window, x, y);
            v0 = (int)max(x - w.base, (int64_t)0), v1 = (int)max(y - w.base, (int64_t)0);
        }
        const int i_lo = (int)max(w.all_lo - w.base, (int64_t)INT_MIN), i_hi = (int)max(w.all_hi - w.base, (int64_t)INT_MIN);
        const float rs = s_rs[r];
        float m = -INFINITY;                                   // the maximum of this warpgroup's tiles: its sum's reference
        uint64_t l2 = f2_pack(0.0f, 0.0f);
        uint64_t acc[D / 4];
#pragma unroll
        for (int k = 0; k < D / 4; ++k) acc[k] = f2_pack(0.0f, 0.0f);
        for (int j = 0; j < nj + 2; ++j) {
            const int at = j & 1;
            if (j >= 2) {                                      // half of tile j - 2's products
                const uint32_t ph = ((j >> 1) - 1) & 1;
                // the products, and after the last tile of the other warpgroup its factors: those of its earlier tiles came with the maxima
                // that this one waited for in its own tile j - 1
                if (!warp_wait(bar.o_done + at, ph, err, abort_flag)) break;
                if (j == nj + 1 && at != a2 && !warp_wait(bar.m_full + at, ph, err, abort_flag)) break;
                const float f = s_f[((j - 2) & 3) * 128 + r];
                const uint64_t ff = f2_pack(f, f);
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    uint32_t x[32];
                    tmem_ld32(to + at * D + 32 * e, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; k += 2)
                        acc[16 * e + (k >> 1)] = f2_fma(acc[16 * e + (k >> 1)], ff, f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
                }
                tc_fence_before();
                warp_arrive(bar.o_free + at, lane);
            }
            if (j >= nj || at != a2) continue;
            if (!warp_wait2(bar.info_full + j % kPfInfo, bar.s_full + at, (j / kPfInfo) & 1, (j >> 1) & 1, err, abort_flag)) break;
            tc_fence_after();
            const PfInfo &o = info[j % kPfInfo];
            const int t0 = j * kPfN;
            if (!(t0 >= i_lo && t0 + kPfN <= i_hi)) pf_mask(ts + at * 128, v0 - t0, v1 - t0);
            float top;
            const float mx = pf_tile_max_f32(ts + at * 128, rs, o, top);
            float before = -INFINITY;                          // A after tile j - 1, from the other warpgroup
            if (j > 0) {
                if (!warp_wait(bar.m_full + (at ^ 1), ((j - 1) >> 1) & 1, err, abort_flag)) break;
                before = s_a[((j - 1) & 3) * 128 + r];
            }
            const float mn = fmaxf(m, mx), mb = mn == -INFINITY ? 0.0f : mn, ref = max3(before, top, mn - kRefSpan);
            // their places: the other warpgroup has published tile j - 1's, so it has summed tile j - 4 and is done with these
            s_a[(j & 3) * 128 + r] = ref;
            s_f[(j & 3) * 128 + r] = ref_factor(before, ref);
            warp_arrive(bar.m_full + at, lane);
            const float f = exp2_approx(m - mb);
            m = mn;
            l2 = f2_mul(l2, f2_pack(f, f));
            pf_tile_weights_f32(ts + at * 128, rs, o, kPShift - mb, ref_factor(mn, ref), l2);
            warp_arrive(bar.info_empty + j % kPfInfo, lane);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(bar.p_full + at, lane);
        }
        // the sum of both warpgroups' weights, relative to the larger maximum; the last tile's A is what the outputs are relative to
        float l, l1;
        f2_unpack(l2, l, l1);
        s_l[a2 * 256 + r] = m, s_l[a2 * 256 + 128 + r] = l + l1;
        warp_arrive(bar.l_full, lane);
        warp_wait(bar.l_full, 0, err, abort_flag);
        warp_wait(bar.pages, 0, err, abort_flag);
        const float m0 = s_l[r], m1 = s_l[256 + r], mm = fmaxf(m0, m1), mb = mm == -INFINITY ? 0.0f : mm;
        l = s_l[128 + r] * exp2_approx(m0 - mb) + s_l[384 + r] * exp2_approx(m1 - mb);
        const int piece = abort_flag[1];
        const bool lost = abort_flag[2] != 0;                  // zeros leave, with a sum of weights below zero for the join
        if (lost) l = piece >= 0 ? -1.0f : 0.0f;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l * (nj > 0 ? ref_factor(s_a[((nj - 1) & 3) * 128 + r], mm) : 0.0f);
        if (r < w.nrow) {
            float *dst = static_cast<float *>(a.out) + (w.lo + w.token(r, a.group)) * a.ot + (int64_t)w.head(r, a.group) * a.oh + a2 * (D / 2);
            if (piece >= 0) {
                float *pd = a.part + ((int64_t)piece * C::ROWS + r) * (D + 4);
                if (a2 == 0) *reinterpret_cast<float2 *>(pd + D) = make_float2(mm, l);
                dst = pd + a2 * (D / 2);
            }
#pragma unroll
            for (int k = 0; k < D / 2; k += 4) {
                float y[4];
                f2_unpack(acc[k / 2], y[0], y[1]);
                f2_unpack(acc[k / 2 + 1], y[2], y[3]);
#pragma unroll
                for (int z = 0; z < 4; ++z) y[z] = lost ? 0.0f : y[z] * inv;
                store4(dst + k, y);
            }
        }
    }
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the pieces of the row tiles that were cut: a CTA per row tile and 8 rows, a warp per row.  Lane p has piece p's maximum and sum.
constexpr int kPfMostPieces = 32, kPfJoinRows = 8;
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_tiles_join_kernel(PfArgs a) {
    constexpr int V = D / 32, ROWS = PfCfg<D, sizeof(T) == 4>::ROWS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_launch();
    grid_dep_wait();
    PfTile w;
    if (!w.init(a, ROWS, (uint32_t)(a.tiles * a.c.n_seqs * a.c.H - a.cut) + blockIdx.x, -1, nullptr)) return;
    const int each = pf_each(w.nj, a.pieces), r = blockIdx.y * kPfJoinRows + warp;
    if (each >= w.nj || r >= w.nrow) return;                   // done in one piece; no such row
    const int n = (w.nj + each - 1) / each;
    const int64_t step = (int64_t)ROWS * (D + 4);
    const float *src = a.part + (int64_t)blockIdx.x * a.pieces * step + (int64_t)r * (D + 4);
    const float2 ml = lane < n ? *reinterpret_cast<const float2 *>(src + lane * step + D) : make_float2(-INFINITY, 0.0f);
    float m = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = ml.y * exp2_approx(ml.x - (m == -INFINITY ? 0.0f : m));   // of its mean
    float l = f, acc[V];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
#pragma unroll 8
    for (int p = 0; p < n; ++p) {
        const float fp = __shfl_sync(0xffffffffu, f, p);
        float y[V];
        if constexpr (V == 4) load4(src + p * step + V * lane, y);
        else *reinterpret_cast<float2 *>(y) = *reinterpret_cast<const float2 *>(src + p * step + V * lane);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += fp * y[e];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const bool lost = __any_sync(0xffffffffu, ml.y < 0.0f);    // a page was not there
    T *dst = static_cast<T *>(a.out) + (w.lo + w.token(r, a.group)) * a.ot + (int64_t)w.head(r, a.group) * a.oh + V * lane;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = lost ? 0.0f : acc[e] * inv;
    if constexpr (V == 4) {
        store4(dst, acc);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) dst[e] = T(acc[e]);
    }
}

// Which row tiles are cut.  A CTA takes a row tile, and a wave one per SM: what does not fill a wave leaves SMs idle for as long as a
// row tile takes, so the last row tiles (the shortest) are cut along the tokens, all of them where there are not enough for a wave.
// Whole / cut in us, 4 KV heads of 128: f32, 112 rows on a sequence of 4096 tokens 66 / 22, on 4 of 32768 493 / 76, on 48 of 2048 (192 row
// tiles) 83 / 71; bf16, 511 rows on 4 of 32768 428 / 128, 1400 on 8 of 4096 132 / 108.  The lengths are the device's, so max_kv stands for
// all: ragged sequences gain less (256 us for 48 of 100 to 16384 tokens, half of it the longest one's).
struct PfCut {
    int64_t tiles, cut;         // row tiles of the longest sequence; those (of all sequences and heads) that do not fill a wave
    int most;                   // pieces at most: three waves of partials are room enough
};
PfCut pf_cut(int32_t n_seqs, int32_t H, int rows, int group, int64_t n_tokens, int64_t max_q) {
    if (max_q > n_tokens) max_q = n_tokens;
    const int64_t sms = sm_count(), tiles = (max_q * group + rows - 1) / rows;
    if ((double)n_seqs * tiles * H > INT_MAX) return {tiles, 0, 1};                  // (refused by the call)
    int64_t jobs = n_seqs * tiles;
    if (n_tokens < n_seqs * max_q) {                           // of ragged sequences about
        const int64_t about = (n_tokens * group + (int64_t)n_seqs * (rows / 2)) / rows;
        jobs = about < n_seqs ? n_seqs : about < jobs ? about : jobs;
    }
    PfCut x = {tiles, jobs * H % sms, 1};
    // (where there are not enough for a wave, those that the estimate has missed too)
    if (jobs * H < sms) x.cut = n_seqs * tiles * H < sms ? n_seqs * tiles * H : sms;
    if (x.cut > 0) x.most = (int)(3 * sms / x.cut < kPfMostPieces ? 3 * sms / x.cut : kPfMostPieces);
    return x;
}
int pf_rows(int dtype) { return dtype == MQKV_F32 ? PfCfg<128, true>::ROWS : PfCfg<128, false>::ROWS; }
// Pieces: what takes the fewest tile steps one after another (within 10% of the best number of pieces nearly everywhere it was tried:
// 1 to 48 sequences, 112 to 1400 rows, 2048 to 32768 tokens).
int pf_pieces(const PfCut &x, const PfArgs &a, int rows, int64_t max_kv) {
    const int64_t last = x.cut / ((int64_t)a.c.n_seqs * a.c.H) + 1;                  // row tiles of a sequence up to the longest that is cut
    int64_t seen = a.causal && last < x.tiles ? max_kv - a.max_q + last * rows / a.group : max_kv;
    seen = seen < 0 ? 0 : seen > max_kv ? max_kv : seen;
    if (a.window > 0 && a.window + rows / a.group < seen) seen = a.window + rows / a.group;
    const double steps = (double)seen / kPfN;
    int best = 1;
    double least = steps + kPfPieceSteps;
    for (int s = 2; s <= x.most && s <= steps; ++s) {
        const double t = (double)((x.cut * s + sm_count() - 1) / sm_count()) * (steps / s + kPfPieceSteps) + kPfJoinSteps + s * kPfPartSteps;
        if (t < least) least = t, best = s;
    }
    return best;
}
constexpr size_t pf_part_bytes(int rows, int D) { return (size_t)rows * (D + 4) * 4; }

template <typename T, int D>
int prefill_t(PfArgs &a, int64_t n_tokens, int64_t max_kv, void *ws, unsigned int *err, cudaStream_t s) {
    using C = PfCfg<D, sizeof(T) == 4>;
    const int slot = kAttrSlotKv + 8 + 2 * (sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 1 : 2) + (D == 128);
    void (*fn)(PfArgs, unsigned int *);
    if constexpr (sizeof(T) == 4) fn = kv_tiles_f32_kernel<D>;
    else fn = kv_tiles_kernel<T, D>;
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(fn), C::SMEM, slot);
    if (rc != MQ_OK) return rc;
    const PfCut x = pf_cut(a.c.n_seqs, a.c.H, C::ROWS, a.group, n_tokens, a.max_q);
    a.pieces = pf_pieces(x, a, C::ROWS, max_kv);
    a.cut = a.pieces > 1 ? (int)x.cut : 0;
    a.part = static_cast<float *>(ws);
    const double grid = (double)a.c.H * a.c.n_seqs * x.tiles + (double)a.cut * (a.pieces - 1);
    if (grid > INT_MAX)
        return set_error(MQ_ERR_SHAPE, "mqkv_attention: %d sequences x %d KV heads x %lld row tiles exceed the grid", a.c.n_seqs, a.c.H, (long long)x.tiles);
    a.tiles = (int)x.tiles;
    rc = cuda_error(launch_pdl(fn, dim3((unsigned)grid), dim3(kPfThreads), C::SMEM, s, a, err), "mqkv_attention (tiles) launch");
    if (rc != MQ_OK || a.cut == 0) return rc;
    const int64_t most = a.max_q * a.group, rows = most < C::ROWS ? most : C::ROWS;
    return cuda_error(launch_pdl(kv_tiles_join_kernel<T, D>, dim3((unsigned)a.cut, (unsigned)((rows + kPfJoinRows - 1) / kPfJoinRows)), dim3(256), 0,
                                 s, a),
                      "mqkv_attention (tiles) join launch");
}

}  // namespace

size_t kv_prefill_ws(int32_t n_seqs, int32_t H, int32_t D, int dtype, int group, int64_t n_tokens, int64_t max_q) {
    const PfCut x = pf_cut(n_seqs, H, pf_rows(dtype), group, n_tokens, max_q);
    return x.most > 1 ? (size_t)x.cut * x.most * pf_part_bytes(pf_rows(dtype), D) : 256;
}

int kv_launch_prefill(const KvView &c, const KvRows &r, const KvAttn &p, void *ws, unsigned int *err, cudaStream_t s) {
    PfArgs a;
    a.c = c, a.r = r, a.q = p.q, a.out = p.out, a.qt = p.qt, a.qh = p.qh, a.ot = p.ot, a.oh = p.oh;
    a.group = p.group, a.causal = p.causal, a.max_q = p.max_q, a.window = p.window;
    a.c_log2 = fabsf(p.scale) * kLog2e;
    a.sign = p.scale < 0.0f ? -1.0f : 1.0f;
    auto go = [&](auto launch) { return launch(a, p.n_tokens, p.max_kv, ws, err, s); };
    if (c.D == 128)
        return p.dtype == MQKV_F32   ? go(prefill_t<float, 128>)
               : p.dtype == MQKV_F16 ? go(prefill_t<__half, 128>)
                                     : go(prefill_t<__nv_bfloat16, 128>);
    return p.dtype == MQKV_F32   ? go(prefill_t<float, 64>)
           : p.dtype == MQKV_F16 ? go(prefill_t<__half, 64>)
                                 : go(prefill_t<__nv_bfloat16, 64>);
}

}  // namespace mq

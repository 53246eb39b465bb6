// mq_kv_attn.cu -- attention over the paged 8-bit cache for few rows per KV head (decode, and checking drafted
// tokens): the cache is streamed from HBM once, every other cost hides under that.
//
// Mathematics.  For one KV head the R rows (new tokens x the query heads of the group) share K and V.  With integer
// codes k, v and block scales dk, dv (one per 32 tokens), s_ij = c dk_j (q_i . k_j), c = scale log2(e); the softmax runs
// in one pass over blocks of 32 tokens with a running maximum m and sum l per row, and
//     o_i = sum_j 2^(s_ij - m_i) dv_j v_j / l_i.
// dv enters the weights (mq_kv_attn.cuh: relative to the row's own largest product of weight and dv), so both products run on exact integers.
//
// Tensor cores.  Decode needs 2 D flops per cached byte and row; the CUDA cores cannot give that at HBM rate for the 7
// rows of a 28:4 head layout (47 TFMA/s of 37), the warp-level m16n8k16 can with 16 rows of which 7 are used (37% of its
// 596 TFLOP/s), and unlike a tcgen05 tile it takes its operands from registers, where the codes are widened to f16.
// f32 rows: rows 0..7 of the 16 hold the leading f16 part of q (and of p'), rows 8..15 the rest, so f32 accuracy costs
// nothing for up to 8 rows.
#include <cuda.h>

#include <type_traits>

#include "mq_kv_attn.cuh"
#include "mq_kv_join.h"

namespace mq {
namespace {

constexpr int kAtWarps = 4, kAtThreads = 32 * kAtWarps;
// what the beginning and end of a row pass cost, in blocks: 0 took 53.0 us for 48 ragged sequences (41.3 and, of f32 rows, 51.0 for 24 windows of
// 20 rows), 2 47.2 (39.4, 50.1), 3 46.7 (38.3, 49.8), 4 46.5 (38.4, 50.0), 8 46.7 (39.0, 51.7)
constexpr uint32_t kAtExtra = 3;
constexpr int kAtSmemSeqs = 256;                // sequences whose plan fits the CTA's shared memory beside two CTAs' rings

struct AtArgs {
    KvView c;
    KvRows r;
    const void *q;
    void *out;
    int64_t qt, qh, ot, oh;
    int32_t group, causal, layer, workers;
    int32_t max_q;
    int64_t window;
    float c_log2, sign;         // |scale| * log2(e), the sign of scale (it goes into q: score factors are not negative)
    uint32_t *prefix;           // [n_seqs + 1][2]: places and units before each sequence
    struct AtJoin *join;        // [workers]
    float *part;                // [worker][2][R rows][D + 4]: the mean, m, l
};

// equal shares of the places: the first rem of them have one more
struct AtShare {
    uint32_t base, rem;
    __device__ __forceinline__ AtShare(uint32_t total, uint32_t n) : base(total / n), rem(total - total / n * n) {}
    __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * base + min(c, rem); }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {
        const uint32_t big = (base + 1) * rem;
        return u < big ? u / (base + 1) : rem + (u - big) / base;
    }
};

// sum += a b, rounded to nearest.  The tensor core cuts its f32 sums toward zero, always the same way, and a share has no longest length: with
// the products added up there, f32 rows over 430 blocks of values of one sign were off by 6.9e-5 and over 1725 by 2.0e-4 (now 3.6e-7 and
// 8.2e-7); two additions more per MMA cost 1 to 3% of the time.
__device__ __forceinline__ void mma16816_add(float (&sum)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    float d[4];
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    f2_unpack(f2_add(f2_pack(sum[0], sum[1]), f2_pack(d[0], d[1])), sum[0], sum[1]);
    f2_unpack(f2_add(f2_pack(sum[2], sum[3]), f2_pack(d[2], d[3])), sum[2], sum[3]);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// CTAs per SM: as many as the registers leave room for without spills (of 128-wide heads three with them took 76 us where two took 49)
constexpr int at_ctas_per_sm(int D, int MT) { return D == 64 && MT == 1 ? 3 : 2; }

// MT: 16-row MMA tiles that share the codes
template <typename T, int D, int MT>
struct AtCfg {
    static constexpr bool TWO = sizeof(T) == 4;
    static constexpr int RT = TWO ? 8 : 16, R = RT * MT;      // rows of an MMA tile, of a pass
    static constexpr int RING = 3;                            // blocks in flight per warp
    static constexpr int BLK = kKB * D, SLOT = 2 * BLK;       // bytes of one 32-token block of K or V
    static constexpr int LD = D + 4;                          // floats of a row of sums
    static constexpr int OFF_BAR = kAtWarps * RING * SLOT;
    static constexpr int OFF_PLAN = OFF_BAR + kAtWarps * RING * 8 + 64;
    static constexpr int SMEM = OFF_PLAN + 1008;              // then the plan
};

// what the call's sequences have to do: R-row passes over the blocks that any of a sequence's rows sees (one block where none
// sees anything, so that its rows are written)
struct AtSeq {
    int64_t lo;                                 // first token row
    int32_t n, len, tiles;                      // new tokens (max_q at most), cached ones, passes
    uint32_t b_lo, nb;                          // first block, blocks
    int64_t first;                              // position of row 0's token
    __device__ __forceinline__ void init(const AtArgs &a, int b, int R, unsigned int *err, bool tell) {
        int64_t hi;
        a.r.of(b, lo, hi);
        n = (int)min(hi - lo, (int64_t)a.max_q), len = a.c.len[b], first = len - (hi - lo);
        if (tell && hi - lo > a.max_q) kv_error(err, KV_ERR_ROWS);
        tiles = (n * a.group + R - 1) / R;
        if (len < 0 || (len > 0 && ((len - 1) >> a.c.tshift) >= a.c.max_pages)) {
            if (tell && n > 0) kv_error(err, KV_ERR_LEN);
            len = 0;
        }
        int64_t x0, y0, x1, y1;
        row_range(first, len, a.causal, a.window, x0, y0);
        row_range(first + n - 1, len, a.causal, a.window, x1, y1);
        b_lo = (uint32_t)((y0 > x0 ? x0 : 0) / kKB);
        nb = max((uint32_t)((max(y0, y1) + kKB - 1) / kKB) - b_lo, 1u);
    }
    // a row pass takes nb places for its blocks after kAtExtra for its beginning and end
    __device__ __forceinline__ uint2 size(int H) const { return make_uint2((uint32_t)(tiles * H) * (nb + kAtExtra), (uint32_t)(tiles * H) * nb); }
};

// places and units before each sequence into prefix[0 .. n_seqs], by one CTA of THREADS threads.  (Their sums stay below 2^32: the
// host has checked it for whole table rows.)
template <int THREADS>
__device__ __forceinline__ void at_plan(const AtArgs &a, int R, uint2 *prefix, uint2 *s_warp, unsigned int *err, bool tell) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint2 before = make_uint2(0, 0);
#pragma unroll 1
    for (int base = 0; base < a.c.n_seqs; base += THREADS) {
        const int b = base + threadIdx.x;
        uint2 v = make_uint2(0, 0);
        if (b < a.c.n_seqs) {
            AtSeq q;
            q.init(a, b, R, err, tell);
            v = q.size(a.c.H);
        }
        uint2 x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x.x, o), z = __shfl_up_sync(0xffffffffu, x.y, o);
            if (lane >= o) x.x += y, x.y += z;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        uint2 w = before;
#pragma unroll 4
        for (int i = 0; i < THREADS / 32; ++i) {
            const uint2 y = s_warp[i];
            if (i < warp) w.x += y.x, w.y += y.y;
            before.x += y.x, before.y += y.y;
        }
        if (b < a.c.n_seqs) prefix[b] = make_uint2(w.x + x.x - v.x, w.y + x.y - v.y);
        __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.c.n_seqs] = before;
    __syncthreads();
}

__global__ void __launch_bounds__(1024) kv_attn_plan_kernel(AtArgs a, int R, unsigned int *err) {
    __shared__ uint2 s_warp[32];
    grid_dep_launch();
    grid_dep_wait();
    uint2 *prefix = reinterpret_cast<uint2 *>(a.prefix);
    at_plan<1024>(a, R, prefix, s_warp, err, true);
}

// the last sequence that begins at or before unit u (one with units)
__device__ __forceinline__ int at_find(const uint2 *prefix, int n_seqs, uint32_t u) {
    int lo = 0, hi = n_seqs - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid].y <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Work is split by units of one block of 32 tokens for one KV head and row pass.  Every warp of the grid (a worker) takes an equal,
// contiguous share of them (of their places: a pass has kAtExtra more than its blocks), whatever the lengths, and walks it through its
// own ring of K / V blocks; loads run ahead over the ends of row passes and no warp waits for another.  Where a row pass ends, or the share does, the sums leave: divided where the pass lies
// in the share whole, else as a partial for the join kernel.  (Shares of whole CTAs, their warps joined in shared memory at the end of
// each pass, left fewer partials but made every end of a pass cost 5 us: 77 us against 49 for a ragged batch of 48 sequences.)
// With its join: 48 sequences of 100 to 16384 tokens, 28 f32 query heads on 4 of 128: 46 us, 198 MB at 4.3 TB/s (fixed latencies of the
// 8 warps per SM bound it: issue 42%, DRAM 61%); two bf16 ones of 200k and 262k: 87 us, 5.5 TB/s.
template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAtThreads, at_ctas_per_sm(D, MT)) kv_attn_kernel(const __grid_constant__ CUtensorMap tm, AtArgs a, unsigned int *err) {
    using C = AtCfg<T, D, MT>;
    constexpr bool TWO = C::TWO;
    constexpr int NT = D / 8, KS = D / 16, RING = C::RING;    // n-tiles of the output, k-steps of the scores
    constexpr int RT = TWO ? 1 : 2;                           // rows of this thread in an MMA tile: g (and g + 8)
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, cc = lane & 3;
    uint8_t *ring = sm + warp * RING * C::SLOT;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR) + warp * RING;
    if (lane == 0) {
        for (int i = 0; i < RING; ++i) mbar_init(bar + i, 1);
        mbar_init_fence();
        if (warp == 0) prefetch_tmap(&tm);
    }
    grid_dep_launch();
    grid_dep_wait();
    const uint2 *prefix = reinterpret_cast<const uint2 *>(a.prefix);
    if (a.c.n_seqs <= kAtSmemSeqs) {
        uint2 *mine = reinterpret_cast<uint2 *>(sm + C::OFF_PLAN);
        at_plan<kAtThreads>(a, C::R, mine, reinterpret_cast<uint2 *>(sm + C::OFF_BAR + kAtWarps * RING * 8), err, blockIdx.x == 0);
        prefix = mine;
    }
    __syncthreads();
    const uint32_t total = prefix[a.c.n_seqs].x, workers = min((uint32_t)a.workers, total), worker = blockIdx.x * kAtWarps + warp;
    if (lane == 0) a.join[worker].nrow = 0;                   // until there is one: the join must not follow what an earlier call has left
    if (worker >= workers) return;                            // every share has a place at least
    const AtShare shares(total, workers);
    const int H = a.c.H, G = a.group;
    // the first unit at or after a place
    auto unit_at = [&](uint32_t place) -> uint32_t {
        if (place >= total) return prefix[a.c.n_seqs].y;
        int lo = 0, hi = a.c.n_seqs - 1;
#pragma unroll 1
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid].x <= place) lo = mid; else hi = mid - 1;
        }
        AtSeq q;
        q.init(a, lo, C::R, err, false);
        const uint32_t r = place - prefix[lo].x, it = r / (q.nb + kAtExtra), in = r - it * (q.nb + kAtExtra);
        return prefix[lo].y + it * q.nb + (in > kAtExtra ? in - kAtExtra : 0);
    };
    uint32_t edge = lane < 2 ? unit_at(shares.begin(worker + lane)) : 0;
    const uint32_t u0 = __shfl_sync(0xffffffffu, edge, 0);
    const int mine = (int)(__shfl_sync(0xffffffffu, edge, 1) - u0);
    if (mine == 0) return;

    // 32 of the warp's units at a time, one a lane: page, scales, where in the page and which head
    int pg = -1, at = 0;
    float dk = 0.0f, dv = 0.0f;
    auto fetch = [&](int k) {
        pg = -1, at = 0, dk = dv = 0.0f;
        if (k + lane < mine) {
            const uint32_t u = u0 + k + lane;
            const int b = at_find(prefix, a.c.n_seqs, u);
            AtSeq q;
            q.init(a, b, C::R, err, false);
            const uint32_t r = u - prefix[b].y, it = r / q.nb, blk = q.b_lo + (r - it * q.nb);
            const int h = (int)(it % H), spp = a.c.T / kKB, sb = (int)blk & (spp - 1);
            at = h << 3 | sb;
            if ((int64_t)blk * kKB < q.len) {
                pg = a.c.table[(int64_t)b * a.c.max_pages + (blk >> (a.c.tshift - 5))];
                if (pg < 0 || pg >= a.c.n_pages) {
                    kv_error(err, KV_ERR_PAGE);
                    pg = -1;
                    dk = -INFINITY;                           // no scale: the passes over the block are lost
                } else {
                    const float *sc = reinterpret_cast<const float *>(a.c.pool + pg * a.c.page_bytes + a.c.off_s);
                    dk = sc[h * spp + sb];
                    dv = sc[(H + h) * spp + sb];
                }
            }
        }
    };
    auto issue = [&](int k, int slot) {                       // the warp's unit k into its ring (a page of -1 reads as zeros)
        const int page = __shfl_sync(0xffffffffu, pg, k & 31), w = __shfl_sync(0xffffffffu, at, k & 31);
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + slot, C::SLOT);
            tma_load_5d(ring + slot * C::SLOT, &tm, 0, (w & 7) * kKB, w >> 3, a.layer, page, bar + slot);
            tma_load_5d(ring + slot * C::SLOT + C::BLK, &tm, 0, (w & 7) * kKB, H + (w >> 3), a.layer, page, bar + slot);
        }
    };
    fetch(0);
    for (int k = 0; k < RING && k < mine; ++k) issue(k, k);
    float dk0 = dk, dv0 = dv;                                 // scales of the batch that is being consumed

    // the current row pass
    int b = at_find(prefix, a.c.n_seqs, u0);
    uint32_t blk = 0;                                         // its first block in this share
    int h = 0, nrow = 0, r0 = 0;                              // first row
    int64_t tok = 0;                                          // token row of row 0's token
    uint32_t last = 0;                                        // the pass's last place
    int all_lo = 0, all_hi = 0;                               // what every row of the pass sees
    int v_lo[MT][RT], v_hi[MT][RT];
    uint32_t qa[MT][KS][4];
    float rs[MT][RT], m[MT][RT], ra[MT][RT], l[MT][RT];       // q's scale, the references m and A, the sum of weights
    float o[MT][NT][4];
    bool lost = false;                                        // a block of this share's part of the pass has no page

    // the row pass of unit u: its rows' q and ranges; how many units of it are left
    auto begin = [&](uint32_t u, bool &fresh) -> uint32_t {
        while (u >= prefix[b + 1].y) ++b;
        AtSeq q;
        q.init(a, b, C::R, err, false);
        const uint32_t r = u - prefix[b].y, it = r / q.nb;
        const int tile = (int)it / H;
        h = (int)it - tile * H;
        blk = q.b_lo + (r - it * q.nb);
        fresh = blk == q.b_lo;                                // the pass begins here
        const uint32_t left = q.nb - (r - it * q.nb);
        last = prefix[b].x + (it + 1) * (q.nb + kAtExtra) - 1;
        tok = q.lo;
        r0 = tile * C::R;
        nrow = min(C::R, q.n * G - r0);
        int64_t x0, y0, x1, y1;
        row_range(q.first + r0 / G, q.len, a.causal, a.window, x0, y0);
        row_range(q.first + (r0 + nrow - 1) / G, q.len, a.causal, a.window, x1, y1);
        all_lo = (int)x1, all_hi = y0 > x0 ? (int)y0 : 0;
        lost = false;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int e = 0; e < RT; ++e) {
                const int rr = t * C::RT + g + 8 * e;
                v_lo[t][e] = v_hi[t][e] = 0;
                m[t][e] = ra[t][e] = -INFINITY, l[t][e] = 0.0f;
                float x[D / 4];
                if (rr < nrow) {
                    const int i = (r0 + rr) / G;
                    row_range(q.first + i, q.len, a.causal, a.window, x0, y0);
                    v_lo[t][e] = (int)x0, v_hi[t][e] = (int)y0;
                    const T *p = static_cast<const T *>(a.q) + (tok + i) * a.qt + (int64_t)(h * G + (r0 + rr - i * G)) * a.qh + cc * (D / 4);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) load4(p + 4 * j, x + 4 * j);
                } else {
#pragma unroll
                    for (int j = 0; j < D / 4; ++j) x[j] = 0.0f;
                }
                float amax = 0.0f;
                bool fin = true;
#pragma unroll
                for (int j = 0; j < D / 4; ++j) {
                    amax = fmaxf(amax, fabsf(x[j]));
                    fin = fin && fabsf(x[j]) <= 3.402823466e38f;
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                fin = (__ballot_sync(0xffffffffu, fin) >> (lane & ~3) & 15u) == 15u;
                const int ex = fin ? row_exponent(amax) : 0;
                // a row with a NaN or an infinity becomes NaN
                const float down = fin ? pow2i(-ex) * a.sign : __int_as_float(0x7fc00000);
                rs[t][e] = pow2i(ex) * a.c_log2;
#pragma unroll
                for (int j = 0; j < D / 4; ++j) x[j] = fin ? x[j] * down : down;
                // k order of the products: k-step ks = 4 hh + s takes the values 16 (2 cc + hh) + 4 s ..+3 (D = 128) or
                // 16 cc + 4 s ..+3 (D = 64) of the row: the 16 bytes that one shared-memory load of K gives
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const float y0 = x[4 * ks], y1 = x[4 * ks + 1], y2 = x[4 * ks + 2], y3 = x[4 * ks + 3];
                    uint32_t w[4];
                    w[e] = pack_f16(y0, y1);
                    w[2 + e] = pack_f16(y2, y3);
                    if constexpr (TWO) {
                        const float2 h0 = unpack_f16(w[0]), h1 = unpack_f16(w[2]);
                        w[1] = pack_f16(y0 - h0.x, y1 - h0.y);
                        w[3] = pack_f16(y2 - h1.x, y3 - h1.y);
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (TWO || (z & 1) == e) qa[t][ks][z] = w[z];
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
        }
        return left;
    };
    // the rows' means leave: into the output where the pass is whole, else as partial `which` of this worker.  Of a lost pass zeros leave, with a sum of
    // weights below zero for the join
    auto end = [&](bool whole, int which) {
        if (lost) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < RT; ++e) {
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 1);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 2);
                if (lost) l[t][e] = whole ? 0.0f : -1.0f;
                const int rr = t * C::RT + g + 8 * e;
                if (rr < nrow) {
                    const float f = l[t][e] == 0.0f ? 0.0f : 1.0f / l[t][e] * ref_factor(ra[t][e], m[t][e]);
                    const int i = (r0 + rr) / G;
                    float *part = a.part + ((int64_t)(2 * worker + which) * C::R + rr) * (D + 4);
                    T *dst = static_cast<T *>(a.out) + (tok + i) * a.ot + (int64_t)(h * G + (r0 + rr - i * G)) * a.oh + cc * (D / 4);
                    // this thread's values 32 cc .. 32 cc + 31 of the row (D = 128): column 2 cc + z of n-tile j is value (2 cc + z) D / 8 + j
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int j = 0; j < NT; j += 4) {
                            float x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) x[k] = (TWO ? o[t][j + k][z] + o[t][j + k][2 + z] : o[t][j + k][2 * e + z]) * f;
                            if (whole) store4(dst + z * NT + j, x);
                            else store4(part + cc * (D / 4) + z * NT + j, x);
                        }
                    if (!whole && cc == 0) *reinterpret_cast<float2 *>(part + D) = make_float2(m[t][e], l[t][e]);
                }
            }
    };

    AtJoin join = {0, 0, 0, 0, 0};
    int slot = 0;                                             // ring slot of the next unit
    uint32_t phase = 0;
    for (int k = 0; k < mine;) {
      bool fresh;
      const uint32_t left = begin(u0 + k, fresh);
      const int k0 = k, stop = k + (int)min((uint32_t)(mine - k), left);
#pragma unroll 1
      for (; k < stop; ++k) {
        const int li = k & 31;
        if (!__all_sync(0xffffffffu, mbar_wait(bar + slot, phase, err, KV_ERR_WAIT, nullptr))) {
            for (int i = 0; i < RING && k + i < mine; ++i) {  // the copies in flight end (again with a limit) before their memory goes
                mbar_wait(bar + slot, phase, err, KV_ERR_WAIT, nullptr);
                if (++slot == RING) slot = 0, phase ^= 1;
            }
            return;
        }
        const uint8_t *sk = ring + slot * C::SLOT, *sv = sk + C::BLK;
        // scores of 32 tokens: four n-tiles of 8
        float s[MT][4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int x = 0; x < MT; ++x) s[x][t][0] = s[x][t][1] = s[x][t][2] = s[x][t][3] = 0.0f;
            const int row = 8 * t + g;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh) {
                const int chunk = D == 128 ? ((2 * cc + hh) ^ (row & 7)) : (cc ^ ((row >> 1) & 3));
                const uint4 w = *reinterpret_cast<const uint4 *>(sk + row * D + chunk * 16);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    uint32_t x, y;
                    codes_f16(ww[z], x, y);
#pragma unroll
                    for (int k = 0; k < MT; ++k) mma16816(s[k][t], qa[k][4 * hh + z], x, y);
                }
            }
        }
        const float dkb = __shfl_sync(0xffffffffu, dk0, li), dvb = __shfl_sync(0xffffffffu, dv0, li);
        lost = lost || dkb == -INFINITY;
        const int t0 = (int)(blk + (k - k0)) * kKB;
        const bool inner = t0 >= all_lo && t0 <= all_hi - kKB;
        const float lgv = log2_approx(dvb);
        bool grow = false;
        float mx[MT][RT], kk[MT][RT];
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int e = 0; e < RT; ++e) {
                // at least 2^-120, so that a masked score stays minus infinity under a scale of zero
                kk[x][e] = fmaxf(rs[x][e] * dkb, 0x1p-120f);
                if constexpr (TWO) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        f2_unpack(f2_add(f2_pack(s[x][t][0], s[x][t][1]), f2_pack(s[x][t][2], s[x][t][3])), s[x][t][0], s[x][t][1]);
                }
                if (!inner) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const int pos = t0 + 8 * t + 2 * cc + z;
                            if (pos < v_lo[x][e] || pos >= v_hi[x][e]) s[x][t][2 * e + z] = -INFINITY;
                        }
                }
                const int f = 2 * e;
                float y = max3(s[x][0][f], s[x][0][f + 1], s[x][1][f]);
                y = max3(y, s[x][1][f + 1], s[x][2][f]);
                y = max3(y, s[x][2][f + 1], s[x][3][f]);
                mx[x][e] = fmaxf(y, s[x][3][f + 1]) * kk[x][e];
                grow = grow || mx[x][e] > m[x][e] + kTau || mx[x][e] + lgv > ra[x][e] + kTau || (m[x][e] == -INFINITY && mx[x][e] > m[x][e]);
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int x = 0; x < MT; ++x) {
                float f[RT];
#pragma unroll
                for (int e = 0; e < RT; ++e) {
                    float y = fmaxf(mx[x][e], __shfl_xor_sync(0xffffffffu, mx[x][e], 1));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                    float ref = fmaxf(ra[x][e], y + lgv);
                    y = fmaxf(y, m[x][e]);
                    ref = fmaxf(ref, y - kRefSpan);
                    l[x][e] *= y == -INFINITY ? 1.0f : exp2_approx(m[x][e] - y);
                    m[x][e] = y;
                    f[e] = ref == -INFINITY ? 1.0f : exp2_approx(ra[x][e] - ref);
                    ra[x][e] = ref;
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[x][j][0] *= f[0], o[x][j][1] *= f[0];
                    o[x][j][2] *= f[RT - 1], o[x][j][3] *= f[RT - 1];
                }
            }
        }
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int e = 0; e < RT; ++e) {
                const float pv = v_factor(dvb, ref_factor(m[x][e], ra[x][e]));
                const uint64_t pv2 = f2_pack(pv, pv);
                const float off = kLazyShift - (m[x][e] == -INFINITY ? 0.0f : m[x][e]);
                const uint64_t off2 = f2_pack(off, off), k2 = f2_pack(kk[x][e], kk[x][e]);
                uint64_t sum = f2_pack(0.0f, 0.0f);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float y, z;
                    f2_unpack(f2_fma(f2_pack(s[x][t][2 * e], s[x][t][2 * e + 1]), k2, off2), y, z);
                    const uint64_t p = f2_pack(exp2_approx(y), exp2_approx(z));
                    sum = f2_add(sum, p);
                    f2_unpack(f2_mul(p, pv2), s[x][t][2 * e], s[x][t][2 * e + 1]);
                }
                float y, z;
                f2_unpack(sum, y, z);
                l[x][e] += y + z;
            }
        // o += p' v: two k-steps of 16 tokens
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
            uint32_t pa[MT][4];
#pragma unroll
            for (int x = 0; x < MT; ++x) {
                float (&sx)[4][4] = s[x];
                pa[x][0] = pack_f16(sx[2 * t2][0], sx[2 * t2][1]);
                pa[x][2] = pack_f16(sx[2 * t2 + 1][0], sx[2 * t2 + 1][1]);
                if constexpr (TWO) {
                    float2 y = unpack_f16(pa[x][0]);
                    pa[x][1] = pack_f16(sx[2 * t2][0] - y.x, sx[2 * t2][1] - y.y);
                    y = unpack_f16(pa[x][2]);
                    pa[x][3] = pack_f16(sx[2 * t2 + 1][0] - y.x, sx[2 * t2 + 1][1] - y.y);
                } else {
                    // the weights of 16-bit rows in one f16 part, for half the MMAs: f16 rows of drafted tokens are 2.6e-4 off, with the
                    // rounding of the outputs alone 2.1e-4; bf16 ones show nothing (1.7e-3)
                    pa[x][1] = pack_f16(sx[2 * t2][2], sx[2 * t2][3]);
                    pa[x][3] = pack_f16(sx[2 * t2 + 1][2], sx[2 * t2 + 1][3]);
                }
            }
            uint32_t w[4][D / 32];                            // tokens 2cc, 2cc+1, 2cc+8, 2cc+9 of the step: D / 8 codes each
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int row = 16 * t2 + 2 * cc + (z & 1) + 8 * (z >> 1);
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(sv + row * D + ((g ^ (row & 7)) * 16));
                    w[z][0] = x.x, w[z][1] = x.y, w[z][2] = x.z, w[z][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(sv + row * D + (((g >> 1) ^ ((row >> 1) & 3)) * 16) + (g & 1) * 8);
                    w[z][0] = x.x, w[z][1] = x.y;
                }
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                // bytes of two tokens side by side: (token, d), (token + 1, d), (token, d + 1), ...
                const uint32_t x0 = __byte_perm(w[0][k], w[1][k], 0x5140), x1 = __byte_perm(w[0][k], w[1][k], 0x7362);
                const uint32_t y0 = __byte_perm(w[2][k], w[3][k], 0x5140), y1 = __byte_perm(w[2][k], w[3][k], 0x7362);
                uint32_t p0, p1, q0, q1;
                codes_f16(x0, p0, p1);
                codes_f16(y0, q0, q1);
#pragma unroll
                for (int x = 0; x < MT; ++x) {
                    mma16816_add(o[x][4 * k + 0], pa[x], p0, q0);
                    mma16816_add(o[x][4 * k + 1], pa[x], p1, q1);
                }
                codes_f16(x1, p0, p1);
                codes_f16(y1, q0, q1);
#pragma unroll
                for (int x = 0; x < MT; ++x) {
                    mma16816_add(o[x][4 * k + 2], pa[x], p0, q0);
                    mma16816_add(o[x][4 * k + 3], pa[x], p1, q1);
                }
            }
        }
        // the slot goes back to the copy engine once every lane's loads are done
        __threadfence_block();
        __syncwarp();
        if (li == 31) dk0 = dk, dv0 = dv;                     // the next unit's batch is the one that was fetched last
        if (k + RING < mine) {
            if (((k + RING) & 31) == 0) fetch(k + RING);
            if (lane == 0) fence_proxy_async_smem();
            issue(k + RING, slot);
        }
        if (++slot == RING) slot = 0, phase ^= 1;
      }
      const bool on = (uint32_t)(k - k0) < left;              // the pass goes on with the next workers
      end(fresh && !on, on);
      if (fresh && on) join = AtJoin{nrow, (int)shares.owner(last), h, r0, tok};
    }
    if (lane == 0) a.join[worker] = join;
}

// Joins one row (the grid's y) of the row passes that several workers share.  Few partials each (FEW): a warp looks at one worker and joins
// what it began alone.  Many: a CTA looks at 8 workers, a lane each, and its 8 warps take every eighth partial.
template <typename T, int D, bool FEW>
__global__ void __launch_bounds__(FEW ? 128 : 256) kv_attn_join_kernel(AtArgs a, int R) {
    constexpr int V = D / 32, JW = FEW ? 1 : 8;
    __shared__ float s_o[FEW ? 1 : JW - 1][D], s_ml[JW][2];
    grid_dep_launch();
    grid_dep_wait();
    const int row = blockIdx.y, lane = threadIdx.x & 31, warp = FEW ? 0 : threadIdx.x >> 5;
    const int mine = FEW ? blockIdx.x * 4 + (threadIdx.x >> 5) : lane < 8 ? blockIdx.x * 8 + lane : a.workers;
    AtJoin w = {0, 0, 0, 0, 0};
    if (mine < a.workers && (!FEW || lane == 0)) {
        w = a.join[mine];
        if (!at_join_holds(w, mine, a.workers, R, a.c.H, a.group, a.r.n_tokens)) w.nrow = 0;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, row < w.nrow); todo != 0; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, first = __shfl_sync(0xffffffffu, mine, from);
        const int last = __shfl_sync(0xffffffffu, w.last, from), n = last - first + 1;
        const float *base = a.part + row * (int64_t)(D + 4);
        auto part = [&](int c) { return base + (2 * (int64_t)c + (c < last)) * R * (D + 4); };
        float mm = -INFINITY, ll = 0.0f, acc[V];
        bool lost = false;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
        // 32 of this warp's partials at a time: a lane has the maximum and the sum of one
        for (int p0 = warp; p0 < n; p0 += 32 * JW) {
            const int p = p0 + JW * lane;
            const float2 ml = p < n ? *reinterpret_cast<const float2 *>(part(first + p) + D) : make_float2(-INFINITY, 0.0f);
            lost = lost || __any_sync(0xffffffffu, ml.y < 0.0f);
            float mn = fmaxf(ml.x, mm);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            const float mb = mn == -INFINITY ? 0.0f : mn, old = exp2_approx(mm - mb), f = ml.y * exp2_approx(ml.x - mb);   // of its mean
            mm = mn;
            float x = f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            ll = ll * old + x;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] *= old;
            const int cnt = min(32, (n - p0 + JW - 1) / JW);
#pragma unroll 8
            for (int j = 0; j < cnt; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, j);
                const float *src = part(first + p0 + JW * j) + V * lane;
                float y[V];
                if constexpr (V == 4) load4(src, y);
                else *reinterpret_cast<float2 *>(y) = *reinterpret_cast<const float2 *>(src);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] += fj * y[e];
            }
        }
        float sum = ll;
        if constexpr (!FEW) {
            if (lane == 0) s_ml[warp][0] = mm, s_ml[warp][1] = lost ? -1.0f : ll;
            if (warp > 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) s_o[warp - 1][V * lane + e] = acc[e];
            }
            __syncthreads();
            if (warp == 0) {
                float all = -INFINITY;
#pragma unroll
                for (int x = 0; x < JW; ++x) all = fmaxf(all, s_ml[x][0]);
                const float mb = all == -INFINITY ? 0.0f : all;
                sum = 0.0f;
#pragma unroll
                for (int x = 0; x < JW; ++x) {
                    const float f = exp2_approx(s_ml[x][0] - mb);
                    lost = lost || s_ml[x][1] < 0.0f;
                    sum += s_ml[x][1] * f;
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = x == 0 ? acc[e] * f : acc[e] + s_o[x - 1][V * lane + e] * f;
                }
            }
        }
        const int r0 = __shfl_sync(0xffffffffu, w.r0, from), h = __shfl_sync(0xffffffffu, w.h, from);
        const int64_t tok = __shfl_sync(0xffffffffu, w.tok, from);
        if (warp == 0) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int i = (r0 + row) / a.group;
            T *dst = static_cast<T *>(a.out) + (tok + i) * a.ot + (int64_t)(h * a.group + (r0 + row - i * a.group)) * a.oh + V * lane;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = lost ? 0.0f : acc[e] * inv;
            if constexpr (V == 4) {
                store4(dst, acc);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) dst[e] = T(acc[e]);
            }
        }
        if constexpr (!FEW) __syncthreads();
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int kv_tensor_map(CUtensorMap *tm, const mqkv_cache &c, const mqkv_layout &lay) {
    EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (enc == nullptr) return set_error(MQ_ERR_CUDA, "cuTensorMapEncodeTiled entry point not available");
    const cuuint64_t dims[5] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_tokens, (cuuint64_t)(2 * c.n_kv_heads),
                                (cuuint64_t)c.n_layers, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.head_dim * c.page_tokens, (cuuint64_t)lay.layer_bytes,
                                   (cuuint64_t)lay.page_bytes};
    const cuuint32_t box[5] = {(cuuint32_t)c.head_dim, kKB, 1, 1, 1}, es[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, c.pool, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(MQ_ERR_CUDA, "cuTensorMapEncodeTiled (cache) failed (%d)", (int)r);
    return MQ_OK;
}

// MMA tiles per pass of 64-wide heads: two where the rows do not fit one, so that the codes are widened once for both (one: 34 us for 31 for 14
// f32 rows, 55 for 47 for 28, on 4 sequences of 32768 tokens, 40 for 38 and 67 for 57 on 48 of 100 to 16384; 28 16-bit rows 38 for 38, 56 for 47).
// Of 128-wide heads one: the sums of two leave no registers for the additions that keep them exact (spills: 55 us for 51 for 14 f32 rows, 85 for 86
// for 28, on 4 of 32768; 66 for 54 for 28 16-bit rows).
int pass_tiles(int D, int dtype, int64_t rows) { return D == 64 && rows > (dtype == MQKV_F32 ? 8 : 16) ? 2 : 1; }
int pass_rows(int D, int dtype, int64_t rows) { return (dtype == MQKV_F32 ? 8 : 16) * pass_tiles(D, dtype, rows); }
// Beyond 32 f32 rows per KV head, 64 16-bit ones: the tcgen05 tiles of mq_kv_prefill.cu.  The passes share work evenly whatever the lengths, row
// tiles are as long as their sequence, and the host does not know the lengths: on both sides of the rule one kind of batch would be up to 45% faster
// with the other kernel.  Passes / tiles in us, 4 KV heads:
//                          4 x 32768 tokens          48 x 2048             48 x 100 to 16384         1 x 4096
//   D 128, f32,  28 rows         85 / 70               71 / 64                105 / 251               16 / 20
//                42             123 / 72               97 / 66                149 / 252               16 / 20
//          bf16, 42              73 / 61               62 / 55                 87 / 210               19 / 17
//                56              91 / 61               77 / 56                111 / 211               18 / 18
//                84             129 / 62              106 / 58                158 / 212               19 / 18
//   D 64,  f32,  32              47 / 57               40 / 51                 57 / 195               17 / 17
//                48              64 / 57               53 / 53                 77 / 195               18 / 17
//          bf16, 48              56 / 50               50 / 47                 70 / 167               21 / 16
//                64              57 / 50               51 / 47                 72 / 167               22 / 16
bool use_tiles(int dtype, int64_t rows) { return rows > (dtype == MQKV_F32 ? 32 : 64); }
// CTAs: as many as are resident, or as there are units for their warps at most
int64_t share_ctas(int32_t n_seqs, int32_t H, int D, int dtype, int64_t rows, int64_t max_kv) {
    const int64_t passes = (rows + pass_rows(D, dtype, rows) - 1) / pass_rows(D, dtype, rows), blocks = (max_kv + kKB - 1) / kKB;
    const int64_t units = passes * H * (blocks > 0 ? blocks : 1) * n_seqs, most = at_ctas_per_sm(D, pass_tiles(D, dtype, rows)) * sm_count();
    return (units + kAtWarps - 1) / kAtWarps < most ? (units + kAtWarps - 1) / kAtWarps : most;
}
size_t plan_bytes(int32_t n_seqs, size_t workers) { return ((((size_t)n_seqs + 4) & ~size_t(3)) * 8 + workers * sizeof(AtJoin) + 255) & ~size_t(255); }

template <typename T, int D, int MT>
int attn_t(const CUtensorMap &tm, const AtArgs &a, int64_t ctas, unsigned int *err, cudaStream_t s) {
    using C = AtCfg<T, D, MT>;
    const int slot = kAttrSlotKv + 2 * (sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 1 : 2) + (D == 128) + (MT == 2 ? 16 : 0);
    const bool in_smem = a.c.n_seqs <= kAtSmemSeqs;
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(&kv_attn_kernel<T, D, MT>), C::SMEM + 8 * (kAtSmemSeqs + 1), slot);
    if (rc == MQ_OK && !in_smem)
        rc = cuda_error(launch_pdl(kv_attn_plan_kernel, dim3(1), dim3(1024), 0, s, a, (int)C::R, err), "mqkv_attention plan launch");
    if (rc != MQ_OK) return rc;
    const size_t smem = C::SMEM + (in_smem ? 8 * (a.c.n_seqs + 1) : 0);
    rc = cuda_error(launch_pdl(kv_attn_kernel<T, D, MT>, dim3((unsigned)ctas), dim3(kAtThreads), smem, s, tm, a, err), "mqkv_attention launch");
    if (rc != MQ_OK) return rc;
    const unsigned rows = (unsigned)(a.max_q * a.group < C::R ? a.max_q * a.group : C::R);
    // Many partials to a pass, from 16 workers a pass on: 14.8 us with them, 34 without, for one sequence of 4096 tokens (128 workers a pass),
    // 17.6 and 24 for 8 (38); 30.6 and 29.0 for 48 of 2048 (6).
    if (a.workers >= 16 * (int64_t)a.c.n_seqs * a.c.H)
        return cuda_error(launch_pdl(kv_attn_join_kernel<T, D, false>, dim3((unsigned)(a.workers + 7) / 8, rows), dim3(256), 0, s, a, (int)C::R),
                          "mqkv_attention join launch");
    return cuda_error(launch_pdl(kv_attn_join_kernel<T, D, true>, dim3((unsigned)(a.workers + 3) / 4, rows), dim3(128), 0, s, a, (int)C::R),
                      "mqkv_attention join launch");
}
template <typename T>
int attn_d(const CUtensorMap &tm, const AtArgs &a, int tiles, int64_t ctas, unsigned int *err, cudaStream_t s) {
    if (a.c.D == 128) return attn_t<T, 128, 1>(tm, a, ctas, err, s);
    return tiles == 1 ? attn_t<T, 64, 1>(tm, a, ctas, err, s) : attn_t<T, 64, 2>(tm, a, ctas, err, s);
}

}  // namespace

size_t kv_attention_ws(int32_t n_seqs, int32_t H, int32_t D, int dtype, int32_t n_q_heads, int64_t n_tokens, int64_t max_q,
                       int64_t max_kv) {
    const int64_t rows = max_q * (n_q_heads / H);
    if (use_tiles(dtype, rows)) return kv_prefill_ws(n_seqs, H, D, dtype, n_q_heads / H, n_tokens, max_q);
    const size_t workers = (size_t)share_ctas(n_seqs, H, D, dtype, rows, max_kv) * kAtWarps;
    return plan_bytes(n_seqs, workers) + workers * 2 * pass_rows(D, dtype, rows) * (D + 4) * 4;
}

int kv_launch_attention(const mqkv_cache &cache, const mqkv_layout &lay, int layer, const KvView &c, const KvRows &r,
                        const KvAttn &p, void *ws, unsigned int *err, cudaStream_t s) {
    const int64_t rows = p.max_q * p.group;
    if (use_tiles(p.dtype, rows)) return kv_launch_prefill(c, r, p, ws, err, s);
    const int64_t passes = (rows + pass_rows(c.D, p.dtype, rows) - 1) / pass_rows(c.D, p.dtype, rows);
    if ((double)c.n_seqs * c.H * passes * ((double)c.max_pages * (c.T / kKB) + kAtExtra + 1) >= 4294967296.0)
        return set_error(MQ_ERR_SHAPE, "mqkv_attention: %d sequences of up to %d pages have too many blocks for one call", c.n_seqs, c.max_pages);
    CUtensorMap tm;
    int rc = kv_tensor_map(&tm, cache, lay);
    if (rc != MQ_OK) return rc;
    AtArgs a;
    a.c = c, a.r = r, a.q = p.q, a.out = p.out, a.qt = p.qt, a.qh = p.qh, a.ot = p.ot, a.oh = p.oh;
    a.group = p.group, a.causal = p.causal, a.layer = layer, a.max_q = (int32_t)p.max_q, a.window = p.window;
    const int64_t ctas = share_ctas(c.n_seqs, c.H, c.D, p.dtype, rows, p.max_kv);
    a.workers = (int)ctas * kAtWarps;
    a.c_log2 = fabsf(p.scale) * kLog2e;
    a.sign = p.scale < 0.0f ? -1.0f : 1.0f;
    a.prefix = static_cast<uint32_t *>(ws);
    a.join = reinterpret_cast<AtJoin *>(a.prefix + 2 * ((c.n_seqs + 4) & ~3));
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + plan_bytes(c.n_seqs, (size_t)a.workers));
    const int tiles = pass_tiles(c.D, p.dtype, rows);
    return p.dtype == MQKV_F32   ? attn_d<float>(tm, a, tiles, ctas, err, s)
           : p.dtype == MQKV_F16 ? attn_d<__half>(tm, a, tiles, ctas, err, s)
                                 : attn_d<__nv_bfloat16>(tm, a, tiles, ctas, err, s);
}

}  // namespace mq

// mq_kv_attn.cu -- attention over the paged 8-bit cache for few rows per KV head (decode, and checking drafted
// tokens): the cache is streamed from HBM once, every other cost hides under that.
//
// Mathematics.  For one KV head the R rows (new tokens x the query heads of the group) share K and V.  With integer
// codes k, v and block scales dk, dv (one per 32 tokens), s_ij = c dk_j (q_i . k_j), c = scale log2(e); the softmax runs
// in one pass over blocks of 32 tokens with a running maximum m and sum l per row, and
//     o_i = sum_j 2^(s_ij - m_i) dv_j v_j / l_i.
// dv enters the weights, p' = 2^(s - m) dv / g with g the largest dv so far, so both products run on exact integers.
//
// Tensor cores.  Decode needs 2 D flops per cached byte and row; the CUDA cores cannot give that at HBM rate for the 7
// rows of a 28:4 head layout (47 TFMA/s of 37), the warp-level m16n8k16 can with 16 rows of which 7 are used (37% of its
// 596 TFLOP/s), and unlike a tcgen05 tile it takes its operands from registers, where the codes are widened to f16.
// f32 rows: rows 0..7 of the 16 hold the leading f16 part of q (and of p'), rows 8..15 the rest, so f32 accuracy costs
// nothing for up to 8 rows.
#include <cuda.h>

#include <type_traits>

#include "mq_kv_attn.cuh"

namespace mq {
namespace {

constexpr int kAtWarps = 4, kAtThreads = 32 * kAtWarps, kAtRing = 3;

struct AtArgs {
    KvView c;
    KvRows r;
    const void *q;
    void *out;
    int64_t qt, qh, ot, oh;
    int32_t group, causal, tiles, nsplit, layer;
    int64_t max_q, window;
    float c_log2;               // scale * log2(e)
    float *part;                // [row][split][D + 2]: o, m, l
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct AtCfg {
    static constexpr int BLK = kKB * D;                       // bytes of one 32-token block of K or V
    static constexpr int SLOT = 2 * BLK;
    static constexpr int OFF_BAR = kAtWarps * kAtRing * SLOT;
    static constexpr int SMEM = OFF_BAR + kAtWarps * kAtRing * 8 + 1024;
    static constexpr int LD = D + 4;                          // merge buffer row (floats)
    static_assert(kAtWarps * 16 * LD * 4 + kAtWarps * 16 * 8 <= OFF_BAR, "the merge buffer reuses the ring");
};

// One CTA: (split, KV head, row tile, sequence).
template <typename T, int D>
__global__ void __launch_bounds__(kAtThreads, 2) kv_attn_kernel(const __grid_constant__ CUtensorMap tm, AtArgs a, unsigned int *err) {
    using C = AtCfg<D>;
    constexpr bool TWO = sizeof(T) == 4;                      // two f16 parts per operand
    constexpr int R = TWO ? 8 : 16;                           // rows of a tile
    constexpr int NT = D / 8;                                 // n-tiles of the output
    constexpr int KS = D / 16;                                // k-steps of the scores
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, cc = lane & 3;
    uint8_t *ring = sm + warp * kAtRing * C::SLOT;
    uint64_t *bar = bars + warp * kAtRing;
    if (lane == 0) {
        for (int i = 0; i < kAtRing; ++i) mbar_init(bar + i, 1);
        mbar_init_fence();
    }
    __syncwarp();
    grid_dep_launch();
    grid_dep_wait();

    int64_t u = blockIdx.x;
    const int split = (int)(u % a.nsplit);
    u /= a.nsplit;
    const int h = (int)(u % a.c.H);
    u /= a.c.H;
    const int tile = (int)(u % a.tiles), b = (int)(u / a.tiles);
    int64_t lo, hi;
    a.r.of(b, lo, hi);
    int64_t n = hi - lo;
    if (n > a.max_q) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_ROWS);
        n = a.max_q;
    }
    const int64_t len = a.c.len[b], first = len - (hi - lo);  // position of row lo
    const int G = a.group;
    const int64_t rows = n * G, r0 = (int64_t)tile * R;
    if (r0 >= rows) return;
    const bool bad = len < 0 || (len > 0 && ((len - 1) >> a.c.tshift) >= a.c.max_pages);
    if (bad && threadIdx.x == 0) kv_error(err, KV_ERR_LEN);
    const int nrow = (int)min((int64_t)R, rows - r0);

    // what the tile sees, and what each of this thread's rows does
    int64_t t_lo = INT64_MAX, t_hi = 0, all_lo = 0, all_hi = INT64_MAX;
    if (!bad) {
        const int64_t i0 = r0 / G, i1 = (r0 + nrow - 1) / G;
        int64_t x, y;
        for (int64_t i = i0; i <= i1; ++i) {
            row_range(first + i, len, a.causal, a.window, x, y);
            if (y > x) t_lo = min(t_lo, x), t_hi = max(t_hi, y);
            all_lo = max(all_lo, x), all_hi = min(all_hi, y);
        }
    }
    if (t_hi == 0) t_lo = 0;
    const int64_t b_lo = t_lo / kKB, b_hi = (t_hi + kKB - 1) / kKB, nb = b_hi - b_lo;
    const int64_t s_lo = b_lo + nb * split / a.nsplit, s_hi = b_lo + nb * (split + 1) / a.nsplit;

    // rows of this thread: g and (one part) g + 8
    constexpr int RT = TWO ? 1 : 2;
    int64_t v_lo[RT], v_hi[RT];
    uint32_t qa[KS][4];
    float rs[RT];
#pragma unroll
    for (int e = 0; e < RT; ++e) {
        const int rr = g + 8 * e;
        v_lo[e] = v_hi[e] = 0;
        rs[e] = 0.0f;
        float x[D / 4];
        const bool in = rr < nrow;
        if (in) {
            const int64_t r = r0 + rr, i = r / G;
            const int gq = (int)(r - i * G);
            row_range(first + i, len, a.causal, a.window, v_lo[e], v_hi[e]);
            const T *p = static_cast<const T *>(a.q) + (lo + i) * a.qt + (int64_t)(h * G + gq) * a.qh + cc * (D / 4);
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
        const float down = pow2i(-ex);
        rs[e] = fin ? pow2i(ex) * a.c_log2 : __int_as_float(0x7fc00000);    // a row with a NaN or an infinity becomes NaN
        // k order of the products: k-step ks = 4 hh + s takes the values 16 (2 cc + hh) + 4 s ..+3 (D = 128)
        // or 16 cc + 4 s ..+3 (D = 64) of the row: the 16 bytes that one shared-memory load of K gives
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const float y0 = fin ? x[4 * ks] * down : 0.0f, y1 = fin ? x[4 * ks + 1] * down : 0.0f;
            const float y2 = fin ? x[4 * ks + 2] * down : 0.0f, y3 = fin ? x[4 * ks + 3] * down : 0.0f;
            const uint32_t p0 = pack_f16(y0, y1), p1 = pack_f16(y2, y3);
            qa[ks][e] = p0;
            qa[ks][2 + e] = p1;
            if constexpr (TWO) {
                const float2 h0 = unpack_f16(p0), h1 = unpack_f16(p1);
                qa[ks][1] = pack_f16(y0 - h0.x, y1 - h0.y);
                qa[ks][3] = pack_f16(y2 - h1.x, y3 - h1.y);
            }
        }
    }

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[RT], l[RT];
#pragma unroll
    for (int e = 0; e < RT; ++e) m[e] = -INFINITY, l[e] = 0.0f;
    float gmax = 0.0f;                                        // the largest V scale so far

    // this warp's blocks: s_lo + warp, + kAtWarps, ...; pages and scales of 32 of them at a time, one a lane
    const int64_t mine = s_hi - s_lo > warp ? (s_hi - s_lo - warp + kAtWarps - 1) / kAtWarps : 0;
    int pg = -1;
    float dk = 0.0f, dv = 0.0f;
    auto fetch = [&](int64_t base) {
        pg = -1, dk = dv = 0.0f;
        if (base + lane < mine) {
            const int64_t blk = s_lo + warp + (base + lane) * kAtWarps;
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
    auto issue = [&](int64_t i, int page) {                   // lane 0: block i of this warp into its ring slot
        const int slot = (int)(i % kAtRing);
        const int tok = (int)(((s_lo + warp + i * kAtWarps) * kKB) & (a.c.T - 1));
        mbar_arrive_expect_tx(bar + slot, C::SLOT);
        tma_load_5d(ring + slot * C::SLOT, &tm, 0, tok, h, a.layer, page, bar + slot);
        tma_load_5d(ring + slot * C::SLOT + C::BLK, &tm, 0, tok, a.c.H + h, a.layer, page, bar + slot);
    };

    // pages of the batch after the one in (pg, dk, dv), for loads issued ahead of their batch
    fetch(0);
    int pg_n = pg;
    float dk_n = 0.0f, dv_n = 0.0f;
    {
        const int pg0 = pg;
        const float dk0 = dk, dv0 = dv;
        fetch(32);
        pg_n = pg, dk_n = dk, dv_n = dv;
        pg = pg0, dk = dk0, dv = dv0;
    }
    for (int i = 0; i < kAtRing && i < mine; ++i) {
        const int page = __shfl_sync(0xffffffffu, pg, i);
        if (lane == 0) issue(i, page);
    }
    bool dead = false;
    for (int64_t i = 0; i < mine; ++i) {
        const int li = (int)(i & 31), slot = (int)(i % kAtRing);
        if (li == 0 && i > 0) {
            pg = pg_n, dk = dk_n, dv = dv_n;
            const int pg0 = pg;
            const float dk0 = dk, dv0 = dv;
            fetch(i + 32);
            pg_n = pg, dk_n = dk, dv_n = dv;
            pg = pg0, dk = dk0, dv = dv0;
        }
        if (!mbar_wait(bar + slot, (uint32_t)(i / kAtRing) & 1, err, KV_ERR_WAIT, nullptr)) {
            dead = true;
            break;
        }
        const uint8_t *sk = ring + slot * C::SLOT, *sv = sk + C::BLK;
        // scores of 32 tokens: four n-tiles of 8
        float s[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
            const int row = 8 * t + g;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh) {
                const int chunk = D == 128 ? ((2 * cc + hh) ^ (row & 7)) : (cc ^ ((row >> 1) & 3));
                const uint4 w = *reinterpret_cast<const uint4 *>(sk + row * D + chunk * 16);
                uint32_t x, y;
                codes_f16(w.x, x, y);
                mma16816(s[t], qa[4 * hh + 0], x, y);
                codes_f16(w.y, x, y);
                mma16816(s[t], qa[4 * hh + 1], x, y);
                codes_f16(w.z, x, y);
                mma16816(s[t], qa[4 * hh + 2], x, y);
                codes_f16(w.w, x, y);
                mma16816(s[t], qa[4 * hh + 3], x, y);
            }
        }
        const float dkb = __shfl_sync(0xffffffffu, dk, li), dvb = __shfl_sync(0xffffffffu, dv, li);
        const int64_t t0 = (s_lo + warp + i * kAtWarps) * kKB;
        const bool inner = t0 >= all_lo && t0 + kKB <= all_hi;
        const float gnew = fmaxf(gmax, dvb);
        const float gold = gnew > 0.0f ? gmax / gnew : 1.0f, pv = gnew > 0.0f ? dvb / gnew : 0.0f;
        gmax = gnew;
        float f[RT];
#pragma unroll
        for (int e = 0; e < RT; ++e) {
            const float k = rs[e] * dkb;
            float mx = -INFINITY;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    float y = TWO ? (s[t][z] + s[t][2 + z]) * k : s[t][2 * e + z] * k;
                    if (!inner) {
                        const int64_t pos = t0 + 8 * t + 2 * cc + z;
                        if (pos < v_lo[e] || pos >= v_hi[e]) y = -INFINITY;
                    }
                    s[t][2 * e + z] = y;
                    mx = fmaxf(mx, y);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[e], mx);
            const float mb = mn == -INFINITY ? 0.0f : mn;
            f[e] = exp2_approx(m[e] - mb);
            m[e] = mn;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float p = exp2_approx(s[t][2 * e + z] - mb + kPShift);
                    sum += p;
                    s[t][2 * e + z] = p * pv;
                }
            l[e] = l[e] * f[e] + sum;
            f[e] *= gold;
        }
        bool same = f[0] == 1.0f;
        if constexpr (RT == 2) same = same && f[1] == 1.0f;
        if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j][0] *= f[0], o[j][1] *= f[0];
                o[j][2] *= f[RT - 1], o[j][3] *= f[RT - 1];
            }
        }
        // o += p' v: two k-steps of 16 tokens
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
            uint32_t pa[4];
            pa[0] = pack_f16(s[2 * t2][0], s[2 * t2][1]);
            pa[2] = pack_f16(s[2 * t2 + 1][0], s[2 * t2 + 1][1]);
            if constexpr (TWO) {
                float2 x = unpack_f16(pa[0]);
                pa[1] = pack_f16(s[2 * t2][0] - x.x, s[2 * t2][1] - x.y);
                x = unpack_f16(pa[2]);
                pa[3] = pack_f16(s[2 * t2 + 1][0] - x.x, s[2 * t2 + 1][1] - x.y);
            } else {
                pa[1] = pack_f16(s[2 * t2][2], s[2 * t2][3]);
                pa[3] = pack_f16(s[2 * t2 + 1][2], s[2 * t2 + 1][3]);
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
                mma16816(o[4 * k + 0], pa, p0, q0);
                mma16816(o[4 * k + 1], pa, p1, q1);
                codes_f16(x1, p0, p1);
                codes_f16(y1, q0, q1);
                mma16816(o[4 * k + 2], pa, p0, q0);
                mma16816(o[4 * k + 3], pa, p1, q1);
            }
        }
        // the slot goes back to the copy engine once every lane's loads are done
        __threadfence_block();
        __syncwarp();
        if (i + kAtRing < mine) {
            const int64_t nx = i + kAtRing;
            const int page = __shfl_sync(0xffffffffu, (nx >> 5) == (i >> 5) ? pg : pg_n, (int)(nx & 31));
            if (lane == 0) {
                fence_proxy_async_smem();
                issue(nx, page);
            }
        }
    }
    (void)dead;

    // join the warps
#pragma unroll
    for (int e = 0; e < RT; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    __syncthreads();                                          // every warp is done with its ring
    float *so = reinterpret_cast<float *>(sm);                // [warp][16][LD]
    float *sml = so + kAtWarps * 16 * C::LD;                  // [warp][16][2]
#pragma unroll
    for (int e = 0; e < RT; ++e) {
        float *row = so + (warp * 16 + g + 8 * e) * C::LD + cc * (D / 4);
        if (cc == 0) sml[(warp * 16 + g + 8 * e) * 2] = m[e], sml[(warp * 16 + g + 8 * e) * 2 + 1] = l[e];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float x = TWO ? o[j][z] + o[j][2 + z] : o[j][2 * e + z];
                row[z * NT + j] = x * gmax;
            }
    }
    __syncthreads();
    // warp w writes rows w, w + 4, ...; a lane holds D / 32 values
    for (int r = warp; r < nrow; r += kAtWarps) {
        float mm = -INFINITY, ll = 0.0f, acc[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) acc[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < kAtWarps; ++w) mm = fmaxf(mm, sml[(w * 16 + r) * 2]);
        const float mb = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
        for (int w = 0; w < kAtWarps; ++w) {
            const float f = exp2_approx(sml[(w * 16 + r) * 2] - mb);
            ll += f * sml[(w * 16 + r) * 2 + 1];
#pragma unroll
            for (int j = 0; j < D / 32; ++j) acc[j] += f * so[(w * 16 + r) * C::LD + (D / 32) * lane + j];
        }
        const int64_t rr = r0 + r, i = rr / G;
        const int gq = (int)(rr - i * G);
        if (a.nsplit == 1) {
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
            T *dst = static_cast<T *>(a.out) + (lo + i) * a.ot + (int64_t)(h * G + gq) * a.oh + (D / 32) * lane;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) acc[j] *= inv;
            if constexpr (D == 128) {
                store4(dst, acc);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) dst[j] = T(acc[j]);
            }
        } else {
            float *dst = a.part + (((lo + i) * (int64_t)(a.c.H * G) + h * G + gq) * a.nsplit + split) * (D + 2);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) dst[(D / 32) * lane + j] = acc[j];
            if (lane == 0) dst[D] = mm, dst[D + 1] = ll;
        }
    }
}

// joins the splits: a warp per row
template <typename T, int D>
__global__ void __launch_bounds__(128) kv_attn_join_kernel(AtArgs a, int64_t n_rows) {
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= n_rows) return;
    const int hq = a.c.H * a.group;
    const float *p = a.part + row * a.nsplit * (D + 2);
    float mm = -INFINITY;
    for (int s = lane; s < a.nsplit; s += 32) mm = fmaxf(mm, p[s * (D + 2) + D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float mb = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f, acc[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] = 0.0f;
    for (int s = 0; s < a.nsplit; ++s) {
        const float f = exp2_approx(p[s * (D + 2) + D] - mb);
        ll += f * p[s * (D + 2) + D + 1];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) acc[j] += f * p[s * (D + 2) + (D / 32) * lane + j];
    }
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    T *dst = static_cast<T *>(a.out) + (row / hq) * a.ot + (row % hq) * a.oh + (D / 32) * lane;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) dst[j] = T(acc[j] * inv);
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

int64_t tiles_of(int dtype, int64_t rows) { return dtype == MQKV_F32 ? (rows + 7) / 8 : (rows + 15) / 16; }

// rows per KV head from which the tcgen05 tiles of mq_kv_prefill.cu are taken
bool use_tiles(int64_t rows) { return rows > 64; }

int splits_of(int32_t n_seqs, int32_t H, int64_t tiles, int64_t max_kv) {
    const int64_t ctas = (int64_t)n_seqs * H * tiles, blocks = (max_kv + kKB - 1) / kKB;
    int64_t s = (2 * sm_count() + ctas - 1) / ctas;
    const int64_t most = (blocks + 2 * kAtWarps - 1) / (2 * kAtWarps);
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s);
}

template <typename T, int D>
int attn_t(const CUtensorMap &tm, const AtArgs &a, int64_t n_tokens, unsigned int *err, cudaStream_t s) {
    using C = AtCfg<D>;
    const int slot = kAttrSlotKv + 2 * (sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 1 : 2) + (D == 128);
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(&kv_attn_kernel<T, D>), C::SMEM, slot);
    if (rc != MQ_OK) return rc;
    rc = cuda_error(launch_pdl(kv_attn_kernel<T, D>, dim3((unsigned)((int64_t)a.nsplit * a.c.H * a.tiles * a.c.n_seqs)), dim3(kAtThreads), C::SMEM, s, tm, a, err),
                    "mqkv_attention launch");
    if (rc != MQ_OK || a.nsplit == 1) return rc;
    const int64_t rows = n_tokens * a.c.H * a.group;
    return cuda_error(launch_pdl(kv_attn_join_kernel<T, D>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a, rows),
                      "mqkv_attention join launch");
}

}  // namespace

size_t kv_attention_ws(int32_t n_seqs, int32_t H, int32_t D, int dtype, int32_t n_q_heads, int64_t n_tokens, int64_t max_q,
                       int64_t max_kv) {
    if (use_tiles(max_q * (n_q_heads / H))) return 256;
    const int n = splits_of(n_seqs, H, tiles_of(dtype, max_q * (n_q_heads / H)), max_kv);
    return n == 1 ? 256 : (size_t)n_tokens * n_q_heads * n * (D + 2) * 4;
}

int kv_launch_attention(const mqkv_cache &cache, const mqkv_layout &lay, int layer, const KvView &c, const KvRows &r,
                        const KvAttn &p, void *ws, unsigned int *err, cudaStream_t s) {
    if (use_tiles(p.max_q * p.group)) return kv_launch_prefill(c, r, p, err, s);
    CUtensorMap tm;
    int rc = kv_tensor_map(&tm, cache, lay);
    if (rc != MQ_OK) return rc;
    AtArgs a;
    a.c = c, a.r = r, a.q = p.q, a.out = p.out, a.qt = p.qt, a.qh = p.qh, a.ot = p.ot, a.oh = p.oh;
    a.group = p.group, a.causal = p.causal, a.layer = layer, a.max_q = p.max_q, a.window = p.window;
    a.tiles = (int)tiles_of(p.dtype, p.max_q * p.group);
    a.nsplit = splits_of(c.n_seqs, c.H, a.tiles, p.max_kv);
    a.c_log2 = p.scale * kLog2e;
    a.part = static_cast<float *>(ws);
    if (c.D == 128)
        return p.dtype == MQKV_F32   ? attn_t<float, 128>(tm, a, r.n_tokens, err, s)
               : p.dtype == MQKV_F16 ? attn_t<__half, 128>(tm, a, r.n_tokens, err, s)
                                     : attn_t<__nv_bfloat16, 128>(tm, a, r.n_tokens, err, s);
    return p.dtype == MQKV_F32   ? attn_t<float, 64>(tm, a, r.n_tokens, err, s)
           : p.dtype == MQKV_F16 ? attn_t<__half, 64>(tm, a, r.n_tokens, err, s)
                                 : attn_t<__nv_bfloat16, 64>(tm, a, r.n_tokens, err, s);
}

}  // namespace mq

// mqd_beam.cu -- one step of beam search: the best continuations over beams and vocabulary.
//
//   score(b, t) = s_b + x_bt - ln sum_t' exp(x_bt')
//
// Two kernels.  The scan reads the logits once: a block takes a piece of a row, keeps the sum of exponentials relative to the largest value met
// (online: a thread rescales its sum when a tile brings a larger one) and, beside it, the piece's best n_cand values, found by a threshold
// that only few values pass.  The join has a block per group: the rows' sums, then n_cand times the best of all lists' heads.
// Within a row the order of the scores is that of the logits, so only the join needs the sums; it compares f32 pairs, 48 bits.
#include <cfloat>
#include <type_traits>

#include "mq_rms.cuh"
#include "mqd.cuh"

namespace mq {
namespace {

constexpr int kScanThreads = 256, kScanPer = 16, kTile = kScanThreads * kScanPer;    // values of a thread, of a block at a time
constexpr int kBuffer = 256, kMaxCand = 64, kMaxLists = 1024;

// order of f32 values (no NaN; +-0 are to be made one before) as unsigned integers, and back
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float exp_neg(float x) { return ex2(x * kLog2e); }

struct BeamPiece {
    float m;            // largest value (-inf: none)
    int32_t n;          // candidates in the list
    float s, e;         // sum of exp(x - m), and what its roundings left out
};
struct BeamWs {
    BeamPiece *piece;   // [rows][pieces]
    float2 *list;       // [rows][pieces][n_cand]: value, token (as bits), the best first
    int pieces;         // of a row
    int64_t length;     // of a piece, a multiple of 8
};

// values of the tile at place e0 in registers, -inf where there is none; vectors of 16 bytes from the boundary at or before the row's beginning (bytes of
// a vector that holds a value of the row lie in that value's 16-byte granule, so no read leaves memory)
template <typename T>
__device__ __forceinline__ void load_tile(const T *base, int first, int stop, int e0, float (&x)[kScanPer]) {
    constexpr int V = 16 / sizeof(T);
    const T *p = base + e0 + threadIdx.x * V;
    uint4 w[kScanPer / V];
    if (e0 >= first && stop - e0 >= kTile) {                // nearly always
#pragma unroll
        for (int j = 0; j < kScanPer / V; ++j) w[j] = __ldcs(reinterpret_cast<const uint4 *>(p + j * kScanThreads * V));
    } else {
        const uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
        for (int j = 0; j < kScanPer / V; ++j) {
            const int e = e0 + (j * kScanThreads + (int)threadIdx.x) * V;
            w[j] = make_uint4(none, none, none, none);
            if (e + V > first && e < stop) w[j] = __ldcs(reinterpret_cast<const uint4 *>(p + j * kScanThreads * V));
        }
    }
#pragma unroll
    for (int j = 0; j < kScanPer / V; ++j) {
        if constexpr (V == 4) {
            x[4 * j] = __uint_as_float(w[j].x), x[4 * j + 1] = __uint_as_float(w[j].y);
            x[4 * j + 2] = __uint_as_float(w[j].z), x[4 * j + 3] = __uint_as_float(w[j].w);
        } else {
            float v[8];
            unpack8(Raw8<T>{w[j]}, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[8 * j + i] = v[i];
        }
    }
    if (!(e0 >= first && stop - e0 >= kTile)) {
#pragma unroll
        for (int j = 0; j < kScanPer; ++j) {
            const int e = e0 + (j / V * kScanThreads + (int)threadIdx.x) * V + j % V;
            if (e < first || e >= stop) x[j] = -INFINITY;
        }
    }
}

// an entry of a list: value and token in the order of unsigned integers, the larger value first and of equals the lower token
__device__ __forceinline__ uint64_t entry(float v, int token) { return ((uint64_t)ordered(v + 0.0f) << 32) | ~(uint32_t)token; }

// the best k of the n entries in s_buf, sorted, to its front; returns how many.  A thread counts what is better than its entry: n^2 / 256 steps a thread,
// for a few dozen entries
__device__ __forceinline__ int keep_best(uint64_t *s_buf, uint64_t *s_best, int n, int k) {
    if (threadIdx.x == 0) s_buf[n] = 0;                     // (pairs are read)
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
        const uint64_t a = s_buf[i];
        const ulonglong2 *two = reinterpret_cast<const ulonglong2 *>(s_buf);
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; j += 2) {
            const ulonglong2 b = two[j / 2];
            rank += (int)(b.x > a) + (int)(b.y > a);
        }
        if (rank < k) s_best[rank] = a;
    }
    __syncthreads();
    n = min(n, k);
    if (threadIdx.x < n) s_buf[threadIdx.x] = s_best[threadIdx.x];
    __syncthreads();
    return n;
}

// sum of exp(v - m)
__device__ __forceinline__ float tile_sum(const float (&v)[kScanPer], float m) {
    const uint64_t neg = f2_pack(-m, -m), l = f2_pack(kLog2e, kLog2e);
    uint64_t sum = f2_pack(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kScanPer; i += 2) {
        float a, b;
        f2_unpack(f2_mul(f2_add(f2_pack(v[i], v[i + 1]), neg), l), a, b);
        sum = f2_add(sum, f2_pack(ex2(a), ex2(b)));
    }
    float a, b;
    f2_unpack(sum, a, b);
    return a + b;
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const T *logits, int64_t stride, int64_t V, const float *scores, int k, BeamWs ws) {
    constexpr int VEC = 16 / sizeof(T);
    __shared__ __align__(16) uint64_t s_buf[kTile + kBuffer + 2];
    __shared__ uint64_t s_best[kMaxCand];
    __shared__ uint32_t s_key[kScanThreads / 32];
    __shared__ int s_hits[kScanThreads / 32];
    __shared__ uint2 s_bar;
    __shared__ float s_m[kScanThreads / 32], s_s[kScanThreads / 32];
    __shared__ int s_n;
    grid_dep_launch();
    grid_dep_wait();
    const int64_t row = blockIdx.x / ws.pieces;
    const int piece = (int)(blockIdx.x - row * ws.pieces), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    BeamPiece *out = ws.piece + blockIdx.x;
    if (!(scores[row] > -INFINITY)) {                       // not alive
        if (threadIdx.x == 0) *out = {-INFINITY, 0, 0.0f, 0.0f};
        return;
    }
    const T *p = logits + row * stride;
    const int first = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    const T *base = p - first;
    const int e0 = (int)(piece * ws.length), stop = (int)min(first + V, e0 + ws.length);
    if (threadIdx.x == 0) s_n = 0;
    float m = -INFINITY, s = 0.0f, thr = -INFINITY;
    int have = 0;

    // token of place i of the tile at `at`
    auto token = [&](int at, int i) { return at - first + ((i / VEC) * kScanThreads + (int)threadIdx.x) * VEC + i % VEC; };
    // NaN and +inf as what they count as; the largest
    auto clean = [&](float(&v)[kScanPer]) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) {
            v[i] = v[i] == v[i] ? fminf(v[i], FLT_MAX) : -INFINITY;
            top = fmaxf(top, v[i]);
        }
        return top;
    };
    // values past the bar (those equal to it: up to token `last`) into the list, as far as it has room
    auto push = [&](const float(&v)[kScanPer], int at, float bar, int last) {
#pragma unroll
        for (int j = 0; j < kScanPer; j += 4) {
            if (!(fmaxf(fmaxf(v[j], v[j + 1]), fmaxf(v[j + 2], v[j + 3])) >= bar)) continue;
#pragma unroll
            for (int i = j; i < j + 4; ++i)
                if ((v[i] > bar) | ((v[i] == bar) & (token(at, i) <= last) & (v[i] > -INFINITY))) {
                    const int n = atomicAdd(&s_n, 1);
                    if (n < kTile + kBuffer) s_buf[n] = entry(v[i], token(at, i));
                }
        }
    };
    // (all threads, after a barrier) entries in the list; nobody adds to it before all know
    auto count = [&]() {
        const int n = s_n;
        __syncthreads();
        return n;
    };
    // (all threads) the best k of the n entries stay; what does not pass their last one is out
    auto settle = [&](int n) {
        if (n > have) {
            have = keep_best(s_buf, s_best, n, k);
            if (threadIdx.x == 0) s_n = have;
            if (have == k) thr = from_ordered((uint32_t)(s_buf[k - 1] >> 32));
            __syncthreads();
        }
    };

    float x[kScanPer];
    load_tile(base, first, stop, e0, x);
    int span = e0, tiles = 1;                               // the list is settled after 1, 2, 4, 8 .. tiles
#pragma unroll 1
    for (int at = e0; at < stop; at += kTile) {
        float v[kScanPer], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) {
            v[i] = x[i];
            top = fmaxf(top, v[i]);                         // (NaN aside)
        }
        if (at + kTile < stop) load_tile(base, first, stop, at + kTile, x);
        float sum = tile_sum(v, fmaxf(top, m));
        if (!(sum <= FLT_MAX)) {                            // a NaN or +inf, or nothing yet but -inf
            top = clean(v);
            sum = fmaxf(top, m) > -INFINITY ? tile_sum(v, fmaxf(top, m)) : 0.0f;
        }
        if (top > m) {
            s *= exp_neg(m - top);                          // (m = -inf: zero)
            m = top;
        }
        s += sum;
        if (at == e0) {
            // every warp's ceil(k / 8)-th largest of its threads' largest values: at least k values are not below the least of these
            const uint32_t own = top > -INFINITY ? ordered(top + 0.0f) : 0u;
            uint32_t key = own, best = 0;
            for (int j = 0; j < (k + 7) / 8; ++j) {
                best = __reduce_max_sync(kFull, key);
                if (lane == __ffs(__ballot_sync(kFull, key == best)) - 1) key = 0;
            }
            if (lane == 0) s_key[warp] = best;
            __syncthreads();
            uint32_t least = s_key[0];
#pragma unroll
            for (int w = 1; w < kScanThreads / 32; ++w) least = min(least, s_key[w]);
            float bar = least != 0 ? from_ordered(least) : -INFINITY;
            int last = INT32_MAX, hits = 0;
            if (top >= bar) {
#pragma unroll
                for (int i = 0; i < kScanPer; ++i) hits += v[i] >= bar;
            }
            hits = __reduce_add_sync(kFull, hits);
            if (lane == 0) s_hits[warp] = hits;
            __syncthreads();
            hits = 0;
#pragma unroll
            for (int w = 0; w < kScanThreads / 32; ++w) hits += s_hits[w];
            if (hits > kBuffer) {
                // a warp has too few values (the end of a row, a mask) or many are equal: the k-th of all threads' largest, by value and token
                uint2 *s_all = reinterpret_cast<uint2 *>(s_buf);
                int at_top = INT32_MAX;
#pragma unroll
                for (int i = kScanPer - 1; i >= 0; --i)
                    if (v[i] == top) at_top = token(at, i);
                s_all[threadIdx.x] = make_uint2(own, (uint32_t)at_top);
                __syncthreads();
                int rank = 0;
#pragma unroll 8
                for (int j = 0; j < kScanThreads; ++j) {
                    const uint2 o = s_all[j];
                    rank += (o.x > own) | ((o.x == own) & (o.y < (uint32_t)at_top));
                }
                const bool kth = own != 0 && rank == k - 1;
                if (kth) s_bar = make_uint2(own, (uint32_t)at_top);
                if (__syncthreads_or(kth)) bar = from_ordered(s_bar.x), last = (int)s_bar.y;
            }
            if (top >= bar) push(v, at, bar, last);
            __syncthreads();
            settle(count());
            span = at + kTile;
            continue;
        }
        if (top > thr) push(v, at, thr, INT32_MIN);         // (of equals the first, which the list holds)
        if (at + kTile - span < tiles * kTile && at + kTile < stop) continue;
        __syncthreads();
        const int n = count();
        if (n > kTile + kBuffer) {
            // more than the list has room for: the span again, tile by tile
            if (threadIdx.x == 0) s_n = have;
            for (int again = span; again <= at; again += kTile) {
                __syncthreads();
                load_tile(base, first, stop, again, v);
                if (clean(v) > thr) push(v, again, thr, INT32_MIN);
                __syncthreads();
                settle(count());
            }
        } else {
            settle(n);
        }
        span = at + kTile;
        tiles = min(2 * tiles, 1 << 16);
    }
    for (int i = threadIdx.x; i < have; i += kScanThreads) 
        ws.list[(int64_t)blockIdx.x * k + i] = make_float2(from_ordered((uint32_t)(s_buf[i] >> 32)), __uint_as_float(~(uint32_t)s_buf[i]));
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (m > -INFINITY) s *= exp_neg(m - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) s_m[warp] = top, s_s[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const float part = lane < kScanThreads / 32 ? s_m[lane] : -INFINITY;
        float all = part, sum = 0.0f, rest = 0.0f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kFull, all, o));
        if (part > -INFINITY) sum = s_s[lane] * exp_neg(part - all);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) pair_add(sum, rest, __shfl_xor_sync(kFull, sum, o), __shfl_xor_sync(kFull, rest, o));
        if (lane == 0) *out = {all, have, sum, rest};
    }
}

// ln(sh + sl) of a positive normal number, as a pair: 2^n f with f in [0.7, 1.42), ln f = 2 (t + t^3 / 3 + .. ) with t = (f - 1) / (f + 1) as a pair; the
// series through t^11 leaves out 2e-11.  (The f64 pipe of this GPU issues ~1.7 operations per clock per SM: log() of a double for every row, with scores in f64
// below, took ten times the rest of this kernel.)
__device__ __forceinline__ void pair_log(float sh, float sl, float &h, float &l) {
    const int n = (int)((__float_as_uint(sh) - 0x3f333333u) >> 23) - (__float_as_uint(sh) < 0x3f333333u ? 512 : 0);
    const float scale = __uint_as_float((uint32_t)(127 - n) << 23);
    const float fh = sh * scale, fl = sl * scale, num = fh - 1.0f;
    float dh, de;
    two_sum(fh, 1.0f, dh, de);
    const float t = __fdiv_rn(num, dh);
    const float r = __fadd_rn(__fmaf_rn(-t, dh, num), __fmaf_rn(-t, __fadd_rn(de, fl), fl));
    const float t1 = __fdiv_rn(r, dh), z = t * t;
    float p = 1.0f / 11.0f;
    p = __fmaf_rn(p, z, 1.0f / 9.0f);
    p = __fmaf_rn(p, z, 1.0f / 7.0f);
    p = __fmaf_rn(p, z, 1.0f / 5.0f);
    p = __fmaf_rn(p, z, 1.0f / 3.0f);
    const float nf = (float)n;
    two_sum(nf * 0.693145751953125f, 2.0f * t, h, l);           // ln 2 in two parts, the product with the first exact
    l = __fadd_rn(l, __fmaf_rn(nf, 1.42860682e-6f, 2.0f * __fmaf_rn(t * z, p, t1)));
}

// a candidate's score cum + x - (lh + ll) as an f32 pair (the rounded sum, the rest: 48 bits) in the order of unsigned integers (0: none)
__device__ __forceinline__ uint64_t score_key(float cum, float x, float lh, float ll) {
    float d, e, h, l;
    two_sum(x, -lh, d, e);                                      // (|x| and the logarithm may be far apart either way)
    e = __fsub_rn(e, ll);
    two_sum(cum, d, h, l);
    const bool fits = fabsf(h) <= FLT_MAX;                      // (past f32 there is no rest)
    l = fits ? __fadd_rn(l, e) : 0.0f;
    const float s = __fadd_rn(h, l);
    l = fits ? __fsub_rn(l, __fsub_rn(s, h)) : 0.0f;
    return ((uint64_t)ordered(s + 0.0f) << 32) | ordered(l + 0.0f);
}
// where it lies: beam, token (of equal scores the lowest comes first)
__device__ __forceinline__ uint64_t place(int beam, float token) { return ((uint64_t)(uint32_t)beam << 32) | __float_as_uint(token); }

// A block per group.  The lists are sorted, so of the lists only the k with the best heads can hold one of the k best (every rank counted: a thread
// per list; lists come in the order of beams and tokens, which decides between equals), and of those only what is not below the k-th head: k^2 entries at most, a
// few k as a rule, whose ranks are counted again.
__global__ void __launch_bounds__(kMaxLists) beam_join_kernel(BeamWs ws, int B, const float *scores, int k, int stop, float *cand_score_out,
                                                              int32_t *cand_row, int32_t *cand_token, float *next_score, int32_t *next_row,
                                                              int32_t *next_token) {
    extern __shared__ __align__(16) uint64_t s_keys[];      // of the heads [lists, even], then key and place of the entries [2][k * min(k, lists)]
    __shared__ uint64_t s_final[2][kMaxCand];
    __shared__ int s_list[kMaxCand], s_n, s_lists;
    __shared__ float s_cum[kMaxCand], s_lh[kMaxCand], s_ll[kMaxCand];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t g = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, P = ws.pieces, lists = B * P, l = threadIdx.x;
    const int beam = l < lists ? l / P : 0;
    const float2 *list = ws.list + g * lists * k;
    float2 head = make_float2(0.0f, 0.0f);
    int n = 0;
    if (l < lists) n = ws.piece[g * lists + l].n, head = list[l * k];   // (not written where n is 0)
    if (threadIdx.x == 0) s_n = 0, s_lists = 0;
    for (int b = warp; b < B; b += warps) {                 // a warp per row: its sum of exponentials
        const BeamPiece *piece = ws.piece + (g * B + b) * P;
        float m = -INFINITY;
        for (int i = lane; i < P; i += 32) m = fmaxf(m, piece[i].m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        float s = 0.0f, e = 0.0f;
        for (int i = lane; i < P; i += 32)
            if (piece[i].m > -INFINITY) {
                const float f = exp_neg(piece[i].m - m), p = __fmul_rn(piece[i].s, f);
                pair_add(s, e, p, __fmaf_rn(piece[i].s, f, -p) + piece[i].e * f);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) pair_add(s, e, __shfl_xor_sync(kFull, s, o), __shfl_xor_sync(kFull, e, o));
        if (lane == 0) {
            float h = 0.0f, c = 0.0f, a, d;                 // (a row without a value has no candidate)
            if (s > 0.0f) pair_log(s, e, h, c);
            two_sum(m > -INFINITY ? m : 0.0f, h, a, d);
            s_lh[b] = a, s_ll[b] = __fadd_rn(d, c);
            s_cum[b] = scores[g * B + b];
        }
    }
    __syncthreads();
    const int even = (lists + 1) & ~1;
    const uint64_t key = n > 0 ? score_key(s_cum[beam], head.x, s_lh[beam], s_ll[beam]) : 0;
    if (l < even) s_keys[l] = key;
    __syncthreads();
    if (n > 0) {
        int rank = 0;
        const ulonglong2 *two = reinterpret_cast<const ulonglong2 *>(s_keys);
#pragma unroll 4
        for (int j = 0; j < even; j += 2) {
            const ulonglong2 o = two[j / 2];
            rank += (o.x > key) | ((o.x == key) & (j < l));
            rank += (o.y > key) | ((o.y == key) & (j + 1 < l));
        }
        if (rank < k) s_list[atomicAdd(&s_lists, 1)] = l;
        if (rank == k - 1) s_final[0][0] = key, s_final[1][0] = place(beam, head.y);
    }
    __syncthreads();
    const int left = s_lists;
    const uint64_t bar = left == k ? s_final[0][0] : 0, at_bar = left == k ? s_final[1][0] : ~0ull;     // the k-th head, where there are as many
    uint64_t *keys = s_keys + even, *places = keys + k * min(k, lists);
    for (int i = warp; i < left; i += warps) {
        const int from = s_list[i], of = from / P, len = ws.piece[g * lists + from].n;
        for (int j = lane; j < len; j += 32) {
            const float2 x = list[from * k + j];
            const uint64_t y = score_key(s_cum[of], x.x, s_lh[of], s_ll[of]), at = place(of, x.y);
            if (y > bar || (y == bar && at <= at_bar)) {
                const int c = atomicAdd(&s_n, 1);
                keys[c] = y, places[c] = at;
            }
        }
    }
    __syncthreads();
    const int all = s_n;
    for (int i = threadIdx.x; i < all; i += blockDim.x) {
        const uint64_t y = keys[i], at = places[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < all; ++j) rank += (keys[j] > y) | ((keys[j] == y) & (places[j] < at));
        if (rank < k) s_final[0][rank] = y, s_final[1][rank] = at;
    }
    __syncthreads();
    if (warp != 0) return;
    const int got = min(all, k);
    int live = 0;                                           // candidates so far that do not end
    for (int i = lane; i < k + lane; i += 32) {             // (all lanes as often)
        const bool in = i < got;
        const float score = in ? from_ordered((uint32_t)(s_final[0][i] >> 32)) : -INFINITY;
        const int row = in ? (int)(g * B + (int64_t)(s_final[1][i] >> 32)) : -1, token = in ? (int)(uint32_t)s_final[1][i] : -1;
        if (i < k) {
            cand_score_out[g * k + i] = score;
            cand_row[g * k + i] = row;
            cand_token[g * k + i] = token;
        }
        const uint32_t goes = __ballot_sync(kFull, in && token != stop);
        const int at = live + __popc(goes & ((1u << lane) - 1));
        if (next_row != nullptr && (goes >> lane & 1) && at < B) {
            next_score[g * B + at] = score;
            next_row[g * B + at] = row;
            next_token[g * B + at] = token;
        }
        live += __popc(goes);
    }
    if (next_row != nullptr)
        for (int i = live + lane; i < B; i += 32) {
            next_score[g * B + i] = -INFINITY;
            next_row[g * B + i] = -1;
            next_token[g * B + i] = -1;
        }
}

// pieces of a row, and their length: some for every SM, none longer than the others (a piece of a few values would have no threshold)
void beam_split(int64_t rows, int B, int64_t V, BeamWs *ws) {
    const int64_t all = (V + 7 + kTile - 1) / kTile;        // (a row begins up to seven places past a boundary)
    const int64_t most = kMaxLists / B;                     // lists of a group: one per thread of the join
    int64_t n = 4 * sm_count() / rows;                      // one wave of blocks, four to an SM
    if (n > all) n = all;
    if (n < 1) n = 1;
    if (n > most) n = most;
    ws->pieces = (int)n;
    ws->length = ((V + 7 + n - 1) / n + 7) / 8 * 8;
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t beam_ws(int64_t n_groups, int B, int64_t V, int n_cand) {
    BeamWs ws;
    beam_split(n_groups * B, B, V, &ws);
    const size_t n = (size_t)n_groups * B * ws.pieces;
    return round256(n * sizeof(BeamPiece)) + round256(n * n_cand * sizeof(float2));
}

int launch_beam_select(int dtype, const void *logits, int64_t stride, int64_t n_groups, int B, int64_t V, const float *scores, int k, int stop,
                       float *cand_score, int32_t *cand_row, int32_t *cand_token, float *next_score, int32_t *next_row, int32_t *next_token,
                       void *workspace, cudaStream_t s) {
    BeamWs ws;
    beam_split(n_groups * B, B, V, &ws);
    const int64_t n = n_groups * B * ws.pieces;
    if (n > INT32_MAX) return set_error(MQ_ERR_SHAPE, "mqd_beam_select: %lld pieces of rows, below 2^31 wanted (fewer groups a call)", (long long)n);
    ws.piece = static_cast<BeamPiece *>(workspace);
    ws.list = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) + round256((size_t)n * sizeof(BeamPiece)));
    const dim3 grid((unsigned)n), block(kScanThreads);
    cudaError_t e = dtype == MQD_F32   ? launch_pdl(beam_scan_kernel<float>, grid, block, 0, s, static_cast<const float *>(logits), stride, V, scores, k, ws)
                    : dtype == MQD_F16 ? launch_pdl(beam_scan_kernel<__half>, grid, block, 0, s, static_cast<const __half *>(logits), stride, V, scores, k, ws)
                                       : launch_pdl(beam_scan_kernel<__nv_bfloat16>, grid, block, 0, s, static_cast<const __nv_bfloat16 *>(logits), stride, V, scores, k, ws);
    // a thread per list, a warp per row, at least eight warps
    const int lists = B * ws.pieces, threads = lists > 256 || B > 8 ? (lists > 32 * B ? (lists + 31) / 32 * 32 : 32 * B < 1024 ? 32 * B : 1024) : 256;
    const int entries = (lists + 1) / 2 * 2 + 2 * k * (k < lists ? k : lists);
    if (e == cudaSuccess) {
        const int rc = ensure_smem_attr(reinterpret_cast<const void *>(beam_join_kernel), (kMaxLists + 2 * kMaxCand * kMaxCand) * 8, kAttrSlotBeam);
        if (rc != MQ_OK) return rc;
        e = launch_pdl(beam_join_kernel, dim3((unsigned)n_groups), dim3(threads), entries * 8, s, ws, B, scores, k, stop, cand_score, cand_row,
                       cand_token, next_score, next_row, next_token);
    }
    return cuda_error(e, "mqd_beam_select launch");
}

}  // namespace mq

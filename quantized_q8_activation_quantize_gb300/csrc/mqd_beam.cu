// mqd_beam.cu -- one step of beam search: the best continuations over beams and vocabulary.
//
//   score(b, t) = s_b + x_bt - ln sum_t' exp(x_bt')
//
// Two kernels.  The scan reads the logits once: a block takes a piece of a row, keeps the sum of exponentials relative to a value met
// (online: a thread rescales its sum when a tile brings a much larger one) and, beside it, the piece's best n_cand values, found by a threshold
// that only few values pass.  The join has a block per group: the rows' sums, then ranks, of many lists first of their heads and then of the entries that are left, or mergers of the lists.
// Within a row the order of the scores is that of the logits, so only the join needs the sums; it compares f32 pairs, 48 bits.
//
// 128 rows of 152064 f32 logits (77.9 MB) in groups of four, eight candidates: 21.4 us in a graph; their bytes alone are 11.5 at the copy rate.  What is above it: a first tile's
// threshold and list before any other tile counts, the ends of the pieces, and the join's chain (sums, heads, ranks).  4 rows: 9.3 us, the two chains.
#include <cfloat>
#include <type_traits>

#include "mq_rms.cuh"
#include "mqd.cuh"
#include "mqd_beam_merge.h"

namespace mq {
namespace {

constexpr int kScanThreads = 256, kScanPer = 16, kTile = kScanThreads * kScanPer;    // values of a thread, of a block at a time
constexpr int kStages = 3;          // tiles of a block in flight or in work: 48 KB (f32), so that three blocks fit an SM.  128 rows: 22.3 us, two stages 22.7, four 28.5, through registers 27
constexpr int kBuffer = 256, kMaxCand = 64, kMaxLists = 1024, kRoom = 2048 + kMaxCand;     // room of a piece's list while it is made

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504f;
constexpr float kLag = 4.0f;            // how far above a thread's reference its values may rise before its sum is rescaled
__device__ __forceinline__ float exp_neg(float x) { return ex2(x * kLog2e); }

struct BeamPiece {
    float m;            // what the sum is relative to, a value of the piece (-inf: it has none)
    int32_t n;          // candidates in the list
    float s, e;         // sum of exp(x - m), and what its roundings left out
};
struct BeamWs {
    BeamPiece *piece;   // [rows][pieces]
    float2 *list;       // [rows][pieces][n_cand]: value, token (as bits), the best first
    int pieces;         // of a row
    int64_t length;     // of a piece, a multiple of 8
};

// A tile on its way: every thread copies its own vectors of 16 bytes into its own slots of a stage and waits for its own copies only, so stages need no
// barriers.  Vectors begin at the boundary at or before the row's beginning, those without a value of the row are left out (bytes of a vector that
// holds one lie in that value's 16-byte granule, so no read leaves memory).
template <typename T>
__device__ __forceinline__ void ask_tile(const T *base, int first, int stop, int e0, uint4 *stage) {
    constexpr int V = 16 / sizeof(T);
    const T *p = base + e0 + threadIdx.x * V;
    const uint32_t to = smem_u32(stage + threadIdx.x);
    if (e0 >= first && stop - e0 >= kTile) {                // nearly always
#pragma unroll
        for (int j = 0; j < kScanPer / V; ++j)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + j * kScanThreads * 16), "l"(p + j * kScanThreads * V) : "memory");
    } else {
#pragma unroll
        for (int j = 0; j < kScanPer / V; ++j) {
            const int e = e0 + (j * kScanThreads + (int)threadIdx.x) * V;
            if (e + V > first && e < stop)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + j * kScanThreads * 16), "l"(p + j * kScanThreads * V) : "memory");
        }
    }
}
__device__ __forceinline__ void ask_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ask_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// its values, -inf where the row has none
template <typename T>
__device__ __forceinline__ void read_tile(const uint4 *stage, int first, int stop, int e0, float (&x)[kScanPer]) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < kScanPer / V; ++j) {
        const uint4 w = stage[j * kScanThreads + threadIdx.x];
        if constexpr (V == 4) {
            x[4 * j] = __uint_as_float(w.x), x[4 * j + 1] = __uint_as_float(w.y), x[4 * j + 2] = __uint_as_float(w.z), x[4 * j + 3] = __uint_as_float(w.w);
        } else {
            float v[8];
            unpack8(Raw8<T>{w}, v);
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

// the best k of the n entries in s_buf, sorted, to s_best and to its front (there for all after the next barrier); returns how many.  A thread counts what is
// better than its entry: n^2 / 512 steps a thread, for a few dozen entries
__device__ __forceinline__ int keep_best(uint64_t *s_buf, uint64_t *s_best, int n, int k) {
    const ulonglong2 *two = reinterpret_cast<const ulonglong2 *>(s_buf);
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
        const uint64_t a = s_buf[i];
        int rank = (n & 1) ? (int)(s_buf[n - 1] > a) : 0;
#pragma unroll 4
        for (int j = 0; j < n / 2; ++j) {
            const ulonglong2 b = two[j];
            rank += (int)(b.x > a) + (int)(b.y > a);
        }
        if (rank < k) s_best[rank] = a;
    }
    __syncthreads();
    n = min(n, k);
    if (threadIdx.x < n) s_buf[threadIdx.x] = s_best[threadIdx.x];
    return n;
}

// sum of exp(v - m), added up as a tree
__device__ __forceinline__ float tile_sum(const float (&v)[kScanPer], float m) {
    const uint64_t neg = f2_pack(-m, -m), l = f2_pack(kLog2e, kLog2e);
    uint64_t sum[kScanPer / 2];
#pragma unroll
    for (int i = 0; i < kScanPer / 2; ++i) {
        float a, b;
        f2_unpack(f2_mul(f2_add(f2_pack(v[2 * i], v[2 * i + 1]), neg), l), a, b);
        sum[i] = f2_pack(ex2(a), ex2(b));
    }
#pragma unroll
    for (int o = kScanPer / 4; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) sum[i] = f2_add(sum[i], sum[i + o]);
    float a, b;
    f2_unpack(sum[0], a, b);
    return a + b;
}

// the largest f32 below x, which is finite
__device__ __forceinline__ float below(float x) {
    const uint32_t u = ordered(x + 0.0f);
    return from_ordered(u - (u == 0x80000000u ? 2u : 1u));  // (minus zero is not below zero)
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads, 3) beam_scan_kernel(const T *logits, int64_t stride, int64_t V, const float *scores, int k, BeamWs ws) {
    constexpr int VEC = 16 / sizeof(T), kStageVecs = kTile / VEC;
    extern __shared__ uint4 s_stage[];                      // [kStages][kStageVecs]
    __shared__ __align__(16) uint64_t s_buf[kRoom + 2];
    __shared__ uint64_t s_best[kMaxCand];
    __shared__ uint32_t s_key[kScanThreads / 32];
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
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (e0 + i * kTile < stop) ask_tile(base, first, stop, e0 + i * kTile, s_stage + i * kStageVecs);
        ask_done();
    }
    if (threadIdx.x == 0) s_n = 0;
    float m = -INFINITY, high = -INFINITY, s = 0.0f, rest = 0.0f, thr = -INFINITY;     // high: m + kLag; the sum relative to m, and what its last rounding left out
    int have = 0;

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
    // Values past the bar into the list, as far as it has room; their count in any case.  Few pass: a mask of them, then one after the other, its value
    // again from where it came (of the values that are equal to `tie` those up to token `last` pass too).
    auto push = [&](const float(&v)[kScanPer], const T *from, int at, float bar, float tie, int last) {
        const int t0 = at - first + (int)threadIdx.x * VEC;
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) mask |= (uint32_t)(v[i] > bar) << i;
        if (last != INT32_MIN) {
#pragma unroll
            for (int i = 0; i < kScanPer; ++i)
                mask |= (uint32_t)((v[i] == tie) & (t0 + i / VEC * (kScanThreads * VEC) + i % VEC <= last)) << i;
        }
        if (mask == 0) return;
        int n = atomicAdd(&s_n, __popc(mask));
#pragma unroll 1
        for (; mask != 0; mask &= mask - 1, ++n) {
            const int i = __ffs(mask) - 1, e = i / VEC * (kScanThreads * VEC) + i % VEC;
            if (n < kRoom) s_buf[n] = entry(fminf(to_f32(from[(int)threadIdx.x * VEC + e]), FLT_MAX), t0 + e);
        }
    };
    // (all threads) a bar that at least k values of a tile pass, where it has as many, and no more than the larger of kBuffer and 16 k: those above it, and of those equal to `tie` those up to token `last`
    auto tile_bar = [&](const float(&v)[kScanPer], float top, int at, float &bar, float &tie, int &last) {
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
        bar = least != 0 ? below(from_ordered(least)) : -INFINITY;
        int hits = 0;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) hits += v[i] > bar;
        // a warp has too few values (the end of a row, a mask) or many are equal: the k-th of all threads' largest, by value and token
        if (__syncthreads_or(__reduce_add_sync(kFull, hits) > kBuffer / (kScanThreads / 32))) {
            uint2 *s_all = reinterpret_cast<uint2 *>(s_buf + kMaxCand);       // (the list's own entries lie before)
            int at_top = INT32_MAX;
#pragma unroll
            for (int i = kScanPer - 1; i >= 0; --i)
                if (v[i] == top) at_top = at - first + ((i / VEC) * kScanThreads + (int)threadIdx.x) * VEC + i % VEC;
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
            if (__syncthreads_or(kth)) bar = tie = from_ordered(s_bar.x), last = (int)s_bar.y;
        }
    };
    // (all threads, after a barrier) the best k of the list's n entries stay; what does not pass their last one is out
    auto settle = [&](int n) {
        if (n > have) {
            have = keep_best(s_buf, s_best, n, k);
            if (threadIdx.x == 0) s_n = have;
            if (have == k) thr = from_ordered((uint32_t)(s_best[k - 1] >> 32));
        }
        __syncthreads();                                    // nobody adds to the list before all know its count
    };

    int span = e0, tiles = 1, slot = 0;                     // the list is settled after 1, 2, 4, 8 .. tiles
#pragma unroll 1
    for (int at = e0; at < stop; at += kTile) {
        {
            const int next = at + (kStages - 1) * kTile, into = slot == 0 ? kStages - 1 : slot - 1;     // (the stage that was read last)
            if (next < stop) ask_tile(base, first, stop, next, s_stage + into * kStageVecs);
            ask_done();
            ask_wait<kStages - 1>();
        }
        float v[kScanPer], top = -INFINITY;
        const uint4 *tile = s_stage + slot * kStageVecs;
        read_tile<T>(tile, first, stop, at, v);
        slot = slot == kStages - 1 ? 0 : slot + 1;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) top = fmaxf(top, v[i]);                                      // (NaN aside)
        // A sum that was rescaled with every tile of a rising row would take that factor's error as often; so only where values rise by kLag, and the running
        // sum keeps its roundings: what a row's logarithm is off by does not grow with the row (460 rows of 2^22 equal logits below a peak were off by 1.9e-5 so, by 8e-8 now).
        float ref = top > high ? top : m, sum = tile_sum(v, ref);
        if (!(sum <= FLT_MAX)) {                            // a NaN or +inf, or nothing yet but -inf
            top = clean(v);
            ref = top > high ? top : m;
            sum = ref > -INFINITY ? tile_sum(v, ref) : 0.0f;
        }
        if (ref > m) {
            const float f = exp_neg(m - ref);               // (m = -inf: zero)
            s *= f, rest *= f, m = ref, high = m + kLag;
        }
        const float more = __fadd_rn(sum, rest), next_s = __fadd_rn(s, more);   // (Kahan)
        rest = __fsub_rn(more, __fsub_rn(next_s, s));
        s = next_s;
        float bar = thr, tie = 0.0f;                        // (of equals the first, which the list holds)
        int last = INT32_MIN;
        const bool begin = at == e0;
        if (begin) {
            tile_bar(v, top, at, bar, tie, last);
        }
        if (top > bar || last != INT32_MIN) push(v, reinterpret_cast<const T *>(tile), at, bar, tie, last);
        if (!begin && at + kTile - span < tiles * kTile && at + kTile < stop) continue;
        __syncthreads();
        const int n = s_n;
        if (n > kRoom) {
            // more than the list has room for (rows that rise): the span again, a tile at a time, each by a bar of its own (128 rising rows 145 us; settled after every
            // 2048 values, of which all passed, 8.6 ms)
            __syncthreads();
            if (threadIdx.x == 0) s_n = have;
#pragma unroll 1
            for (int again = span; again <= at; again += kTile) {
                __syncthreads();
                float z[kScanPer];
#pragma unroll
                for (int i = 0; i < kScanPer; ++i) {
                    const int e = again + ((i / VEC) * kScanThreads + (int)threadIdx.x) * VEC + i % VEC;
                    z[i] = e >= first && e < stop ? to_f32(base[e]) : -INFINITY;
                }
                const float most = clean(z);
                float own_bar = -INFINITY, own_tie = 0.0f;
                int own_last = INT32_MIN;
                tile_bar(z, most, again, own_bar, own_tie, own_last);
                if (own_bar < thr) own_bar = thr, own_last = INT32_MIN;
                if (most > own_bar || own_last != INT32_MIN) push(z, base + again, again, own_bar, own_tie, own_last);
                __syncthreads();
                settle(s_n);
            }
        } else {
            settle(n);
        }
        span = at + kTile;
        if (!begin) tiles = min(2 * tiles, 1 << 16);
    }
    for (int i = threadIdx.x; i < have; i += kScanThreads)
        ws.list[(int64_t)blockIdx.x * k + i] = make_float2(from_ordered((uint32_t)(s_buf[i] >> 32)), __uint_as_float(~(uint32_t)s_buf[i]));
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    s = m > -INFINITY ? (s + rest) * exp_neg(m - top) : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) s_m[warp] = top, s_s[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const float part = lane < kScanThreads / 32 ? s_m[lane] : -INFINITY;
        float all = part, sum = 0.0f, left = 0.0f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kFull, all, o));
        if (part > -INFINITY) sum = s_s[lane] * exp_neg(part - all);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) pair_add(sum, left, __shfl_xor_sync(kFull, sum, o), __shfl_xor_sync(kFull, left, o));
        if (lane == 0) *out = {all, have, sum, left};
    }
}

// How many of the n (a multiple of 4) numbers are larger than this one (EQUAL: or the same).  Four lanes share the count; all of them get it.
template <bool EQUAL>
__device__ __forceinline__ int rank_of(const uint32_t *his, int n, uint32_t hi) {
    const uint4 *four = reinterpret_cast<const uint4 *>(his);
    const uint32_t x = EQUAL ? hi - 1 : hi;                 // (hi > 0)
    int rank = 0;
#pragma unroll 4
    for (int j = threadIdx.x & 3; j < n / 4; j += 4) {
        const uint4 o = four[j];
        rank += (int)(o.x > x) + (int)(o.y > x) + (int)(o.z > x) + (int)(o.w > x);
    }
    rank += __shfl_xor_sync(kFull, rank, 1);
    return rank + __shfl_xor_sync(kFull, rank, 2);
}
// The rank of item i among n by upper halves, where it is below k (else k); items that look the same: by lower halves and place(j), the lowest first.  All four lanes
// of an item, all lanes of a warp.
template <typename Place>
__device__ __forceinline__ int rank_below(const uint32_t *his, const uint32_t *los, int n, int n4, int i, int k, Place place) {
    const uint32_t hi = his[i];
    int rank = rank_of<false>(his, n4, hi);
    const bool in = hi != 0 && rank < k;
    if (!__any_sync(kFull, in)) return k;
    const int same = rank_of<true>(his, n4, max(hi, 1u));
    if (__any_sync(kFull, in && same > rank + 1)) {
        int more = 0;
        const uint32_t lo = los[i], at = place(i);
#pragma unroll 4
        for (int j = threadIdx.x & 3; j < n; j += 4)
            more += (int)((his[j] == hi) & ((los[j] > lo) | ((los[j] == lo) & (place(j) < at))));
        more += __shfl_xor_sync(kFull, more, 1);
        rank += more + __shfl_xor_sync(kFull, more, 2);
    }
    return in ? rank : k;
}

constexpr int kJoinThreads = 512;      // with 40 registers: room beside the scan's blocks, so that it waits on its SM when they end.  4 rows 9.3 us, 256 threads 10.1, 1024 9.4;
                                       // 96 rows in groups of 16 (32 candidates) 18.7, 22.2, 17.3
// Whether the join ranks every entry of a group's lists by all others: where four lanes of the block have each.  32 groups of 12 lists of 8: 21.4 us, by heads first
// 22.5; one of 8 of 2 6.1 and 7.1.
__host__ __device__ inline bool join_few(int lists, int k) { return lists * k <= kJoinThreads / 4; }
constexpr int kJoinRanked = 256;       // entries that it still ranks so after a choice of lists, in two rounds
// words of its shared memory: keys and tokens of few entries; else the heads' keys where there are more lists than k, and two buffers of entries (keys, places)
__host__ __device__ inline int join_heads(int lists, int k) { return lists > k ? lists + 3 & ~3 : 0; }
inline int join_words(int lists, int k) {
    const int merged = 6 * (lists < k ? lists : k) * k;
    return join_few(lists, k) ? 4 * (lists * k + 4) : 2 * join_heads(lists, k) + (merged > 4 * kJoinRanked ? merged : 4 * kJoinRanked);
}

// Merges `left` lists of up to k entries, those of list_of(0), list_of(1) .. , until the k best are in order: their scores, rows and tokens; returns how many there are
template <typename ListOf>
__device__ __forceinline__ int join_merge(uint32_t *buffers, int room, int left, int k, int P, ListOf list_of, const float2 *list, const int *s_len, const float *s_cum, const float *s_lh,
                                          const float *s_ll, float *s_score, int *s_row, int *s_token) {
    uint64_t *key = reinterpret_cast<uint64_t *>(buffers), *key2 = key + room;
    uint32_t *place = reinterpret_cast<uint32_t *>(key2 + room), *place2 = place + room;        // list, and where in it
    const int dq = kJoinThreads / k, dj = kJoinThreads - dq * k, q0 = threadIdx.x / k, j0 = threadIdx.x - q0 * k;       // (entry i of list i / k, without a division each)
    // (both buffers begin with places of the lists: whatever a slot holds leads to memory of the call)
    for (int i = threadIdx.x, q = q0, j = j0; i < left * k; i += kJoinThreads) {
        const int from = list_of(q), of = from / P;
        key[i] = j < s_len[from] ? score_key(s_cum[of], list[from * k + j].x, s_lh[of], s_ll[of]) : 0;
        place[i] = place2[i] = from * kMaxCand + j;
        q += dq, j += dj;
        if (j >= k) j -= k, ++q;
    }
    __syncthreads();
    // A list is in the order of its logits, its keys only nearly so (score_key): where one is not, each is taken as no larger than those before it, a warp a list
    bool rises = false;
    for (int i = threadIdx.x, j = j0; i < left * k; i += kJoinThreads) {
        rises |= j != 0 && key[i] > key[i - 1];
        j += dj;
        if (j >= k) j -= k;
    }
    if (__syncthreads_or(rises)) {
        const int lane = threadIdx.x & 31;
        for (int q = threadIdx.x >> 5; q < left; q += kJoinThreads / 32) {
            uint64_t least = ~(uint64_t)0;
            for (int j = lane; j < k + lane; j += 32) {     // (all lanes as often)
                uint64_t x = j < k ? key[q * k + j] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(kFull, x, o);
                    if (lane >= o && y < x) x = y;
                }
                x = x < least ? x : least;
                least = __shfl_sync(kFull, x, 31);
                if (j < k) key[q * k + j] = x;
            }
        }
        __syncthreads();
    }
    for (int s = 1, runs = left; s < left; s *= 2, runs = (runs + 1) / 2) {         // list a of this round lies at slot a * s
        for (int i = threadIdx.x, a = q0, j = j0; i < runs * k; i += kJoinThreads) {
            const int to = merge_slot(key, runs, s, k, a, j);
            if (to >= 0) key2[to] = key[a * s * k + j], place2[to] = place[a * s * k + j];
            a += dq, j += dj;
            if (j >= k) j -= k, ++a;
        }
        __syncthreads();
        uint64_t *const old = key;
        uint32_t *const oldp = place;
        key = key2, key2 = old, place = place2, place2 = oldp;
    }
    const bool in = (int)threadIdx.x < k && key[threadIdx.x] != 0;
    if (in) {
        const int at = place[threadIdx.x], from = at / kMaxCand;
        s_score[threadIdx.x] = from_ordered((uint32_t)(key[threadIdx.x] >> 32)), s_row[threadIdx.x] = from / P;
        s_token[threadIdx.x] = __float_as_int(list[from * k + at % kMaxCand].y);
    }
    return __syncthreads_count(in);
}

// A block per group.  Few entries are ranked each by all others.  Of more lists, which are sorted, only the k with the best heads can hold one of the k best (the heads' ranks
// are counted; lists come in the order of beams and tokens, which decides between equals), and of those only what is not below the k-th head: a few k entries as a rule, which are
// ranked.  Many equal scores, or many candidates of few lists, can leave k^2: then the lists merge in pairs of neighbours, the k best of each pair, until one is left; an entry's
// place is its own and what a binary search finds before it in the other list.  (Ranks alone took 143 us for 64 candidates of 4 rows of 50000 bf16 logits, 16.5 so, and 25 for 32
// of 152 in pairs, 20.7 so; mergers alone 37 for 27 for 64 of 16 rows of 152064 in one group, 10.7 for 9.6 for 8 of 4.  The best of all heads k times cost 300 clocks each.)
__global__ void __launch_bounds__(kJoinThreads, 3) beam_join_kernel(BeamWs ws, int B, const float *scores, int k, int stop, float *cand_score_out,
                                                                 int32_t *cand_row, int32_t *cand_token, float *next_score, int32_t *next_row,
                                                                 int32_t *next_token) {
    extern __shared__ __align__(16) uint32_t s_keys[];      // (join_words)
    __shared__ uint32_t s_take[kMaxLists / 32], s_bar[3];   // lists that may hold one of the best; the worst of their heads, and its list
    __shared__ float s_score[kMaxCand];
    __shared__ int s_row[kMaxCand], s_token[kMaxCand], s_list[kMaxCand], s_n, s_lists;
    __shared__ float s_cum[kMaxCand], s_lh[kMaxCand], s_ll[kMaxCand];
    __shared__ int s_len[kMaxLists];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t g = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kJoinThreads / 32, P = ws.pieces, lists = B * P;
    const float2 *list = ws.list + g * lists * k;
    const bool few = join_few(lists, k);
    float head[kMaxLists / kJoinThreads];
    float2 own;                                             // of few entries, a thread's
#pragma unroll
    for (int i = 0; i < kMaxLists / kJoinThreads; ++i) {
        const int l = threadIdx.x + i * kJoinThreads;
        if (l < lists) s_len[l] = ws.piece[g * lists + l].n, head[i] = list[l * k].x;   // (not written where there is none)
    }
    if (few && threadIdx.x < lists * k) own = list[threadIdx.x];
    if (threadIdx.x < kMaxLists / 32) s_take[threadIdx.x] = 0;
    if (threadIdx.x == 0) s_n = 0, s_lists = 0;
    for (int b = warp; b < B; b += warps) {                 // a warp per row: its sum of exponentials
        const float4 *piece = reinterpret_cast<const float4 *>(ws.piece + (g * B + b) * P);
        float m = -INFINITY, s = 0.0f, e = 0.0f;
        for (int i = lane; i < P; i += 32) {
            const float4 o = piece[i];                      // m, n, s, e
            if (!(o.x > -INFINITY)) continue;
            if (o.x > m) {
                const float f = exp_neg(m - o.x);           // (m = -inf: zero)
                s *= f, e *= f, m = o.x;
            }
            const float f = exp_neg(o.x - m), p = __fmul_rn(o.z, f);
            pair_add(s, e, p, __fmaf_rn(o.z, f, -p) + o.w * f);
        }
        float all = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kFull, all, o));
        if (m > -INFINITY) {
            const float f = exp_neg(m - all), p = __fmul_rn(s, f);
            e = __fmaf_rn(s, f, -p) + e * f, s = p;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) pair_add(s, e, __shfl_xor_sync(kFull, s, o), __shfl_xor_sync(kFull, e, o));
        if (lane == 0) {
            float h = 0.0f, c = 0.0f, a, d;                 // (a row without a value has no candidate)
            if (s > 0.0f) pair_log(s, e, h, c);
            two_sum(all > -INFINITY ? all : 0.0f, h, a, d);
            s_lh[b] = a, s_ll[b] = __fadd_rn(d, c);
            s_cum[b] = scores[g * B + b];
        }
    }
    __syncthreads();
    int got;                                                // candidates
    if (few) {
        const int n = lists * k, n4 = (n + 3) & ~3, from = threadIdx.x / k, of = from / P, j = threadIdx.x - from * k;
        uint32_t *hi = s_keys, *lo = hi + n4;               // (the upper halves padded with zeros)
        const bool in = (int)threadIdx.x < n && j < s_len[from];
        const uint64_t y = in ? score_key(s_cum[of], own.x, s_lh[of], s_ll[of]) : 0;
        if ((int)threadIdx.x < n4) hi[threadIdx.x] = (uint32_t)(y >> 32), lo[threadIdx.x] = (uint32_t)y;
        float *token = reinterpret_cast<float *>(lo + n4);
        if ((int)threadIdx.x < n) token[threadIdx.x] = own.y;
        got = min(__syncthreads_count(in), k);
        const int i = threadIdx.x >> 2, at = min(i, n4 - 1);
        const int rank = rank_below(hi, lo, n, n4, at, k, [](int a) { return (uint32_t)a; });
        if (i < n && rank < k && (threadIdx.x & 3) == 0) s_score[rank] = from_ordered(hi[i]), s_row[rank] = i / k / P, s_token[rank] = __float_as_int(token[i]);
    } else {
        const int n4 = join_heads(lists, k);
        int left = lists, n = INT32_MAX;
        uint32_t *buffers = s_keys + 2 * n4;
        if (n4 != 0) {
            uint32_t *hi = s_keys, *lo = hi + n4;
#pragma unroll
            for (int i = 0; i < kMaxLists / kJoinThreads; ++i) {
                const int l = threadIdx.x + i * kJoinThreads, of = l < lists ? l / P : 0;
                const uint64_t key = l < lists && s_len[l] > 0 ? score_key(s_cum[of], head[i], s_lh[of], s_ll[of]) : 0;
                if (l < n4) hi[l] = (uint32_t)(key >> 32), lo[l] = (uint32_t)key;
            }
            __syncthreads();
            for (int i = threadIdx.x >> 2; i < (n4 + 7 & ~7); i += kJoinThreads / 4) {   // (whole warps: eight items)
                const int at = min(i, n4 - 1);
                const int rank = rank_below(hi, lo, n4, n4, at, k, [](int a) { return (uint32_t)a; });
                if (i >= lists || rank >= k || (threadIdx.x & 3) != 0) continue;
                s_list[atomicAdd(&s_lists, 1)] = i;
                atomicOr(&s_take[i / 32], 1u << i % 32);
                if (rank == k - 1) s_bar[0] = hi[i], s_bar[1] = lo[i], s_bar[2] = (uint32_t)i;
            }
            __syncthreads();
            left = s_lists;
            // the k-th head, where there are as many
            const uint64_t bar = left == k ? ((uint64_t)s_bar[0] << 32) | s_bar[1] : 0;
            const int at_bar = left == k ? (int)s_bar[2] : lists;
            uint32_t *ehi = buffers, *elo = ehi + kJoinRanked, *etoken = elo + kJoinRanked, *eplace = etoken + kJoinRanked;     // (place: list, and where in it)
            for (int i = warp; i < left; i += warps) {
                const int from = s_list[i], of = from / P;
                for (int j = lane; j < s_len[from]; j += 32) {
                    const float2 x = list[from * k + j];
                    const uint64_t y = score_key(s_cum[of], x.x, s_lh[of], s_ll[of]);
                    // (of equal scores all that lie in lists up to the bar's: of its own, k at most)
                    if ((y > bar) | ((y == bar) & (from <= at_bar))) {
                        const int c = atomicAdd(&s_n, 1);
                        if (c < kJoinRanked) ehi[c] = (uint32_t)(y >> 32), elo[c] = (uint32_t)y, etoken[c] = __float_as_uint(x.y), eplace[c] = from * kMaxCand + j;
                    }
                }
            }
            __syncthreads();
            n = s_n;
            if (n <= kJoinRanked) {
                const int e4 = (n + 3) & ~3;
                if (threadIdx.x < e4 - n) ehi[n + threadIdx.x] = 0;
                __syncthreads();
                for (int i = threadIdx.x >> 2; i < (e4 + 7 & ~7); i += kJoinThreads / 4) {
                    const int rank = rank_below(ehi, elo, n, e4, min(i, e4 - 1), k, [&](int a) { return eplace[a]; });
                    if (i < n && rank < k && (threadIdx.x & 3) == 0)
                        s_score[rank] = from_ordered(ehi[i]), s_row[rank] = (int)(eplace[i] / kMaxCand) / P, s_token[rank] = (int)etoken[i];
                }
                got = min(n, k);
            } else {                                        // the lists in their order (the buffers lie where the entries were)
                for (int l = threadIdx.x; l < lists; l += kJoinThreads)
                    if (s_take[l / 32] >> l % 32 & 1) {
                        int at = __popc(s_take[l / 32] & ((1u << l % 32) - 1));
                        for (int w = 0; w < l / 32; ++w) at += __popc(s_take[w]);
                        s_list[at] = l;
                    }
                __syncthreads();
            }
        }
        if (n > kJoinRanked)
            got = join_merge(buffers, min(k, lists) * k, left, k, P, [&](int q) { return n4 != 0 ? s_list[q] : q; }, list, s_len, s_cum, s_lh, s_ll, s_score, s_row, s_token);
    }
    __syncthreads();
    if (warp != 0) return;
    int live = 0;                                           // candidates so far that do not end
    for (int i = lane; i < k + lane; i += 32) {             // (all lanes as often)
        const bool in = i < got;
        const float score = in ? s_score[i] : -INFINITY;
        const int row = in ? (int)(g * B) + s_row[i] : -1, token = in ? s_token[i] : -1;
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
    const int64_t most = kMaxLists / B;                     // lists of a group: up to two a thread of the join
    int64_t n = 3 * sm_count() / rows;                      // one wave of blocks, three to an SM (128 rows: 22.3 us, with 2 25.1, 4 26.6, 6 25.5)
    // (where that whole number changes, rows of 50000 bf16 logits, two candidates a beam: 152 rows, three pieces each, 14.1 us; 228, two, 14.3; 229, one, 16.8; 300 18.3; 456 18.0; 457, a
    // second wave, 23.8)
    if (n > all) n = all;
    if (n < 1) n = 1;
    if (n > most) n = most;
    ws->pieces = (int)n;
    ws->length = ((V + 7 + n - 1) / n + 7) / 8 * 8;
}

template <typename T>
int launch_scan(const void *logits, int64_t stride, int64_t V, const float *scores, int k, const BeamWs &ws, int64_t blocks, int slot, cudaStream_t s) {
    constexpr int stages = kStages * kTile * (int)sizeof(T);
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(beam_scan_kernel<T>), stages, slot);
    if (rc != MQ_OK) return rc;
    return cuda_error(launch_pdl(beam_scan_kernel<T>, dim3((unsigned)blocks), dim3(kScanThreads), stages, s, static_cast<const T *>(logits), stride, V, scores, k, ws),
                      "mqd_beam_select launch");
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
    int rc = dtype == MQD_F32   ? launch_scan<float>(logits, stride, V, scores, k, ws, n, kAttrSlotBeam, s)
             : dtype == MQD_F16 ? launch_scan<__half>(logits, stride, V, scores, k, ws, n, kAttrSlotBeam + 1, s)
                                : launch_scan<__nv_bfloat16>(logits, stride, V, scores, k, ws, n, kAttrSlotBeam + 2, s);
    if (rc != MQ_OK) return rc;
    const int lists = B * ws.pieces, words = join_words(lists, k);
    rc = ensure_smem_attr(reinterpret_cast<const void *>(beam_join_kernel), (2 * kMaxLists + 6 * kMaxCand * kMaxCand + 4) * 4, kAttrSlotBeam + 3);
    if (rc != MQ_OK) return rc;
    const cudaError_t e = launch_pdl(beam_join_kernel, dim3((unsigned)n_groups), dim3(kJoinThreads), words * 4, s, ws, B, scores, k, stop, cand_score, cand_row,
                                     cand_token, next_score, next_row, next_token);
    return cuda_error(e, "mqd_beam_select launch");
}

}  // namespace mq

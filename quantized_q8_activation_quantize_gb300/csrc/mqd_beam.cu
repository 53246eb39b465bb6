// mqd_beam.cu -- one step of beam search: the best continuations over beams and vocabulary.
//
//   score(b, t) = s_b + x_bt - ln sum_t' exp(x_bt')
//
// Two kernels.  The scan reads the logits once: a block takes a piece of a row, keeps the sum of exponentials relative to the largest value met
// (online: a thread rescales its sum when a tile brings a larger one) and, beside it, the piece's best n_cand values, found by a threshold
// that only few values pass.  The join has a block per group: the rows' sums, then n_cand times the best of all lists' heads.
// Within a row the order of the scores is that of the logits, so only the join needs the sums; it compares f32 pairs, 48 bits.
#include <cfloat>

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
// exp(x) for x <= 0: x log2(e) with the constant in two parts
__device__ __forceinline__ float exp_neg(float x) { return ex2(__fmaf_rn(x, 1.442695f, __fmul_rn(x, 1.925963e-8f))); }

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

// values of a tile in registers, -inf where there is none; vectors of 16 bytes from the boundary at or before the row's beginning (bytes of
// a vector that holds a value of the row lie in that value's 16-byte granule, so no read leaves memory)
template <typename T>
__device__ __forceinline__ void load_tile(const T *base, int64_t first, int64_t end, int64_t e0, float (&x)[kScanPer]) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < kScanPer / V; ++j) {
        const int64_t e = e0 + ((int64_t)j * kScanThreads + threadIdx.x) * V;
        if (e + V > first && e < end) {
            if constexpr (V == 4) {
                const float4 w = __ldcs(reinterpret_cast<const float4 *>(base + e));
                x[4 * j] = w.x, x[4 * j + 1] = w.y, x[4 * j + 2] = w.z, x[4 * j + 3] = w.w;
            } else {
                float v[8];
                unpack8(Raw8<T>{__ldcs(reinterpret_cast<const uint4 *>(base + e))}, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[8 * j + i] = v[i];
            }
            if (e < first || e + V > end) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e + i < first || e + i >= end) x[V * j + i] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[V * j + i] = -INFINITY;
        }
    }
}

// the best k of the n entries in s_buf, sorted, to its front; returns how many.  A thread counts what is better than its entry: n^2 / 256 steps a thread,
// for a few dozen entries
__device__ __forceinline__ int keep_best(float2 *s_buf, float2 *s_best, int n, int k) {
    for (int i = threadIdx.x; i < n; i += kScanThreads) {
        const float2 a = s_buf[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
            const float2 b = s_buf[j];
            rank += b.x > a.x || (b.x == a.x && __float_as_int(b.y) < __float_as_int(a.y));
        }
        if (rank < k) s_best[rank] = a;
    }
    __syncthreads();
    n = min(n, k);
    if (threadIdx.x < n) s_buf[threadIdx.x] = s_best[threadIdx.x];
    __syncthreads();
    return n;
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads, 4) beam_scan_kernel(const T *logits, int64_t stride, int64_t V, const float *scores, int k, BeamWs ws) {
    constexpr int VEC = 16 / sizeof(T);
    __shared__ float2 s_buf[kTile + kBuffer];
    __shared__ float2 s_best[kMaxCand];
    __shared__ uint2 s_key[kScanThreads / 32];
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
    const int shift = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    const T *base = p - shift;
    const int64_t first = shift, end = shift + V;
    const int64_t e0 = piece * ws.length, stop = min(end, e0 + ws.length);
    if (threadIdx.x == 0) s_n = 0;
    float m = -INFINITY, s = 0.0f, thr = -INFINITY;
    int have = 0;
    bool sorted = true;
    float x[kScanPer];
    load_tile(base, first, stop, e0, x);
#pragma unroll 1
    for (int64_t at = e0; at < stop; at += kTile) {
        float v[kScanPer], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) {
            v[i] = fminf(fmaxf(x[i], -INFINITY), FLT_MAX);  // (a NaN gives way to -inf)
            top = fmaxf(top, v[i]);
        }
        if (at + kTile < stop) load_tile(base, first, stop, at + kTile, x);
        if (top > -INFINITY) {
            if (top > m) {
                s *= exp_neg(m - top);                      // (m = -inf: zero)
                m = top;
            }
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int i = 0; i < kScanPer; i += 2) a += exp_neg(v[i] - m), b += exp_neg(v[i + 1] - m);
            s += a + b;
        }
        const int from = (int)(at - first);                 // token of the tile's first place
        auto token = [&](int i) { return from + ((i / VEC) * kScanThreads + (int)threadIdx.x) * VEC + i % VEC; };
        float bar = thr;                                    // what passes: > bar, or = bar up to token last
        int last = INT32_MIN;
        if (at == e0) {
            // every warp's ceil(k / 8)-th largest of its threads' largest values: at least k values are not below the least of these
            int at_top = INT32_MAX;
#pragma unroll
            for (int i = kScanPer - 1; i >= 0; --i)
                if (v[i] == top) at_top = token(i);
            const uint32_t own = top > -INFINITY ? ordered(top + 0.0f) : 0u;
            uint32_t key = own, best = 0, who = 0;
            for (int j = 0; j < (k + 7) / 8; ++j) {
                best = __reduce_max_sync(kFull, key);
                who = __reduce_min_sync(kFull, key == best ? (uint32_t)at_top : 0xffffffffu);
                if (key == best && (uint32_t)at_top == who) key = 0;
            }
            if (lane == 0) s_key[warp] = make_uint2(best, who);
            __syncthreads();
            uint2 least = s_key[0];
#pragma unroll
            for (int w = 1; w < kScanThreads / 32; ++w) {
                const uint2 o = s_key[w];
                if (o.x < least.x || (o.x == least.x && o.y > least.y)) least = o;
            }
            if (least.x == 0) {
                // a warp has too few values (the end of a row, a mask): the k-th largest of all threads' largest
                uint2 *s_all = reinterpret_cast<uint2 *>(s_buf);
                s_all[threadIdx.x] = make_uint2(own, (uint32_t)at_top);
                __syncthreads();
                int rank = 0;
#pragma unroll 8
                for (int j = 0; j < kScanThreads; ++j) {
                    const uint2 o = s_all[j];
                    rank += o.x > own || (o.x == own && o.y < (uint32_t)at_top);
                }
                if (own != 0 && rank == k - 1) s_key[0] = make_uint2(own, (uint32_t)at_top);
                least = make_uint2(0, 0);
                if (__syncthreads_or(own != 0 && rank == k - 1)) least = s_key[0];
            }
            if (least.x != 0) bar = from_ordered(least.x), last = (int)least.y;
        }
        bool hit = false;
        if (top >= bar && top > -INFINITY) {
#pragma unroll
            for (int i = 0; i < kScanPer; ++i)
                if (v[i] > bar || (v[i] == bar && token(i) <= last)) {
                    s_buf[atomicAdd(&s_n, 1)] = make_float2(v[i], __int_as_float(token(i)));
                    hit = true;
                }
        }
        if (__syncthreads_or(hit)) {
            const int n = s_n;
            __syncthreads();                                // (all have read it before anyone adds to it)
            if (at == e0 || n > kBuffer) {
                have = keep_best(s_buf, s_best, n, k);
                sorted = true;
                if (threadIdx.x == 0) s_n = have;
                if (have == k) thr = s_buf[k - 1].x;
                __syncthreads();
            } else {
                have = n, sorted = false;
            }
        }
    }
    if (!sorted) have = keep_best(s_buf, s_best, have, k);
    for (int i = threadIdx.x; i < have; i += kScanThreads) ws.list[(int64_t)blockIdx.x * k + i] = s_buf[i];
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (m > -INFINITY) s *= exp_neg(m - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) s_m[warp] = top, s_s[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        float all = s_m[0];
#pragma unroll
        for (int w = 1; w < kScanThreads / 32; ++w) all = fmaxf(all, s_m[w]);
        float sum = 0.0f, rest = 0.0f;
#pragma unroll
        for (int w = 0; w < kScanThreads / 32; ++w)
            if (s_m[w] > -INFINITY) pair_add(sum, rest, s_s[w] * exp_neg(s_m[w] - all), 0.0f);
        *out = {all, have, sum, rest};
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

// a candidate of a group: its score as an f32 pair (hi the rounded sum, lo the rest: 48 bits), both in the order of unsigned integers (hi 0: none); beam, token
struct Cand {
    uint32_t hi, lo, beam, token;
};
__device__ __forceinline__ Cand make_cand(float cum, float x, float lh, float ll, uint32_t beam, uint32_t token) {
    float d, e, h, l;
    two_sum(x, -lh, d, e);                                      // (|x| and the logarithm may be far apart either way)
    e = __fsub_rn(e, ll);
    two_sum(cum, d, h, l);
    l = fabsf(h) <= FLT_MAX ? __fadd_rn(l, e) : 0.0f;           // (past f32 there is no rest)
    const float s = __fadd_rn(h, l);
    l = __fsub_rn(l, __fsub_rn(s, h));
    return {ordered(s + 0.0f), ordered(fabsf(h) <= FLT_MAX ? l + 0.0f : 0.0f), beam, token};
}
// whether this lane's is the best of the warp's (false everywhere: there is none left)
__device__ __forceinline__ bool best_of_warp(const Cand &c, bool &none) {
    const uint32_t hi = __reduce_max_sync(kFull, c.hi);
    none = hi == 0;
    bool mine = !none && c.hi == hi;
    const uint32_t lo = __reduce_max_sync(kFull, mine ? c.lo : 0u);
    mine = mine && c.lo == lo;
    if (__popc(__ballot_sync(kFull, mine)) > 1) {           // equal scores: the lowest beam, then the lowest token
        const uint32_t b = __reduce_min_sync(kFull, mine ? c.beam : 0xffffffffu);
        mine = mine && c.beam == b;
        const uint32_t t = __reduce_min_sync(kFull, mine ? c.token : 0xffffffffu);
        mine = mine && c.token == t;
    }
    return mine;
}

constexpr int kJoinWarps = 32;

__global__ void __launch_bounds__(kJoinWarps * 32) beam_join_kernel(BeamWs ws, int B, const float *scores, int k, int stop, float *cand_score_out,
                                                                    int32_t *cand_row, int32_t *cand_token, float *next_score, int32_t *next_row,
                                                                    int32_t *next_token) {
    __shared__ Cand s_list[kJoinWarps][kMaxCand];
    __shared__ int s_n[kJoinWarps];
    __shared__ float s_cum[kMaxCand], s_lh[kMaxCand], s_ll[kMaxCand];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t g = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = ws.pieces;
    for (int b = warp; b < B; b += kJoinWarps) {            // a warp per row: its sum of exponentials
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
            float h = 0.0f, l = 0.0f, a, c;                     // (a row without a value has no candidate)
            if (s > 0.0f) pair_log(s, e, h, l);
            two_sum(m > -INFINITY ? m : 0.0f, h, a, c);
            s_lh[b] = a, s_ll[b] = __fadd_rn(c, l);
            s_cum[b] = scores[g * B + b];
        }
    }
    __syncthreads();
    // a list per thread (neighbours of a row in different warps); every warp takes the best k of its lists
    const int l = lane * kJoinWarps + warp, lists = B * P;
    const int beam = l < lists ? l / P : 0;
    const float2 *list = ws.list + (g * lists + (l < lists ? l : 0)) * k;
    const int n = l < lists ? ws.piece[g * lists + l].n : 0;
    const float cum = s_cum[beam], lh = s_lh[beam], ll = s_ll[beam];
    int pos = 0;
    float2 ahead = n > 1 ? list[1] : make_float2(0.f, 0.f);
    Cand c = {0, 0, 0, 0};
    if (n > 0) c = make_cand(cum, list[0].x, lh, ll, beam, __float_as_uint(list[0].y));
    int got = 0;
    for (; got < k; ++got) {
        bool none;
        const bool mine = best_of_warp(c, none);
        if (none) break;
        if (mine) {
            s_list[warp][got] = c;
            ++pos;
            c = {0, 0, 0, 0};
            if (pos < n) c = make_cand(cum, ahead.x, lh, ll, beam, __float_as_uint(ahead.y));
            if (pos + 1 < n) ahead = list[pos + 1];
        }
    }
    if (lane == 0) s_n[warp] = got;
    __syncthreads();
    if (warp != 0) return;
    // the best k of the warps' lists, one lane each
    const int mine_n = s_n[lane];
    pos = 0;
    c = {0, 0, 0, 0};
    if (mine_n > 0) c = s_list[lane][0];
    int live = 0;                                           // candidates so far that do not end
    for (int i = 0; i < k; ++i) {
        bool none;
        const bool mine = best_of_warp(c, none);
        const int who = none ? 0 : __ffs(__ballot_sync(kFull, mine)) - 1;
        const Cand w = {__shfl_sync(kFull, c.hi, who), __shfl_sync(kFull, c.lo, who), __shfl_sync(kFull, c.beam, who), __shfl_sync(kFull, c.token, who)};
        const float score = none ? -INFINITY : from_ordered(w.hi);
        const int row = none ? -1 : (int)(g * B + w.beam), token = none ? -1 : (int)w.token;
        if (lane == 0) {
            cand_score_out[g * k + i] = score;
            cand_row[g * k + i] = row;
            cand_token[g * k + i] = token;
        }
        if (!none && token != stop && live < B) {
            if (lane == 0 && next_row != nullptr) {
                next_score[g * B + live] = score;
                next_row[g * B + live] = row;
                next_token[g * B + live] = token;
            }
            ++live;
        }
        if (mine && !none) c = ++pos < mine_n ? s_list[lane][pos] : Cand{0, 0, 0, 0};
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
    int64_t n = (6 * sm_count() + rows - 1) / rows;
    if (n > all) n = all;
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
    if (e == cudaSuccess)
        e = launch_pdl(beam_join_kernel, dim3((unsigned)n_groups), dim3(kJoinWarps * 32), 0, s, ws, B, scores, k, stop, cand_score, cand_row, cand_token,
                       next_score, next_row, next_token);
    return cuda_error(e, "mqd_beam_select launch");
}

}  // namespace mq

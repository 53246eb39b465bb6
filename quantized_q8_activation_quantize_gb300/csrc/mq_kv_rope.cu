// mq_kv_rope.cu -- what a layer does between its q | k | v projections and its attention: the queries turned, the keys turned and quantized into their pages
// with the values.
//
// Small calls are one launch: the grid's first blocks take the queries (a few tokens of all heads each, mqd_rope.cuh), the others the keys and values.  Large ones
// are two, since the queries need half the registers (five blocks an SM; 38376 tokens of 32 heads beside the append and the read 207 us, with four 209, with six 218).  The keys are turned in f32 and never rounded before their codes.
#include <cfloat>
#include <type_traits>

#include "mqd_rope.cuh"

namespace mq {
namespace {

constexpr int kTurnThreads = kRopeThreads, kTurnWarps = 4;      // warps of a vector: 8 slots each, two vectors at a time

// Stages of the ring that keys and values pass, one asked for while the other is worked on, and their bytes.  40960 tokens of 8 heads: bf16 67 us, three stages
// 68, four 70, six 81 (what the ring takes the L1 lacks); f32 78, three stages 110.  The next pair in registers: 86 and 102.
constexpr int kTurnStages = 2;
template <typename T, int D>
constexpr int kTurnStage = kKB * D * 2 * (int)sizeof(T);
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from, bool full) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(full ? BYTES : 0) : "memory");
}

struct TurnedRows {
    const void *k, *v;
    int64_t kt, kh, vt, vh;
    int32_t each;               // pairs of vectors of a block
};

// One block of 32 slots of a sequence and `each` pairs of its 2 H vectors (half, head), from pair y0 on: the angles once for all heads, then two vectors at a time, four
// warps each, all of a lane's values in registers between the maximum and the codes, the next vectors on their way into shared memory.  Bound by latency at 16 warps
// an SM (17 instructions a value in 54 % of the issue slots, a quarter of the warps): 40960 tokens of 8 heads of 128 take 67 us from bf16 (3.7 TB/s) and 78 from f32 (5.4 TB/s).
// Before the ring took the loads off its path, one vector at a time by eight warps, half the registers, took 91 and 105 for 86 and 102.  A lane holds two quads of a row that
// are turned with one another (quads j and j + half / 4, or neighbours), so that a turn needs no exchange.  Unit u belongs to the last sequence b with U(b) <= u,
// U(b) = begin(b) / 32 + 2 b, as in mqkv_append, whose arithmetic this is.
template <typename T, int D>
__device__ __forceinline__ void append_turned(const KvView &c, const KvRows &rows, int64_t u, int y0, const RopePlan &plan, const int32_t *pos, const TurnedRows &in,
                                              float *s_cos, float *s_sin, uint8_t *s_ring, unsigned int *err) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, IT = kKB / kTurnWarps / RPW;     // lanes per row, rows per warp and step, steps
    __shared__ float s_amax[2][8];
    int b;
    int64_t u0;
    if (rows.cu == nullptr) {
        const int64_t per = rows.each / kKB + 2;
        b = (int)(u / per);
        u0 = b * per;
        if (b >= c.n_seqs) return;
    } else {
        b = kv_find_seq(rows, c.n_seqs, u, 2, 5);
        u0 = rows.begin(b) / kKB + 2 * (int64_t)b;
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
    const int64_t p0 = len - n, s0 = (p0 / kKB + (u - u0)) * kKB;
    if (s0 >= len) return;
    const int new0 = (int)max(p0 - s0, (int64_t)0), new1 = (int)min(len - s0, (int64_t)kKB), fresh = new1 - new0;  // slots of new tokens
    const int page = c.table[(int64_t)b * c.max_pages + (s0 >> c.tshift)];
    const bool there = page >= 0 && page < c.n_pages, ours = there && (c.refs == nullptr || c.refs[page] == 1);
    if (!ours) {
        if (threadIdx.x == 0) kv_error(err, there ? KV_ERR_SHARED : KV_ERR_PAGE);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LPR, team = warp / kTurnWarps;
    const int r0 = kKB / kTurnWarps * (warp % kTurnWarps) + lane / LPR;         // this lane's first slot
    const int slot0 = (int)(s0 & (c.T - 1)), quads = plan.half / 4;
    uint8_t *slab = c.pool + (int64_t)page * c.page_bytes;
    const int64_t row0 = lo + s0 - p0;                                          // row of slot 0
    const int y1 = min(y0 + in.each, c.H);

    const bool whole = fresh == kKB;                                            // nearly always, in a large call
    // the two quads of a lane (in values), of a turned key and of another vector
    const bool turns = j < quads;
    const int ka = plan.interleaved ? 8 * j : turns ? 4 * j : 2 * plan.half + 8 * (j - quads), kz = !plan.interleaved && turns ? ka + plan.half : ka + 4;

    // the vectors of pair y on their way into this thread's own slots of a stage of shared memory (so no barriers); zeros where a slot has no new token
    uint8_t *stage = s_ring + threadIdx.x * sizeof(Raw4<T>);
    auto ask = [&](int y, int s) {
        const int vec = 2 * y + team, half = vec >= c.H, h = vec - half * c.H, a = half ? 8 * j : ka, z = half ? 8 * j + 4 : kz;
        const int64_t st = half ? in.vt : in.kt, step = RPW * st;
        const T *src = static_cast<const T *>(half ? in.v : in.k) + h * (half ? in.vh : in.kh) + (row0 + r0) * st;
        uint32_t to = smem_u32(stage + s * kTurnStage<T, D>);
#pragma unroll
        for (int i = 0; i < IT; ++i, src += step, to += 2 * kTurnThreads * sizeof(Raw4<T>)) {
            const bool in_it = whole || (r0 + i * RPW >= new0 && r0 + i * RPW < new1);
            const T *from = in_it ? src : static_cast<const T *>(in.k);
            copy_async<sizeof(Raw4<T>)>(to, from + a, in_it);
            copy_async<sizeof(Raw4<T>)>(to + kTurnThreads * sizeof(Raw4<T>), from + z, in_it);
        }
    };
    ask(y0, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (2 * y0 < c.H) {
        for (int i = threadIdx.x; i < fresh * plan.half; i += kTurnThreads) {
            const int slot = i / plan.half;
            const int64_t p = s0 + new0 + slot;
            const float2 cs = rope_cos_sin(pos != nullptr ? pos[row0 + new0 + slot] : (int32_t)p, plan.turns[i - slot * plan.half], plan.amplitude);
            s_cos[i] = cs.x, s_sin[i] = cs.y;
        }
        __syncthreads();
    }
    int slot = 0;
#pragma unroll 1
    for (int y = y0; y < y1; ++y) {
        const int vec = 2 * y + team, half = vec >= c.H, a = half ? 8 * j : ka, z = half ? 8 * j + 4 : kz;
        if (y + 1 < y1) ask(y + 1, 1 - slot);                                   // (the stage that was read last)
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group %0;" ::"n"(kTurnStages - 1) : "memory");
        float x[IT][8];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const Raw4<T> *raw = reinterpret_cast<const Raw4<T> *>(stage + slot * kTurnStage<T, D>) + i * 2 * kTurnThreads;
            unpack4(raw[0], x[i]), unpack4(raw[kTurnThreads], x[i] + 4);
        }
        slot = 1 - slot;
        uint8_t *codes = slab + (int64_t)vec * c.T * D + (int64_t)slot0 * D;    // (K of every head, then V of every head)
        float *scale = reinterpret_cast<float *>(slab + c.off_s) + vec * (c.T / kKB) + slot0 / kKB;
        float d_old = new0 > 0 ? *scale : 0.0f;                                 // slots of earlier tokens share the block
        if (!(d_old >= 0.0f && d_old <= FLT_MAX)) d_old = 0.0f;
        if (!half && turns) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int at = min(max(r0 + i * RPW - new0, 0), fresh - 1) * plan.half + 4 * j;         // (rows of no new token are zeros)
                const float4 co = *reinterpret_cast<const float4 *>(s_cos + at), si = *reinterpret_cast<const float4 *>(s_sin + at);
                float(&w)[8] = x[i];
                if (plan.interleaved) {
                    f2_unpack(rope_turn_pair(co.x, si.x, f2_pack(w[0], w[1])), w[0], w[1]);
                    f2_unpack(rope_turn_pair(co.y, si.y, f2_pack(w[2], w[3])), w[2], w[3]);
                    f2_unpack(rope_turn_pair(co.z, si.z, f2_pack(w[4], w[5])), w[4], w[5]);
                    f2_unpack(rope_turn_pair(co.w, si.w, f2_pack(w[6], w[7])), w[6], w[7]);
                } else {
                    uint64_t ua = f2_pack(w[0], w[1]), ub = f2_pack(w[2], w[3]), va = f2_pack(w[4], w[5]), vb = f2_pack(w[6], w[7]);
                    rope_turn2(f2_pack(co.x, co.y), f2_pack(si.x, si.y), f2_pack(-si.x, -si.y), ua, va);
                    rope_turn2(f2_pack(co.z, co.w), f2_pack(si.z, si.w), f2_pack(-si.z, -si.w), ub, vb);
                    f2_unpack(ua, w[0], w[1]), f2_unpack(ub, w[2], w[3]), f2_unpack(va, w[4], w[5]), f2_unpack(vb, w[6], w[7]);
                }
            }
        }
        float amax = 0.0f;
        uint64_t bad = f2_pack(0.0f, 0.0f);                                     // NaN where a value is not finite
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                amax = fmaxf(amax, fmaxf(fabsf(x[i][e]), fabsf(x[i][e + 1])));
                bad = f2_fma(f2_pack(x[i][e], x[i][e + 1]), f2_pack(0.0f, 0.0f), bad);
            }
        float bad0, bad1;
        f2_unpack(bad, bad0, bad1);
        const bool finite = bad0 + bad1 == 0.0f;
        if (!finite) {                                                          // (rare) again, infinities aside
            amax = 0.0f;
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[i][e]) <= FLT_MAX ? fabsf(x[i][e]) : 0.0f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) s_amax[y & 1][warp] = amax;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kTurnWarps) : "memory");
        const float *others = s_amax[y & 1] + team * kTurnWarps;
        float d = __fmul_rn(fmaxf(fmaxf(others[0], others[1]), fmaxf(others[2], others[3])), 1.0f / 127.0f);
        if (d < FLT_MIN) d = 0.0f;
        d = fmaxf(d, d_old);
        const float id = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        const uint64_t f = f2_pack(id, id);
        if (!finite) {                                                          // NaN is zero, an infinity the end of the range
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] == x[i][e] ? fminf(fmaxf(x[i][e], -127.0f * d), 127.0f * d) : 0.0f;
        }
        uint8_t *dst = codes + r0 * D;
#pragma unroll
        for (int i = 0; i < IT; ++i, dst += RPW * D) {
            float(&w)[8] = x[i];
            if (whole || (r0 + i * RPW >= new0 && r0 + i * RPW < new1)) {
                *reinterpret_cast<uint32_t *>(dst + a) = pack_codes(f2_mul(f2_pack(w[0], w[1]), f), f2_mul(f2_pack(w[2], w[3]), f));
                *reinterpret_cast<uint32_t *>(dst + z) = pack_codes(f2_mul(f2_pack(w[4], w[5]), f), f2_mul(f2_pack(w[6], w[7]), f));
            }
        }
        if (new0 > 0 && d > d_old) {                                            // earlier codes under a larger scale
            const float shrink = __fdiv_rn(d_old, d);
#pragma unroll 1
            for (int i = 0; i < 2 * IT; ++i) {
                const int r = r0 + (i >> 1) * RPW;
                if (r >= new0) continue;
                uint32_t *dst = reinterpret_cast<uint32_t *>(codes + r * D + (i & 1 ? z : a));
                const uint32_t old = *dst;
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = __fmul_rn(code_value(old, e), shrink);
                *dst = pack_codes(f2_pack(w[0], w[1]), f2_pack(w[2], w[3]));
            }
        }
        if (warp % kTurnWarps == 0 && lane == 0) *scale = d;
    }
}

// position and kind (rope_block's live) of the n tokens from t0 on, by one warp: 0 where a token belongs to no sequence, 2 where its sequence has
// a bad length (the append's blocks report it)
__device__ __forceinline__ void find_tokens(const KvView &c, const KvRows &rows, const int32_t *pos, int64_t t0, int n, int *s_pos, int *s_live) {
    const int lane = threadIdx.x & 31;
    int b = rows.cu == nullptr ? (int)(t0 / rows.each) : kv_find_seq(rows, c.n_seqs, t0, 0, 0);
    if (lane >= n) return;
    const int64_t t = t0 + lane;
    if (rows.cu == nullptr) b = (int)(t / rows.each);
    else
        while (b + 1 < c.n_seqs && rows.begin(b + 1) <= t) ++b;
    int64_t lo, hi;
    rows.of(b, lo, hi);
    const int64_t len = c.len[b];
    const bool bad = len < hi - lo || ((len - 1) >> c.tshift) >= c.max_pages;
    s_live[lane] = t < lo || t >= hi ? 0 : bad ? 2 : 1;
    s_pos[lane] = pos != nullptr ? pos[t] : (int32_t)(len - (hi - lo) + (t - lo));
}

constexpr int kRopeTokens = 4;          // at most, per block of queries

template <typename T, int W>
__device__ __forceinline__ void rope_rows(const KvView &c, const KvRows &rows, const RopePlan &plan, const int32_t *pos, const RopeRows &q, int64_t block,
                                          float *s_cos, float *s_sin) {
    __shared__ int s_pos[kRopeTokens], s_live[kRopeTokens];
    const int64_t t0 = block * q.per_block;
    const int n = (int)min((int64_t)q.per_block, q.n_tokens - t0);
    if (threadIdx.x < 32) find_tokens(c, rows, pos, t0, n, s_pos, s_live);
    __syncthreads();
    bool zeros = false;
    for (int i = 0; i < n; ++i) zeros = zeros || s_live[i] == 2;
    rope_block<T, W>(plan, q, t0, n, s_cos, s_sin, [&](int t) { return s_pos[t]; }, [&](int t) { return s_live[t]; }, zeros);
}

template <typename T, int W>
__global__ void __launch_bounds__(kRopeThreads, 5) kv_rope_rows_kernel(KvView c, KvRows rows, RopePlan plan, const int32_t *pos, RopeRows q) {
    __shared__ __align__(16) float s_cos[kRopePairs], s_sin[kRopePairs];
    grid_dep_launch();
    grid_dep_wait();
    rope_rows<T, W>(c, rows, plan, pos, q, blockIdx.x, s_cos, s_sin);
}

// (three blocks an SM spill: 75 us for 68 from bf16)
template <typename T, int W, int D>
__global__ void __launch_bounds__(kTurnThreads, 2) kv_append_rope_kernel(KvView c, KvRows rows, int gy, RopePlan plan, const int32_t *pos, RopeRows q,
                                                                                             unsigned q_blocks, TurnedRows in, unsigned int *err) {
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ __align__(16) float s_cos[kKB * D / 2], s_sin[kKB * D / 2];      // (kRopeTokens * D / 2 at most for queries)
    grid_dep_launch();
    grid_dep_wait();
    if (blockIdx.x < q_blocks) {
        rope_rows<T, W>(c, rows, plan, pos, q, blockIdx.x, s_cos, s_sin);
        return;
    }
    const unsigned unit = blockIdx.x - q_blocks;
    append_turned<T, D>(c, rows, unit / gy, (int)(unit % gy) * in.each, plan, pos, in, s_cos, s_sin, s_ring, err);
}

template <typename T, int W>
int append_rope_t(const KvView &c, const KvRows &r, const RopePlan &plan, const int32_t *pos, const RopeRows &q, TurnedRows in, unsigned int *err, cudaStream_t s) {
    const int64_t q_all = q.x != nullptr ? (q.n_tokens + q.per_block - 1) / q.per_block : 0;
    // 28:4 heads of bf16, 1216 tokens in one launch 8.9 us, in two 11.4; 2432 16.2 and 15.7; 4864 30.0 and 26.6; 9728 56 and 46
    const bool apart = q_all > 4 * sm_count();
    const int64_t units = r.cu == nullptr ? c.n_seqs * (r.each / kKB + 2) : r.n_tokens / kKB + 2 * (int64_t)c.n_seqs;
    // As many pairs of vectors a block as leave one wave of blocks, two an SM; all where there is more than a wave (the angles are then computed once).  f32, 8
    // heads, with 1, 2, 4, 8 pairs a block: 1024 tokens 6.4 7.9 10.3 14.6 us, 2048 10.2 8.2 11.3 14.9, 4096 18.2 15.6 13.8 20.5, 16384 61 49 46 44; a token of 64
    // sequences 8.5 6.9 8.5 12.7.
    const int64_t about = r.n_tokens / kKB + c.n_seqs, fit = 2 * sm_count() / about;         // blocks of slots that hold a token, nearly
    in.each = fit > 1 ? (int)((c.H + fit - 1) / fit) : c.H;
    const int gy = (c.H + in.each - 1) / in.each;
    const int64_t q_blocks = apart ? 0 : q_all, blocks = q_blocks + units * gy;
    if (blocks > INT32_MAX) return set_error(MQ_ERR_SHAPE, "mqkv_append_rope: %lld blocks, below 2^31 wanted (fewer tokens a call)", (long long)blocks);
    if (apart) {
        const int rc = cuda_error(launch_pdl(kv_rope_rows_kernel<T, W>, dim3((unsigned)q_all), dim3(kRopeThreads), 0, s, c, r, plan, pos, q), "mqkv_append_rope launch");
        if (rc != MQ_OK) return rc;
    }
    auto fn = c.D == 128 ? kv_append_rope_kernel<T, W, 128> : kv_append_rope_kernel<T, W, 64>;
    const int smem = kTurnStages * (c.D == 128 ? kTurnStage<T, 128> : kTurnStage<T, 64>);
    const int slot = kAttrSlotRope + (sizeof(T) == 4 ? 0 : std::is_same_v<T, __half> ? 2 : 6) + (W == 8 ? 2 : 0) + (c.D == 128);
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(fn), smem, slot);
    if (rc != MQ_OK) return rc;
    return cuda_error(launch_pdl(fn, dim3((unsigned)blocks), dim3(kTurnThreads), smem, s, c, r, gy, plan, pos, q, (unsigned)q_blocks, in, err), "mqkv_append_rope launch");
}

}  // namespace

int kv_launch_append_rope(const KvView &c, const KvRows &r, int dtype, const RopePlan &plan, const int32_t *pos, const KvRopeRows &q, const void *k,
                          int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s) {
    RopeRows rows{q.x, q.out, q.xt, q.xh, q.ot, q.oh, r.n_tokens, q.heads, c.D, 1};
    if (q.heads > 0) rows.per_block = rope_tokens(plan, rows);
    const bool wide = rope_wide(plan, rows);
    auto fn = dtype == MQKV_F32   ? append_rope_t<float, 4>
              : dtype == MQKV_F16 ? (wide ? append_rope_t<__half, 8> : append_rope_t<__half, 4>)
                                  : (wide ? append_rope_t<__nv_bfloat16, 8> : append_rope_t<__nv_bfloat16, 4>);
    return fn(c, r, plan, pos, rows, TurnedRows{k, v, kt, kh, vt, vh, 1}, err, s);
}

}  // namespace mq

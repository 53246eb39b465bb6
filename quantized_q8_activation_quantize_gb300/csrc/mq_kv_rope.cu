// mq_kv_rope.cu -- one launch for what a layer does between its q | k | v projections and its attention: the queries turned, the keys
// turned and quantized into their pages with the values.
//
// The grid's first blocks take the queries (a few tokens of all heads each, mqd_rope.cuh), the others a unit of the append each
// (mq_kv_append.cuh); both are bound by HBM where there is much to do and by latency where there is little, so they run beside each other.  The keys are
// turned in f32 and never rounded before their codes.
#include "mq_kv_append.cuh"
#include "mqd_rope.cuh"

namespace mq {
namespace {

struct KeyRope {
    static constexpr bool on = true;
    RopePlan plan;
    const int32_t *pos;         // of the call's rows; nullptr: the cached positions
    float2 *s_cs;               // [new slots][half]
    __device__ __forceinline__ void table(const KvView &c, int64_t s0, int new0, int new1, int64_t row0, int y) const {
        if (y * kAppendVecs >= c.H) return;                                     // values only
        for (int i = threadIdx.x; i < (new1 - new0) * plan.half; i += kAppendThreads) {
            const int slot = i / plan.half;
            const int64_t p = s0 + new0 + slot;
            s_cs[i] = rope_cos_sin(pos != nullptr ? pos[row0 + p] : (int32_t)p, plan.turns[i - slot * plan.half], plan.amplitude);
        }
        __syncthreads();                                                        // (the last block's readers have passed append's own barrier)
    }
    __device__ __forceinline__ void turn(float (&x)[4], int slot, int slots, int quad, int base) const {
        const bool live = slot >= 0 && slot < slots;
        const float2 *cs = s_cs + (live ? slot : 0) * plan.half;
        if (plan.interleaved) {
            if (live && 2 * quad < plan.half) {
                rope_turn(cs[2 * quad], x[0], x[1]);
                rope_turn(cs[2 * quad + 1], x[2], x[3]);
            }
            return;
        }
        const int quads = plan.half / 4;                                        // of each half
        const bool first = quad < quads, second = !first && quad < 2 * quads;
        const int from = base + (first ? quad + quads : second ? quad - quads : quad);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float other = __shfl_sync(0xffffffffu, x[e], from);
            if (live && first) rope_turn(cs[4 * quad + e], x[e], other);
            else if (live && second) rope_turn(cs[4 * (quad - quads) + e], other, x[e]);
        }
    }
};

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

template <typename T, int W, int D>
__global__ void __launch_bounds__(kAppendThreads, 2) kv_append_rope_kernel(KvView c, KvRows rows, int shift, int gy, RopePlan plan, const int32_t *pos, RopeRows q,
                                                                           unsigned q_blocks, const T *k, int64_t kt, int64_t kh, const T *v,
                                                                           int64_t vt, int64_t vh, unsigned int *err) {
    __shared__ float2 s_cs[kKB * D / 2];
    __shared__ int s_pos[kRopeTokens], s_live[kRopeTokens];
    grid_dep_launch();
    grid_dep_wait();
    if (blockIdx.x < q_blocks) {
        const int64_t t0 = (int64_t)blockIdx.x * q.per_block;
        const int n = (int)min((int64_t)q.per_block, q.n_tokens - t0);
        if (threadIdx.x < 32) find_tokens(c, rows, pos, t0, n, s_pos, s_live);
        __syncthreads();
        bool zeros = false;
        for (int i = 0; i < n; ++i) zeros = zeros || s_live[i] == 2;
        rope_block<T, W>(plan, q, t0, n, s_cs, [&](int64_t t) { return s_pos[t - t0]; }, [&](int64_t t) { return s_live[t - t0]; }, zeros);
        return;
    }
    const unsigned unit = blockIdx.x - q_blocks;
    kv_append_unit<T, D>(c, rows, shift, unit / gy, (int)(unit % gy), k, kt, kh, v, vt, vh, err, KeyRope{plan, pos, s_cs});
}

template <typename T, int W>
int append_rope_t(const KvView &c, const KvRows &r, const RopePlan &plan, const int32_t *pos, const RopeRows &q, const void *k, int64_t kt,
                  int64_t kh, const void *v, int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s) {
    const AppendShape a = append_shape(c, r);
    const int64_t q_blocks = q.x != nullptr ? (q.n_tokens + q.per_block - 1) / q.per_block : 0, blocks = q_blocks + a.units * a.gy;
    if (blocks > INT32_MAX) return set_error(MQ_ERR_SHAPE, "mqkv_append_rope: %lld blocks, below 2^31 wanted (fewer tokens a call)", (long long)blocks);
    auto fn = c.D == 128 ? kv_append_rope_kernel<T, W, 128> : kv_append_rope_kernel<T, W, 64>;
    return cuda_error(launch_pdl(fn, dim3((unsigned)blocks), dim3(kAppendThreads), 0, s, c, r, a.shift, a.gy, plan, pos, q, (unsigned)q_blocks,
                                 static_cast<const T *>(k), kt, kh, static_cast<const T *>(v), vt, vh, err),
                      "mqkv_append_rope launch");
}

}  // namespace

int kv_launch_append_rope(const KvView &c, const KvRows &r, int dtype, const RopePlan &plan, const int32_t *pos, const KvRopeRows &q, const void *k,
                          int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s) {
    const RopeRows rows{q.x, q.out, q.xt, q.xh, q.ot, q.oh, r.n_tokens, q.heads, c.D, r.n_tokens <= 4 * sm_count() ? 1 : kRopeTokens};
    const bool wide = rope_wide(plan, rows);
    auto fn = dtype == MQKV_F32   ? append_rope_t<float, 4>
              : dtype == MQKV_F16 ? (wide ? append_rope_t<__half, 8> : append_rope_t<__half, 4>)
                                  : (wide ? append_rope_t<__nv_bfloat16, 8> : append_rope_t<__nv_bfloat16, 4>);
    return fn(c, r, plan, pos, rows, k, kt, kh, v, vt, vh, err, s);
}

}  // namespace mq

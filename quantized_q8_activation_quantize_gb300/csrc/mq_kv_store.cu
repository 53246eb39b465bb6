// mq_kv_store.cu -- the cache's writes and reads of values: quantizing new keys and values into their pages, and the
// values back out of them.  Both move each byte once; the arithmetic is a few instructions a value.
#include "mq_kv_append.cuh"

namespace mq {
namespace {

// One CTA per unit and two vectors (mq_kv_append.cuh).
// Moves 5 (f32) or 3 bytes a value: 32k tokens of 8 heads of 128 in 63 us from f32 (5.2 TB/s), 46 from f16 (4.3), 58 from bf16 (3.4; its
// kernel spills 88 bytes at three CTAs per SM).
template <typename TIN, int D>
__global__ void __launch_bounds__(kAppendThreads, sizeof(TIN) == 4 ? 2 : 3) kv_append_kernel(KvView c, KvRows rows, int shift, const TIN *k, int64_t kt, int64_t kh,
                                                                      const TIN *v, int64_t vt, int64_t vh, unsigned int *err) {
    grid_dep_launch();
    grid_dep_wait();
    kv_append_unit<TIN, D>(c, rows, shift, blockIdx.x, blockIdx.y, k, kt, kh, v, vt, vh, err, NoRope());
}

constexpr int kReadTokens = 16, kReadThreads = 256;

// One CTA per 16 rows of the output, a warp per row and 8 of its 2 H vectors (half, head) at a time: their loads fly together.  Moves 5
// (f32) or 3 bytes a value.
template <typename TOUT, int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(KvView c, KvRows rows, TOUT *k, int64_t kt, int64_t kh, TOUT *v,
                                                               int64_t vt, int64_t vh, const int32_t *start, unsigned int *err) {
    constexpr int LPR = D / 4, RPW = 32 / LPR, B = 8 / RPW;               // lanes per vector, vectors per load, loads in flight
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
    const int spp = c.T / kKB;
    for (int t = warp; t < nt; t += kReadThreads / 32) {
        const uint8_t *slab = s_slab[t];
        const int slot = s_slot[t];
        for (int v0 = 0; v0 < heads; v0 += 8) {
            uint32_t w[B];
            float d[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int vec = v0 + i * RPW + lane / LPR;
                w[i] = 0x80808080u, d[i] = 0.0f;
                if (slab != nullptr && vec < heads) {
                    // K of every head, then V of every head: one run of vectors
                    w[i] = *reinterpret_cast<const uint32_t *>(slab + ((int64_t)vec * c.T + slot) * D + 4 * quad);
                    d[i] = reinterpret_cast<const float *>(slab + c.off_s)[vec * spp + slot / kKB];
                }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int vec = v0 + i * RPW + lane / LPR, half = vec >= c.H, h = vec - half * c.H;
                TOUT *dst = half ? v : k;
                if (vec >= heads || dst == nullptr) continue;
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(code_value(w[i], e), d[i]);
                store4(dst + (t0 + t) * (half ? vt : kt) + h * (half ? vh : kh) + 4 * quad, x);
            }
        }
    }
}

template <typename T>
int append_t(const KvView &c, const KvRows &r, const void *k, int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh,
             unsigned int *err, cudaStream_t s) {
    const AppendShape a = append_shape(c, r);
    const dim3 grid((unsigned)a.units, a.gy);
    auto fn = c.D == 128 ? kv_append_kernel<T, 128> : kv_append_kernel<T, 64>;
    return cuda_error(launch_pdl(fn, grid, dim3(kAppendThreads), 0, s, c, r, a.shift, static_cast<const T *>(k), kt, kh,
                                 static_cast<const T *>(v), vt, vh, err),
                      "mqkv_append launch");
}

template <typename T>
int read_t(const KvView &c, const KvRows &r, void *k, int64_t kt, int64_t kh, void *v, int64_t vt, int64_t vh,
           const int32_t *start, unsigned int *err, cudaStream_t s) {
    const dim3 grid((unsigned)((r.n_tokens + kReadTokens - 1) / kReadTokens));
    auto fn = c.D == 128 ? kv_read_kernel<T, 128> : kv_read_kernel<T, 64>;
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

// mq_kv_store.cu -- the cache's writes and reads of values: quantizing new keys and values into their pages, and the
// values back out of them.  Both move each byte once; the arithmetic is a few instructions a value.
#include <cfloat>

#include "mq_kv.cuh"

namespace mq {
namespace {

constexpr int kAppendThreads = 128;

// One CTA per (block of 32 slots, head, half).  Unit u of the grid's x belongs to the last sequence b with
// U(b) <= u, U(b) = begin(b) / 32 + 2 b: a sequence of n tokens touches at most n / 32 + 2 blocks, so the units of
// the sequences never overlap and need no prefix sum.
template <typename TIN, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(KvView c, KvRows rows, const TIN *k, int64_t kt, int64_t kh,
                                                                   const TIN *v, int64_t vt, int64_t vh, unsigned int *err) {
    constexpr int LPR = D / 4, RPW = 32 / LPR, IT = kKB / (4 * RPW);      // lanes per row, rows per warp and step, steps
    __shared__ float s_amax[4];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t u = blockIdx.x;
    int b;
    int64_t u0;
    if (rows.cu == nullptr) {
        const int64_t per = (rows.each + 2 * kKB - 2) / kKB;
        b = (int)(u / per);
        u0 = b * per;
        if (b >= c.n_seqs) return;
    } else {
        int lo = 0, hi = c.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (rows.begin(mid) / kKB + 2 * (int64_t)mid <= u) lo = mid; else hi = mid - 1;
        }
        b = lo;
        u0 = rows.begin(b) / kKB + 2 * (int64_t)b;
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
    const int64_t p0 = len - n, blk = p0 / kKB + (u - u0), s0 = blk * kKB;
    if (s0 >= len) return;
    const int page = c.table[(int64_t)b * c.max_pages + (s0 >> c.tshift)];
    if (page < 0 || page >= c.n_pages) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_PAGE);
        return;
    }
    if (c.refs != nullptr && c.refs[page] != 1) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_SHARED);
        return;
    }
    const int half = blockIdx.y >= c.H, h = blockIdx.y - half * c.H;
    const int slot0 = (int)(s0 & (c.T - 1));
    uint8_t *slab = c.pool + page * c.page_bytes;
    uint8_t *codes = slab + (half ? c.off_v : 0) + ((int64_t)h * c.T + slot0) * D;
    float *scale = reinterpret_cast<float *>(slab + c.off_s) + (half * c.H + h) * (c.T / kKB) + slot0 / kKB;
    const TIN *src = (half ? v + h * vh : k + h * kh);
    const int64_t st = half ? vt : kt;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane % LPR;

    float x[IT][4];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int64_t pos = s0 + (warp + 4 * i) * RPW + lane / LPR;
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0f;
        if (pos >= p0 && pos < len) {
            load4(src + (lo + pos - p0) * st + 4 * quad, x[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (x[i][e] != x[i][e]) x[i][e] = 0.0f;
                const float a = fabsf(x[i][e]);
                amax = fmaxf(amax, a <= FLT_MAX ? a : 0.0f);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_amax[warp] = amax;
    const bool tail = s0 < p0;                    // slots of earlier tokens
    float d_old = tail ? *scale : 0.0f;
    if (!(d_old >= 0.0f && d_old <= FLT_MAX)) d_old = 0.0f;
    __syncthreads();
    amax = fmaxf(fmaxf(s_amax[0], s_amax[1]), fmaxf(s_amax[2], s_amax[3]));
    float d = __fmul_rn(amax, 1.0f / 127.0f);
    if (d < FLT_MIN) d = 0.0f;
    d = fmaxf(d, d_old);
    const float id = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    const float shrink = d > d_old ? __fdiv_rn(d_old, d) : 1.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = (warp + 4 * i) * RPW + lane / LPR;
        const int64_t pos = s0 + r;
        uint32_t *dst = reinterpret_cast<uint32_t *>(codes + r * D + 4 * quad);
        uint32_t w = 0;
        if (pos >= p0 && pos < len) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q = d > 0.0f ? fminf(fmaxf(roundf(__fmul_rn(x[i][e], id)), -127.0f), 127.0f) : 0.0f;
                w |= (uint32_t)(__float2int_rn(q) + 128) << (8 * e);
            }
            *dst = w;
        } else if (pos < p0 && shrink != 1.0f) {
            const uint32_t old = *dst;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q = roundf(__fmul_rn((float)(int)((old >> (8 * e)) & 255u) - 128.0f, shrink));
                w |= (uint32_t)(__float2int_rn(q) + 128) << (8 * e);
            }
            *dst = w;
        }
    }
    if (threadIdx.x == 0) *scale = d;
}

constexpr int kReadTokens = 16, kReadThreads = 256;

// One CTA per 16 rows of the output; a warp takes (row, half, head) vectors of head_dim values.
template <typename TOUT, int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(KvView c, KvRows rows, TOUT *k, int64_t kt, int64_t kh, TOUT *v,
                                                               int64_t vt, int64_t vh, const int32_t *start, unsigned int *err) {
    constexpr int LPR = D / 4, RPW = 32 / LPR;
    __shared__ const uint8_t *s_slab[kReadTokens];
    __shared__ int s_slot[kReadTokens];
    grid_dep_launch();
    grid_dep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
    const int nt = (int)min((int64_t)kReadTokens, rows.n_tokens - t0);
    if (threadIdx.x < nt) {
        const int64_t t = t0 + threadIdx.x;
        int b;
        if (rows.cu == nullptr) {
            b = (int)(t / rows.each);
        } else {
            int lo = 0, hi = c.n_seqs - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (rows.begin(mid) <= t) lo = mid; else hi = mid - 1;
            }
            b = lo;
        }
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
        s_slab[threadIdx.x] = slab;
        s_slot[threadIdx.x] = (int)(pos & (c.T - 1));
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane % LPR;
    const int heads = 2 * c.H, vecs = nt * heads;
#pragma unroll 4
    for (int i = warp * RPW + lane / LPR; i < vecs; i += (kReadThreads / 32) * RPW) {
        const int t = i / heads, hh = i - t * heads, half = hh >= c.H, h = hh - half * c.H;
        TOUT *dst = half ? v : k;
        if (dst == nullptr) continue;
        dst += (t0 + t) * (half ? vt : kt) + h * (half ? vh : kh) + 4 * quad;
        const uint8_t *slab = s_slab[t];
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (slab != nullptr) {
            const int slot = s_slot[t];
            const uint32_t w = *reinterpret_cast<const uint32_t *>(slab + (half ? c.off_v : 0) + ((int64_t)h * c.T + slot) * D + 4 * quad);
            const float d = reinterpret_cast<const float *>(slab + c.off_s)[(half * c.H + h) * (c.T / kKB) + slot / kKB];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __fmul_rn((float)((int)((w >> (8 * e)) & 255u) - 128), d);
        }
        store4(dst, x);
    }
}

template <typename T>
int append_t(const KvView &c, const KvRows &r, const void *k, int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh,
             unsigned int *err, cudaStream_t s) {
    const int64_t units = r.cu == nullptr ? c.n_seqs * ((r.each + 2 * kKB - 2) / kKB) : r.n_tokens / kKB + 2 * (int64_t)c.n_seqs;
    const dim3 grid((unsigned)units, 2 * c.H);
    auto fn = c.D == 128 ? kv_append_kernel<T, 128> : kv_append_kernel<T, 64>;
    return cuda_error(launch_pdl(fn, grid, dim3(kAppendThreads), 0, s, c, r, static_cast<const T *>(k), kt, kh,
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

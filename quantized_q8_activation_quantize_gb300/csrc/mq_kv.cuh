// mq_kv.cuh -- what the KV cache's kernels share: the cache's geometry, error bits, the rows of a ragged batch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mqkv.h"
#include "mq_device.cuh"
#include "mq_internal.h"

namespace mq {

enum : unsigned int {
    KV_ERR_PAGE = 1u << 0,      // a table entry is not a page of the pool
    KV_ERR_LEN = 1u << 1,       // a length is negative, past the table row, or below the new tokens' count
    KV_ERR_SHARED = 1u << 2,    // append into a page that another sequence shares (or that is free)
    KV_ERR_FULL = 1u << 3,      // too few free pages
    KV_ERR_SEQ = 1u << 4,       // a sequence id out of range, named twice, or a child that is not empty
    KV_ERR_ROWS = 1u << 5,      // more new tokens than max_q
    KV_ERR_WAIT = 1u << 6,      // a bounded wait ran out
};
constexpr int kKvErrBits = 7;

constexpr int kKB = MQKV_BLOCK;

// one layer of a cache, as the kernels see it
struct KvView {
    uint8_t *pool;              // slab of the layer in page 0
    const int32_t *refs;
    int64_t page_bytes;
    int64_t n_pages;
    const int32_t *table;
    const int32_t *len;
    int32_t n_seqs, max_pages;
    int32_t H, D, T, tshift;    // T = 1 << tshift
    int64_t off_v, off_s;
};

// the new tokens of a ragged batch: rows [lo, hi) of sequence b (never outside [0, n_tokens))
struct KvRows {
    const int32_t *cu;
    int64_t n_tokens;
    int64_t each;               // cu == nullptr: rows per sequence
    __device__ __forceinline__ void of(int b, int64_t &lo, int64_t &hi) const {
        if (cu == nullptr) {
            lo = b * each;
            hi = lo + each;
            return;
        }
        lo = min(max((int64_t)cu[b], (int64_t)0), n_tokens);
        hi = min(max((int64_t)cu[b + 1], lo), n_tokens);
    }
    __device__ __forceinline__ int64_t begin(int b) const {
        return cu == nullptr ? b * each : min(max((int64_t)cu[b], (int64_t)0), n_tokens);
    }
};

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// four consecutive values of a row: as they are stored, and as f32
template <typename T>
struct Raw4 {
    uint2 w;
};
template <>
struct Raw4<float> {
    float4 w;
};
__device__ __forceinline__ void unpack4(const Raw4<float> &r, float *x) { x[0] = r.w.x, x[1] = r.w.y, x[2] = r.w.z, x[3] = r.w.w; }
__device__ __forceinline__ void unpack4(const Raw4<__half> &r, float *x) {
    const float2 a = unpack_f16(r.w.x), b = unpack_f16(r.w.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ void unpack4(const Raw4<__nv_bfloat16> &r, float *x) {
    x[0] = __uint_as_float(r.w.x << 16), x[1] = __uint_as_float(r.w.x & 0xffff0000u);
    x[2] = __uint_as_float(r.w.y << 16), x[3] = __uint_as_float(r.w.y & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ void load4(const T *p, float *x) {
    unpack4(*reinterpret_cast<const Raw4<T> *>(p), x);
}
__device__ __forceinline__ void store4(float *p, const float *x) { *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void store4(__half *p, const float *x) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]));
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float *x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Codes and values without conversion instructions (they run at a quarter of the rate): a byte in the low mantissa bits of 2^23.
__device__ __forceinline__ float code_value(uint32_t w, int e) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + e)) - 8388736.0f;              // byte e, minus 128
}
// 128 + round half away from zero of y, |y| clamped to 127; in the low byte.  y + (0.5 - 2^-25), cut to an integer, is that
// rounding: the sum reaches the next integer exactly from the half on.
__device__ __forceinline__ uint32_t value_code(float y) {
    const float n = __fadd_rz(__fadd_rn(fminf(fabsf(y), 127.0f), 0.49999997f), 8388608.0f);
    const uint32_t s = (uint32_t)(__float_as_int(y) >> 31);
    return (__float_as_uint(n) ^ s) - s + 128u;
}
__device__ __forceinline__ uint32_t pack_codes(const float (&y)[4]) {
    const uint32_t a = __byte_perm(value_code(y[0]), value_code(y[1]), 0x0040), b = __byte_perm(value_code(y[2]), value_code(y[3]), 0x0040);
    return __byte_perm(a, b, 0x5410);
}

__device__ __forceinline__ void kv_error(unsigned int *err, unsigned int bit) { atomicOr(err, bit); }

// launchers (arguments already validated)
int kv_launch_append(const KvView &c, const KvRows &r, int dtype, const void *k, int64_t kt, int64_t kh, const void *v,
                     int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s);
int kv_launch_read(const KvView &c, const KvRows &r, int dtype, void *k, int64_t kt, int64_t kh, void *v, int64_t vt,
                   int64_t vh, const int32_t *start, unsigned int *err, cudaStream_t s);

struct KvAttn {
    const void *q;
    void *out;
    int64_t qt, qh, ot, oh;
    int32_t n_q_heads, group, dtype, causal;
    int64_t max_q, max_kv, window;
    float scale;
};
int kv_launch_attention(const mqkv_cache &cache, const mqkv_layout &lay, int layer, const KvView &c, const KvRows &r,
                        const KvAttn &a, void *ws, unsigned int *err, cudaStream_t s);
size_t kv_attention_ws(int32_t n_seqs, int32_t H, int32_t D, int dtype, int32_t n_q_heads, int64_t n_tokens,
                       int64_t max_q, int64_t max_kv);

struct KvPages {
    uint8_t *pool;
    int32_t *refs, *table, *len;
    int64_t page_bytes, layer_bytes, off_s;
    int32_t n_pages, n_seqs, max_pages, tshift, n_layers, H, D;
};
size_t kv_pages_ws(int64_t n_pages, int64_t n_seqs);
int kv_launch_extend(const KvPages &p, const int32_t *add, void *ws, unsigned int *err, cudaStream_t s);
int kv_launch_release(const KvPages &p, const int32_t *ids, int n, unsigned int *err, cudaStream_t s);
int kv_launch_fork(const KvPages &p, const int32_t *parent, const int32_t *child, int n, void *ws, unsigned int *err,
                   cudaStream_t s);
int kv_launch_compact(const KvPages &p, void *ws, unsigned int *err, cudaStream_t s);
int kv_launch_copy(const KvPages &p, const int32_t *src, const int32_t *dst, int n, unsigned int *err, cudaStream_t s);

}  // namespace mq

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

// the last sequence whose rows begin at or before row t (cu not falling): 32 ends at a time, one a lane
__device__ __forceinline__ int kv_find_seq(const KvRows &rows, int n_seqs, int64_t t, int step_per_seq, int shift) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;                                   // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int stride = (n + 31) / 32, at = min(lane * stride, n - 1);
        const int64_t begin = (rows.begin(lo + at) >> shift) + (int64_t)step_per_seq * (lo + at);
        const uint32_t yes = __ballot_sync(0xffffffffu, lane == 0 || begin <= t);
        // lanes past the end repeat the last sequence: the highest lane that says yes names its stride's beginning
        const int k = 31 - __clz(yes), from = min(k * stride, n - 1);
        lo += from;
        n = min(stride, n - from);
    }
    return lo;
}

// pairs of f32 in one register pair: half the issue slots
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

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
// the largest magnitude of four values into amax (NaN aside), and z, which becomes NaN where one of them is a NaN or an infinity
__device__ __forceinline__ void scan4(const Raw4<float> &r, float &amax, uint64_t &z) {
    amax = fmaxf(fmaxf(amax, fabsf(r.w.x)), fabsf(r.w.y));
    amax = fmaxf(fmaxf(amax, fabsf(r.w.z)), fabsf(r.w.w));
    z = f2_fma(f2_pack(r.w.x, r.w.y), f2_pack(0.0f, 0.0f), z);
    z = f2_fma(f2_pack(r.w.z, r.w.w), f2_pack(0.0f, 0.0f), z);
}
template <typename T2>
__device__ __forceinline__ void scan2(uint32_t w, T2 &amax, T2 &z) {
    const uint32_t none = 0;
    const T2 a = *reinterpret_cast<const T2 *>(&w);
    amax = __hmax2(amax, __habs2(a));
    z = __hfma2(a, *reinterpret_cast<const T2 *>(&none), z);
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

// Codes and values without conversion instructions (they run at a quarter of the rate) and with few ALU ones (half the rate): a byte in
// the low mantissa bits of 2^23.
__device__ __forceinline__ float code_value(uint32_t w, int e) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + e)) - 8388736.0f;              // byte e, minus 128
}
__device__ __forceinline__ uint64_t code_values(uint32_t w, int e) {       // of bytes e and e + 1
    return f2_add(f2_pack(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + e)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7541 + e))),
                  f2_pack(-8388736.0f, -8388736.0f));
}
__device__ __forceinline__ uint64_t f2_fma_rz(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// 128 + round half away from zero of two values of at most 127.4, in the low byte of each.  With s the value's sign: y + s (0.5 - 2^-25)
// cut to an integer is that rounding (the sum reaches the next integer exactly from the half on), and adding s 2^23 toward zero cuts.
__device__ __forceinline__ void value_codes2(uint64_t y, uint32_t &a, uint32_t &b) {
    float y0, y1;
    f2_unpack(y, y0, y1);
    const uint64_t s = f2_pack(__uint_as_float((__float_as_uint(y0) & 0x80000000u) | 0x3f800000u),
                               __uint_as_float((__float_as_uint(y1) & 0x80000000u) | 0x3f800000u));
    const uint64_t t = f2_fma(s, f2_pack(0.49999997f, 0.49999997f), y);
    const uint64_t u = f2_fma_rz(s, f2_pack(8388608.0f, 8388608.0f), t);
    const uint64_t n = f2_fma(s, f2_pack(-8388608.0f, -8388608.0f), u);
    f2_unpack(f2_add(n, f2_pack(8388736.0f, 8388736.0f)), y0, y1);
    a = __float_as_uint(y0), b = __float_as_uint(y1);
}
__device__ __forceinline__ uint32_t pack_codes(uint64_t y01, uint64_t y23) {
    uint32_t a, b, c, d;
    value_codes2(y01, a, b);
    value_codes2(y23, c, d);
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ void kv_error(unsigned int *err, unsigned int bit) { atomicOr(err, bit); }

// launchers (arguments already validated)
int kv_launch_append(const KvView &c, const KvRows &r, int dtype, const void *k, int64_t kt, int64_t kh, const void *v,
                     int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s);
// the queries beside a turned append (mq_kv_rope.cu); x: nullptr where there are none
struct KvRopeRows {
    const void *x;
    void *out;
    int64_t xt, xh, ot, oh;
    int32_t heads;
};
struct RopePlan;
int kv_launch_append_rope(const KvView &c, const KvRows &r, int dtype, const RopePlan &plan, const int32_t *pos, const KvRopeRows &q, const void *k,
                          int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh, unsigned int *err, cudaStream_t s);
int kv_launch_read(const KvView &c, const KvRows &r, int dtype, void *k, int64_t kt, int64_t kh, void *v, int64_t vt,
                   int64_t vh, const int32_t *start, unsigned int *err, cudaStream_t s);

struct KvAttn {
    const void *q;
    void *out;
    int64_t qt, qh, ot, oh;
    int32_t n_q_heads, group, dtype, causal;
    int64_t n_tokens, max_q, max_kv, window;
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
constexpr int kKvReorderRows = 4096;        // rows that a reordering may have
int kv_launch_reorder(const KvPages &p, const int32_t *parent, void *ws, unsigned int *err, cudaStream_t s);
int kv_launch_compact(const KvPages &p, void *ws, unsigned int *err, cudaStream_t s);
int kv_launch_copy(const KvPages &p, const int32_t *src, const int32_t *dst, int n, unsigned int *err, cudaStream_t s);

}  // namespace mq

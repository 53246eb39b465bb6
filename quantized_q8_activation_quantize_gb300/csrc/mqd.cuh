// mqd.cuh -- what the kernels between the matrix products and the cache share (include/mqd.h): eight values of a row at a time, and
// the launchers.
#pragma once

#include "../../include/mqd.h"
#include "mq_kv.cuh"

namespace mq {

// eight consecutive values of a row as they are stored (32 or 16 bytes), and as f32
template <typename T>
struct Raw8 {
    uint4 w;
};
template <>
struct Raw8<float> {
    float4 a, b;
};
__device__ __forceinline__ Raw8<float> load8(const float *p) {
    return {*reinterpret_cast<const float4 *>(p), *reinterpret_cast<const float4 *>(p + 4)};
}
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T *p) {
    return {*reinterpret_cast<const uint4 *>(p)};
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&x)[8]) {
    x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w, x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float (&x)[8]) {
    unpack4(Raw4<T>{make_uint2(r.w.x, r.w.y)}, x);
    unpack4(Raw4<T>{make_uint2(r.w.z, r.w.w)}, x + 4);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ Raw8<float> pack8(const float (&x)[8], float) {
    return {make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])};
}
__device__ __forceinline__ Raw8<__half> pack8(const float (&x)[8], __half) {
    return {make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7]))};
}
__device__ __forceinline__ Raw8<__nv_bfloat16> pack8(const float (&x)[8], __nv_bfloat16) {
    return {make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]))};
}
__device__ __forceinline__ void store8(float *p, const Raw8<float> &r) {
    reinterpret_cast<float4 *>(p)[0] = r.a;
    reinterpret_cast<float4 *>(p)[1] = r.b;
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const Raw8<T> &r) {
    *reinterpret_cast<uint4 *>(p) = r.w;
}
// store8 by all lanes of a warp, lane l to base + 8 l.  f32: neighbouring lanes exchange quarters, so that a store fills whole sectors of 32 bytes
__device__ __forceinline__ void store8_row(float *p, const Raw8<float> &r, int lane) {
    const bool odd = lane & 1;
    const float4 give = odd ? r.a : r.b;
    float4 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, 1), got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, 1), got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
    reinterpret_cast<float4 *>(p)[odd ? -1 : 0] = odd ? got : r.a;
    reinterpret_cast<float4 *>(p)[odd ? 1 : 2] = odd ? r.b : got;
}
template <typename T>
__device__ __forceinline__ void store8_row(T *p, const Raw8<T> &r, int) {
    store8(p, r);
}

// launchers (arguments already validated)
struct AddQuantize {
    const void *x, *res;
    void *h;
    int64_t xs, rs, hs, M, K;
    const float *w;
    float eps;
    unsigned sections;
};
int launch_add_quantize(const AddQuantize &a, int dtype, const Plane &p, cudaStream_t s);
int launch_dequantize(const Plane &p, int64_t M, int64_t K, bool q16, int dtype, void *y, int64_t ys, cudaStream_t s);

struct RopePlan {
    const uint64_t *turns;
    int32_t half;               // pairs of a head
    int32_t interleaved;
    float amplitude;
};
struct RopeRows {
    const void *x;
    void *out;
    int64_t xt, xh, ot, oh;
    int64_t n_tokens;
    int32_t heads, dim, per_block;      // tokens per block
};
int launch_rope(const RopePlan &plan, RopeRows r, int dtype, const int32_t *pos, cudaStream_t s);

size_t beam_ws(int64_t n_groups, int B, int64_t V, int n_cand);
int launch_beam_select(int dtype, const void *logits, int64_t stride, int64_t n_groups, int B, int64_t V, const float *scores, int k, int stop,
                       float *cand_score, int32_t *cand_row, int32_t *cand_token, float *next_score, int32_t *next_row, int32_t *next_token,
                       void *workspace, cudaStream_t s);

// checks of the host that the cache's calls share (mqd_abi.cu): MQ_OK or a negative status
int rope_plan_of(const char *fn, const mqd_rope_plan *plan, int32_t head_dim, RopePlan *out);
int check_rope_heads(const char *fn, const char *what, const void *p, int64_t ts, int64_t hs, int32_t dtype);
int check_rope_out(const char *fn, const void *x, int64_t xt, int64_t xh, const void *out, int64_t ot, int64_t oh, int64_t n, int64_t heads, int64_t dim,
                   int32_t dtype);
bool values_apart(const void *a, size_t na, int64_t as, int64_t aw, const void *b, size_t nb, int64_t bs, int64_t bw, int64_t n, int32_t dtype);
size_t heads_span(int64_t n, int64_t heads, int64_t dim, int64_t ts, int64_t hs, int32_t dtype);

}  // namespace mq

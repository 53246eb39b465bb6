// mq_kv_attn.cuh -- what the attention kernels share.
#pragma once

#include <cuda.h>

#include "mq_kv.cuh"

namespace mq {

// the tiled kernel for many rows (mq_kv_prefill.cu)
int kv_launch_prefill(const KvView &c, const KvRows &r, const KvAttn &p, void *ws, unsigned int *err, cudaStream_t s);
size_t kv_prefill_ws(int32_t n_seqs, int32_t H, int32_t D, int dtype, int group, int64_t n_tokens, int64_t max_q);

constexpr float kLog2e = 1.44269504088896341f;
// Every row has two references, both powers of two: m for its scores, of which l = sum 2^(s - m), and A for its weights times V scales, of which
// o = sum 2^(s - A) dv v.  What enters the tensor cores, 2^(s - m + shift) times dv 2^(m - A), is at most 2^shift however the V scales of the
// row's tokens differ, and what the row does not see or hardly weighs takes no bits from the rest.  (With the largest V scale of all blocks met, seen by
// the row or not, as one reference for all rows, a block of 2^16 times the others' scale without weight put f32 rows of a long share 2e-4 off, one
// of 2^28 0.4.)  The result is o 2^(A - m) / l.
// kPShift keeps small weights out of f16's subnormals; where the references move only when the maximum grows by more than kTau, weights
// reach 2^(kLazyShift + kTau) < 65504.
constexpr float kPShift = 12.0f, kTau = 8.0f, kLazyShift = 6.0f;
// A stays above m - kRefSpan, so that 2^(m - A) is finite (a row that has met scales of zero only)
constexpr float kRefSpan = 120.0f;

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(x - y) of references, 0 where there is none yet (y is minus infinity)
__device__ __forceinline__ float ref_factor(float x, float y) { return y == -INFINITY ? 0.0f : exp2_approx(x - y); }
// what a weight relative to m is multiplied by to become one relative to A, for a V scale (finite: a weight of zero stays zero)
__device__ __forceinline__ float v_factor(float dv, float m_over_a) { return fminf(dv * m_over_a, 3.402823466e38f); }

// four codes of a word as two f16 pairs, exactly: byte b becomes the f16 1024 + b, minus 1152
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off), y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<uint32_t *>(&x);
    hi = *reinterpret_cast<uint32_t *>(&y);
}

// 2^e with e such that amax * 2^-e lies in [2^14, 2^15) (1 where amax is 0); a row is multiplied by 2^-e before it
// becomes f16.  Exponents stay where 2^e and 2^-e are normal numbers.
__device__ __forceinline__ int row_exponent(float amax) {
    const int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127 - 14;
    return amax == 0.0f ? 0 : min(max(e, -120), 120);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// positions [lo, hi) that the row at position p of a sequence of len tokens sees
__device__ __forceinline__ void row_range(int64_t p, int64_t len, int causal, int64_t window, int64_t &lo, int64_t &hi) {
    hi = causal ? min(p + 1, len) : len;
    lo = window > 0 ? max(p - window + 1, (int64_t)0) : 0;
    if (hi <= lo) lo = hi = 0;
}

// 5-D tiled copy global -> shared through a CUtensorMap
__device__ __forceinline__ void tma_load_5d(void *dst_smem, const void *tmap, int32_t x, int32_t y, int32_t z, int32_t w, int32_t v, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            smem_u32(dst_smem)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
        : "memory");
}

}  // namespace mq

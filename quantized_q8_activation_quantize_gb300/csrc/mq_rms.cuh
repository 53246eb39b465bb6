// mq_rms.cuh -- what the RMSNorm producers share (mq_quantize.cu; with the residual's addition mqd_add.cu): the sum of squares as
// compensated f32 pairs, r = 1 / sqrt(mean + eps) from it, and the Q8 quantization of a row held in registers.
#pragma once

#include <cuda_fp16.h>

#include "mq_device.cuh"
#include "mq_internal.h"
#include "mq_pair.h"

namespace mq {

constexpr unsigned kFull = 0xffffffffu;

// Error-free product and sum in f32 (Dekker / Knuth): x * x = p + e exactly (e from one fused
// multiply-add), and the running pair (hi, lo) takes p with Knuth's branch-free two-sum, whose
// rounding error goes to lo.  Every step is an explicitly rounded intrinsic, so the compiler can
// neither contract nor reassociate it.
__device__ __forceinline__ void add_square(float v, float &hi, float &lo) {
    const float p = __fmul_rn(v, v);
    const float e = __fmaf_rn(v, v, -p);
    const float s = __fadd_rn(hi, p);
    const float bv = __fsub_rn(s, hi);
    const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bv)), __fsub_rn(p, bv));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(err, e));
}

// (ah, al) += (bh, bl) for pairs of f32 (a value and its small correction): the high parts add
// error-free, the corrections add rounded, and the result is renormalised (|al| <= ulp(ah) / 2).
// The result does not depend on the order of the operands, so a butterfly over the lanes leaves
// the same pair in every lane.
__device__ __forceinline__ void pair_add(float &ah, float &al, float bh, float bl) {
    float s, e;
    two_sum(ah, bh, s, e);
    e = __fadd_rn(e, __fadd_rn(al, bl));
    ah = __fadd_rn(s, e);
    al = __fsub_rn(e, __fsub_rn(ah, s));
}

// r = 1 / sqrt(t / K + eps) rounded once to f32, from the sum of squares t = th + tl (reduced
// from the lanes' pairs by pair_add), in f32 arithmetic only.  The lanes' pairs add as f32 pairs
// (relative error below 2^-43 for these non-negative sums), t / K is an f32 pair (the remainder
// t - q K of the quotient q is exact for K < 2^22), and one Newton step on rsqrtf's estimate y0
// (error below 2^-21) gives y0 + yl within 2^-41 of the value the same lane pairs give in f64.  When every point within 2^-38 y0 of
// y0 + yl rounds to the same f32, that is r, and it equals the rounding of the f64 evaluation;
// otherwise (about one token in 10^4: the value lies near a rounding boundary) or outside the
// normal range the function returns false and the caller evaluates r in f64.  The f64 pipe of
// this GPU issues ~1.7 operations per clock per SM, so its square root and divide (dozens of
// operations each) cost more than the rest of a token's arithmetic.
__device__ __forceinline__ bool rms_scale_from_pair(float th, float tl, int64_t K, float eps, float &r) {
    const float kf = (float)K;
    const float ik = __frcp_rn(kf);
    const float qh = __fmul_rn(th, ik);
    const float rem = __fmaf_rn(-qh, kf, th);
    const float ql = __fmul_rn(__fadd_rn(rem, tl), ik);
    float vh, vl;
    two_sum(qh, eps, vh, vl);
    vl = __fadd_rn(vl, ql);
    // Newton step for 1/sqrt(v): y1 = y0 + y0 (1 - v y0^2) / 2, with y0^2 = p + pe exactly
    const float y0 = rsqrtf(vh);
    const float p = __fmul_rn(y0, y0);
    const float pe = __fmaf_rn(y0, y0, -p);
    const float a = __fmaf_rn(-vh, p, 1.0f);
    const float c = __fsub_rn(a, __fmaf_rn(vh, pe, __fmul_rn(vl, p)));
    const float yl = __fmul_rn(__fmul_rn(0.5f, y0), c);
    const float dl = __fmul_rn(y0, 0x1p-38f);
    const float ra = __fadd_rn(y0, __fsub_rn(yl, dl));
    const float rb = __fadd_rn(y0, __fadd_rn(yl, dl));
    r = ra;
    return ra == rb && vh >= 0x1p-100f && vh <= 0x1p100f;
}

// bar.sync on named barrier `id` (1 .. 15) for `threads` threads (whole warps)
__device__ __forceinline__ void named_bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// packed f32 pairs: each component rounded once to nearest, as __fadd_rn / __fsub_rn / __fmul_rn /
// __fmaf_rn on it (one instruction for both)
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "sub.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// add_square on two independent (hi, lo) chains at once, chain 0 in .x and chain 1 in .y
__device__ __forceinline__ void add_square2(float2 v, float2 &hi, float2 &lo) {
    const float2 p = __fmul2_rn(v, v);
    const float2 e = __ffma2_rn(v, v, make_float2(-p.x, -p.y));
    const float2 s = __fadd2_rn(hi, p);
    const float2 bv = sub2(s, hi);
    const float2 err = __fadd2_rn(sub2(hi, sub2(s, bv)), sub2(p, bv));
    hi = s;
    lo = __fadd2_rn(lo, __fadd2_rn(err, e));
}

// Round half away from zero of two values of less than 2^22 in magnitude, +0 for what rounds to zero; roundf takes five instructions for one.  With s the value's
// sign: y + s (0.5 - 2^-25) cut to an integer is that rounding (the sum reaches the next integer exactly from the half on), and adding s 2^23 toward zero cuts.
__device__ __forceinline__ float2 round_away2(float2 y) {
    const float2 s = make_float2(__uint_as_float((__float_as_uint(y.x) & 0x80000000u) | 0x3f800000u),
                                 __uint_as_float((__float_as_uint(y.y) & 0x80000000u) | 0x3f800000u));
    const float2 t = __ffma2_rn(s, make_float2(0.49999997f, 0.49999997f), y);
    const float2 u = __ffma2_rz(s, make_float2(8388608.0f, 8388608.0f), t);
    return __ffma2_rn(s, make_float2(-8388608.0f, -8388608.0f), u);
}

// Q8 quantization of up to NC <= 4 256-value chunks held by one warp (chunk j: lane l holds values
// 8l .. 8l + 7 of chunk cj = c0 + j * cstep, at columns 256 cj + 8l ..); chunks j >= nvalid are not
// written.  The per-value arithmetic is quantize8's; the per-block arithmetic (d = amax / 127,
// 1 / d, S, d * S and their stores) runs once per block instead of once per lane: the four lanes
// of a block reduce its amax and code sum as in quantize8, then lane 8j + q takes block q of
// chunk j (one block per lane) and hands 1 / d back.
// sect: the plane sections written besides d and S (a constant where the caller's is one).
template <int NC>
__device__ __forceinline__ void quantize_chunks(const float (&v)[NC][8], int nvalid, int c0, int cstep, int lane, unsigned sect,
                                                const Plane &p, int64_t M, int64_t K, int64_t m) {
    float am[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[j][i]));
        a = fmaxf(a, __shfl_xor_sync(kFull, a, 1));
        am[j] = fmaxf(a, __shfl_xor_sync(kFull, a, 2));
    }
    const int jl = lane >> 3, ql = lane & 7;
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const float t = __shfl_sync(kFull, am[j], 4 * ql);
        if (jl == j) amax = t;
    }
    const float d = __fdiv_rn(amax, 127.0f);
    const float id = (d != 0.0f) ? __fdiv_rn(1.0f, d) : 0.0f;
    float fsj[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const float idj = __shfl_sync(kFull, id, 8 * j + (lane >> 2));
        float r[8];
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 n = round_away2(__fmul2_rn(make_float2(v[j][i], v[j][i + 1]), make_float2(idj, idj)));
            r[i] = n.x, r[i + 1] = n.y;
            sum = __fadd2_rn(sum, n);
        }
        float fs = __fadd_rn(sum.x, sum.y);
        if (!(fabsf(fs) < 0x1p20f)) {                       // (rare) a value that is not finite, or whose scale is subnormal: to the end of the range
            fs = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[i] = __fadd_rn(fminf(fmaxf(roundf(__fmul_rn(v[j][i], idj)), -127.0f), 127.0f), 0.0f);
                fs = __fadd_rn(fs, r[i]);
            }
        }
        fs = __fadd_rn(fs, __shfl_xor_sync(kFull, fs, 1));
        fsj[j] = __fadd_rn(fs, __shfl_xor_sync(kFull, fs, 2));
        if (j < nvalid) {
            const int64_t off = m * K + (int64_t)(c0 + j * cstep) * 256 + lane * 8;
            if ((sect & MQ_PLANE_Q8) != 0) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__fadd_rn(r[i], 12582912.0f));
                uint2 b8;
                b8.x = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
                b8.y = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410);
                *reinterpret_cast<uint2 *>(p.q8 + off) = b8;
            }
            if ((sect & MQ_PLANE_Q16) != 0) {
                uint4 h;
                __half2 t;
                t = __floats2half2_rn(r[0], r[1]); h.x = *reinterpret_cast<uint32_t *>(&t);
                t = __floats2half2_rn(r[2], r[3]); h.y = *reinterpret_cast<uint32_t *>(&t);
                t = __floats2half2_rn(r[4], r[5]); h.z = *reinterpret_cast<uint32_t *>(&t);
                t = __floats2half2_rn(r[6], r[7]); h.w = *reinterpret_cast<uint32_t *>(&t);
                *reinterpret_cast<uint4 *>(p.q16 + off) = h;
            }
        }
    }
    float fs = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const float t = __shfl_sync(kFull, fsj[j], 4 * ql);
        if (jl == j) fs = t;
    }
    if (jl < nvalid) {
        const int s = __float2int_rn(fs);
        const int64_t b = (int64_t)(c0 + jl * cstep) * 8 + ql;
        p.d[b * M + m] = d;
        p.s[b * M + m] = s;
        if ((sect & MQ_PLANE_DS) != 0) {
            const float ds = __fmul_rn(d, (float)s);
            const float hi = tf32_rn(ds);
            const float lo = tf32_rn(__fsub_rn(ds, hi));
            float *row = p.ds + m * (2 * (K / kQ8)) + (b >> 3) * 16 + (b & 7);
            row[0] = hi;
            row[8] = lo;
        }
    }
}

}  // namespace mq

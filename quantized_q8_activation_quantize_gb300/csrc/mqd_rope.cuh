// mqd_rope.cuh -- rotary positions: the angle of a pair as a fraction of a turn, its sine and cosine, and the rotation itself
// (mqd_rope and mqkv_append_rope compute the same values, bit for bit).
#pragma once

#include "mqd.cuh"

namespace mq {

// (a cos, a sin) of the angle pos * F / 2^64 turns.  The product modulo 2^64 is exact, so far positions lose nothing; its upper 32 bits are cut
// into the nearest quarter turn and a rest of at most an eighth, |t| <= pi / 4, where the Taylor series through t^9 and t^10 are off
// by 3e-9 and 2e-10 (half an f32 step is 6e-8).  About 25 instructions for both, without a branch.
__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, uint64_t F, float amplitude) {
    const uint32_t phase = (uint32_t)(((uint64_t)(int64_t)pos * F) >> 32);
    const uint32_t quarter = (phase + 0x20000000u) >> 30;                   // (past 7/8 of a turn the sum wraps to quarter 0)
    const float t = __fmul_rn((float)(int32_t)(phase - (quarter << 30)), 1.5707963267948966f * 0x1p-30f);
    const float z = __fmul_rn(t, t);
    float s = 2.75573192e-6f;                                               // 1 / 9!
    s = __fmaf_rn(s, z, -1.98412698e-4f);
    s = __fmaf_rn(s, z, 8.33333333e-3f);
    s = __fmaf_rn(s, z, -1.66666667e-1f);
    s = __fmaf_rn(__fmul_rn(s, z), t, t);
    float c = -2.75573192e-7f;                                              // -1 / 10!
    c = __fmaf_rn(c, z, 2.48015873e-5f);
    c = __fmaf_rn(c, z, -1.38888889e-3f);
    c = __fmaf_rn(c, z, 4.16666667e-2f);
    c = __fmaf_rn(c, z, -0.5f);
    c = __fmaf_rn(c, z, 1.0f);
    const bool odd = quarter & 1;
    const float x = odd ? s : c, y = odd ? c : s;
    const float ax = ((quarter + 1) & 2) ? -amplitude : amplitude, ay = (quarter & 2) ? -amplitude : amplitude;
    return make_float2(__fmul_rn(x, ax), __fmul_rn(y, ay));
}

constexpr int kRopeThreads = 256, kRopePairs = 512;         // pairs whose (cos, sin) a block holds

template <typename T, int W>
struct RawW;
template <>
struct RawW<float, 4> { float4 w; };
template <>
struct RawW<__half, 4> { uint2 w; };
template <>
struct RawW<__nv_bfloat16, 4> { uint2 w; };
template <>
struct RawW<__half, 8> { uint4 w; };
template <>
struct RawW<__nv_bfloat16, 8> { uint4 w; };

template <typename T, int W>
__device__ __forceinline__ void unpack_w(const RawW<T, W> &r, float (&x)[W]) {
    if constexpr (W == 4) unpack4(*reinterpret_cast<const Raw4<T> *>(&r), x);
    else unpack8(*reinterpret_cast<const Raw8<T> *>(&r), x);
}
template <typename T, int W>
__device__ __forceinline__ void store_w(T *p, const float (&x)[W]) {
    if constexpr (W == 4) store4(p, x);
    else store8(p, pack8(x, T()));
}

// (u, v) -> (u c - v s, v c + u s) of two neighbouring pairs, the products with s rounded, the sums fused: u = (u0, u1) and v = (v0, v1), c = (c0, c1), s = (s0, s1)
__device__ __forceinline__ void rope_turn2(uint64_t c, uint64_t s, uint64_t minus_s, uint64_t &u, uint64_t &v) {
    const uint64_t a = f2_fma(u, c, f2_mul(v, minus_s)), b = f2_fma(v, c, f2_mul(u, s));
    u = a, v = b;
}
// two neighbouring values of one pair, x = (u, v): (u c - v s, v c + u s)
__device__ __forceinline__ uint64_t rope_turn_pair(float c, float s, uint64_t x) {
    float u, v;
    f2_unpack(x, u, v);
    return f2_fma(x, f2_pack(c, c), f2_mul(f2_pack(v, u), f2_pack(-s, s)));
}

// Tokens [t0, t0 + n) by the block's threads: their (cos, sin) once for all heads, then a thread turns W pairs at a time, in pieces of 16 bytes (W = 4
// of 16 bits: 8), two neighbouring ones (interleaved) or two that lie half the rotated part apart.  pos(t): position of token t0 + t; live(t): 1, 0 (its
// row stays as it is) or 2 (its row becomes zeros; `zeros`: whether there is one).  s_cos, s_sin: n * half each.
template <typename T, int W, typename Pos, typename Live>
__device__ __forceinline__ void rope_block(const RopePlan &plan, const RopeRows &r, int64_t t0, int n, float *s_cos, float *s_sin, Pos pos, Live live, bool zeros) {
    for (int i = threadIdx.x; i < n * plan.half; i += kRopeThreads) {
        const int t = i / plan.half;
        const float2 cs = rope_cos_sin(pos(t), plan.turns[i - t * plan.half], plan.amplitude);
        s_cos[i] = cs.x, s_sin[i] = cs.y;
    }
    __syncthreads();
    const bool copy = r.x != r.out || zeros;
    const int pairs = plan.half / W, per = pairs + (copy ? (r.dim - 2 * plan.half) / W : 0);     // pieces of a head
    // piece j of head h of token t; the next of this thread is kRopeThreads pieces on
    int j = threadIdx.x % per, h = threadIdx.x / per, t = h / r.heads;
    h -= t * r.heads;
    const int dj = kRopeThreads % per, dr = kRopeThreads / per, dt = dr / r.heads, dh = dr - dt * r.heads;
    const T *x0 = static_cast<const T *>(r.x) + t0 * r.xt;
    T *out0 = static_cast<T *>(r.out) + t0 * r.ot;
#pragma unroll 1
    while (t < n) {
        const T *x = x0 + t * r.xt + h * r.xh;
        T *out = out0 + t * r.ot + h * r.oh;
        const int what = live(t);
        if (what != 0 && j < pairs) {
            const int a = plan.interleaved ? 2 * j * W : j * W, b = plan.interleaved ? a + W : a + plan.half;
            const RawW<T, W> ra = *reinterpret_cast<const RawW<T, W> *>(x + a), rb = *reinterpret_cast<const RawW<T, W> *>(x + b);
            float u[W], v[W], c[W], s[W];
            const float4 *cs = reinterpret_cast<const float4 *>(s_cos + t * plan.half + j * W), *ss = reinterpret_cast<const float4 *>(s_sin + t * plan.half + j * W);
#pragma unroll
            for (int e = 0; e < W; e += 4) {
                const float4 y = cs[e / 4], z = ss[e / 4];
                c[e] = y.x, c[e + 1] = y.y, c[e + 2] = y.z, c[e + 3] = y.w;
                s[e] = z.x, s[e + 1] = z.y, s[e + 2] = z.z, s[e + 3] = z.w;
            }
            unpack_w<T, W>(ra, u);
            unpack_w<T, W>(rb, v);
            if (plan.interleaved) {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                    f2_unpack(rope_turn_pair(c[e], s[e], f2_pack(u[2 * e], u[2 * e + 1])), u[2 * e], u[2 * e + 1]);
                    f2_unpack(rope_turn_pair(c[W / 2 + e], s[W / 2 + e], f2_pack(v[2 * e], v[2 * e + 1])), v[2 * e], v[2 * e + 1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    uint64_t y = f2_pack(u[e], u[e + 1]), z = f2_pack(v[e], v[e + 1]);
                    rope_turn2(f2_pack(c[e], c[e + 1]), f2_pack(s[e], s[e + 1]), f2_pack(-s[e], -s[e + 1]), y, z);
                    f2_unpack(y, u[e], u[e + 1]);
                    f2_unpack(z, v[e], v[e + 1]);
                }
            }
            if (what == 2) {
#pragma unroll
                for (int e = 0; e < W; ++e) u[e] = v[e] = 0.0f;
            }
            store_w<T, W>(out + a, u);
            store_w<T, W>(out + b, v);
        } else if (what != 0) {
            const int a = 2 * plan.half + (j - pairs) * W;
            RawW<T, W> w = *reinterpret_cast<const RawW<T, W> *>(x + a);
            if (what == 2) w.w = {};
            *reinterpret_cast<RawW<T, W> *>(out + a) = w;
        }
        j += dj, h += dh, t += dt;
        if (j >= per) j -= per, ++h;
        if (h >= r.heads) h -= r.heads, ++t;
    }
}

// whether pieces of 8 values of 16 bits fit: whole ones in both halves, and 16-byte boundaries everywhere (20000 tokens of 28 heads: 46 us, in pieces of 4 54)
inline bool rope_wide(const RopePlan &p, const RopeRows &r) {
    return p.half % 8 == 0 && (r.dim - 2 * p.half) % 8 == 0 && aligned(r.x, 16) && aligned(r.out, 16) &&
           (r.xt % 8 | r.xh % 8 | r.ot % 8 | r.oh % 8) == 0;
}

// Tokens of a block: of few tokens as many as its threads turn in one go, else four.  32 heads of 128, bf16: 24 tokens one a block 2.1 us, four 3.3; 304 2.4 and 3.6;
// 608 3.6 and 3.5; 2432 9.2 and 9.6.  8 heads (four in one go): 304 tokens 2.1, one a block 2.3; 608 2.2 and 2.8.  7001 tokens of 40 heads: 25.3 four, 26.0 two, 27.9 eight.
inline int rope_tokens(const RopePlan &p, const RopeRows &r) {
    const int pieces = r.heads * (r.dim / (rope_wide(p, r) ? 16 : 8)), most = kRopePairs / p.half < 4 ? kRopePairs / p.half : 4;
    const int go = kRopeThreads / pieces < 1 ? 1 : kRopeThreads / pieces;
    return r.n_tokens <= 4 * sm_count() && go < most ? go : most;
}

}  // namespace mq

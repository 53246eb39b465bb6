// mqd_add.cu -- the residual's addition with RMSNorm and the Q8 plane, and a plane read back as values.
//
//   h = x + res (f32, rounded once to the stream's type),  r = 1 / sqrt(mean(h^2) + eps),  y = (h r) w,  and per 32 values of y
//   d = amax / 127, q = round_half_away(y (1 / d))
//
// The norm needs all of a row before its first code, so the row stays in registers between the two: every value crosses HBM once
// in (x, res) and once out (h, the plane's sections).  The arithmetic after the addition is mq_quantize_q8's (mq_rms.cuh), so the
// plane is the one that it writes for h.
#include "mq_rms.cuh"
#include "mqd.cuh"

namespace mq {
namespace {

// h = x + res of eight values, as it is stored; v: the same widened to f32
template <typename T>
__device__ __forceinline__ void add8(const Raw8<T> &x, const Raw8<T> &res, float (&v)[8], Raw8<T> &h) {
    float a[8], b[8];
    unpack8(x, a);
    unpack8(res, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(a[i], b[i]);
    h = pack8(v, T());
    if constexpr (sizeof(T) == 2) unpack8(h, v);
}

// r from the pairs (hi, lo) that every lane holds of its part of a row; the row's WT warps are `first` .. first + WT - 1 of the block and
// meet at named barrier `bar`.  s_part, s_partd: a slot per warp
__device__ __forceinline__ float row_scale(float2 hi, float2 lo, int64_t K, float eps, int WT, int first, int warp, int lane, int bar,
                                           float2 *s_part, double *s_partd) {
    float th = hi.x, tl = lo.x;
    pair_add(th, tl, hi.y, lo.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float bh = __shfl_xor_sync(kFull, th, o), bl = __shfl_xor_sync(kFull, tl, o);
        pair_add(th, tl, bh, bl);
    }
    if (WT > 1) {
        if (lane == 0) s_part[warp] = make_float2(th, tl);
        named_bar(bar, WT * 32);
        const float2 part = s_part[first + (lane & WT - 1)];   // (WT is a power of two: every lane ends with all of them)
        th = part.x, tl = part.y;
        for (int o = WT >> 1; o > 0; o >>= 1) {
            const float bh = __shfl_xor_sync(kFull, th, o), bl = __shfl_xor_sync(kFull, tl, o);
            pair_add(th, tl, bh, bl);
        }
    }
    float r;
    if (!rms_scale_from_pair(th, tl, K, eps, r)) {          // (the same in all warps of the row)
        double t = ((double)hi.x + (double)lo.x) + ((double)hi.y + (double)lo.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        if (WT > 1) {
            if (lane == 0) s_partd[warp] = t;
            named_bar(bar, WT * 32);
            t = s_partd[first];
            for (int k = 1; k < WT; ++k) t += s_partd[first + k];
        }
        r = 0.0f;
        if (lane == 0) r = (float)(1.0 / sqrt(t / (double)K + (double)eps));
        r = __shfl_sync(kFull, r, 0);
    }
    return r;
}

// y = fl(fl(h r) w) in place
__device__ __forceinline__ void norm8(float (&v)[8], float r, const float *w) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w)), b = __ldg(reinterpret_cast<const float4 *>(w) + 1);
    const float2 r2 = make_float2(r, r), wv[4] = {{a.x, a.y}, {a.z, a.w}, {b.x, b.y}, {b.z, b.w}};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 y = __fmul2_rn(__fmul2_rn(make_float2(v[i], v[i + 1]), r2), wv[i / 2]);
        v[i] = y.x, v[i + 1] = y.y;
    }
}

// One row per group of WT = 2^wt_log2 warps, warp g of it holding chunks g, g + WT, .. of 256 values (at most NC; lane l: values
// 8 l .. 8 l + 7 of each).  Many rows are bound by HBM: 3314 rows of 3584 f32 values with all sections 26.6 us, 6.9 TB/s of the bytes that they move; 9001 rows of 8192 bf16
// values 111 us, 6.3 TB/s.  Fewer 16-bit values are bound by the latency of a row's chain, at 46 % of the warps and 64 % of the issue slots: with all sections about 6 us
// and 6.6 for every 4 M values (4000 rows of 4096 32.6 us, 4.8 TB/s; 16000 112, 5.6; 2000 of 8192 32.4; from 3648 to 4864 rows, 3 to 4 waves, on one line), with q8 alone,
// a quarter of the bytes less, 6.1 (4000 30.0).  The stores of scales and sums, single words in as many sectors, are 4 %.  Three blocks of eight warps an SM (f32) or four (16 bits), so that one row's sums hide under the others' loads; rows that follow one another in
// a resident block, the next on its way, took 56 us for 40 and 175 for 165 (with the plane read back).
template <typename T, int NC, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : sizeof(T) == 4 ? 3 : 4) add_quantize_regs_kernel(AddQuantize a, Plane p, int wt_log2) {
    __shared__ float2 s_part[32];
    __shared__ double s_partd[32];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int WT = 1 << wt_log2, grp = warp >> wt_log2, g = warp & (WT - 1), ngrp = (blockDim.x >> 5) >> wt_log2;
    const int64_t m = (int64_t)blockIdx.x * ngrp + grp;
    if (m >= a.M) return;                                   // (all warps of a group)
    const int nvalid = min(NC, ((int)(a.K / 256) - g + WT - 1) >> wt_log2);
    const T *x = static_cast<const T *>(a.x) + m * a.xs + lane * 8, *res = static_cast<const T *>(a.res) + m * a.rs + lane * 8;
    T *h = static_cast<T *>(a.h) + m * a.hs + lane * 8;
    float v[NC][8];
    Raw8<T> rx[NC], rr[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        rr[j] = {};
        if (j < nvalid) rr[j] = load8(res + (g + j * WT) * 256);
    }
    if (a.x != nullptr) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            rx[j] = {};
            if (j < nvalid) rx[j] = load8(x + (g + j * WT) * 256);
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            Raw8<T> o;
            add8(rx[j], rr[j], v[j], o);
            if (j < nvalid) store8_row(h + (g + j * WT) * 256, o, lane);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NC; ++j) unpack8(rr[j], v[j]);
    }
    float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll
    for (int j = 0; j < NC; ++j)
        if (j < nvalid) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) add_square2(make_float2(v[j][i], v[j][i + 1]), hi, lo);
        }
    const float r = row_scale(hi, lo, a.K, a.eps, WT, grp << wt_log2, warp, lane, 1 + grp, s_part, s_partd);
#pragma unroll
    for (int j = 0; j < NC; ++j)
        if (j < nvalid) norm8(v[j], r, a.w + (g + j * WT) * 256 + lane * 8);
    quantize_chunks<NC>(v, nvalid, g, WT, lane, a.sections, p, a.M, a.K, m);
}

// Rows too long for registers: a block per row, h written in the first pass and read again (from L2, by the warp that wrote it)
// in the second.  4000 rows of 16384 f32 values take 184 us, 5.5 TB/s of the bytes without that second read.
template <typename T>
__global__ void __launch_bounds__(256) add_quantize_kernel(AddQuantize a, Plane p) {
    __shared__ float2 s_part[8];
    __shared__ double s_partd[8];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nch = (int)(a.K / 256);
    const int64_t m = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + m * a.xs + lane * 8, *res = static_cast<const T *>(a.res) + m * a.rs + lane * 8;
    T *h = static_cast<T *>(a.h) + m * a.hs + lane * 8;
    float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll 2
    for (int c = warp; c < nch; c += 8) {
        float v[8];
        if (a.x != nullptr) {
            Raw8<T> o;
            add8(load8(x + (int64_t)c * 256), load8(res + (int64_t)c * 256), v, o);
            store8_row(h + (int64_t)c * 256, o, lane);
        } else {
            unpack8(load8(res + (int64_t)c * 256), v);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) add_square2(make_float2(v[i], v[i + 1]), hi, lo);
    }
    const float r = row_scale(hi, lo, a.K, a.eps, 8, 0, warp, lane, 1, s_part, s_partd);
    const T *again = a.x != nullptr ? h : res;
    for (int c = warp; c < nch; c += 32) {
        const int nvalid = min(4, (nch - c + 7) / 8);
        float v[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Raw8<T> o = {};
            if (j < nvalid) o = load8(again + (int64_t)(c + 8 * j) * 256);
            unpack8(o, v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < nvalid) norm8(v[j], r, a.w + (int64_t)(c + 8 * j) * 256 + lane * 8);
        quantize_chunks<4>(v, nvalid, c, 8, lane, a.sections, p, a.M, a.K, m);
    }
}

template <typename T>
int add_quantize_t(const AddQuantize &a, const Plane &p, cudaStream_t s) {
    const int64_t nch = a.K / 256;
    cudaError_t e = cudaSuccess;
    const int64_t sms = sm_count();
    int wl = 0;
    // Few rows: a warp for every chunk, up to 32 warps and 4 blocks an SM.  Against four chunks a warp (us in a graph, f32): 1 row of 4096 3.4 and 3.9, 152 4.0 and
    // 5.3, 304 5.2 and 5.5, 608 11.0 and 11.2 (bf16 9.5 and 7.0); 608 rows of 1024 3.5 and 5.1, 1216 6.0 and 5.2; 152 of 8192 5.5 and 5.5, 304 11.8 and 11.0.
    if (nch <= 32 && a.M <= 4 * sms && a.M * nch <= 32 * sms) {
        while ((1 << wl) < nch) ++wl;
        e = launch_pdl(add_quantize_regs_kernel<T, 1, 1024>, dim3((unsigned)a.M), dim3(32u << wl), 0, s, a, p, wl);
    } else if (nch <= 32) {
        while ((4 << wl) < nch) ++wl;
        e = launch_pdl(add_quantize_regs_kernel<T, 4, 256>, dim3((unsigned)((a.M + (8 >> wl) - 1) / (8 >> wl))), dim3(256), 0, s, a, p, wl);
    } else if (sizeof(T) == 2 && nch <= 128) {
        // 1000 rows of bf16: of 16384 values 36 us, in the loop 50; of 32768 82 and 93; of 20480 (a warp then holds two or three chunks) 63 and 64.  f32 rows
        // would spill: 58 and 56 at 16384.
        if constexpr (sizeof(T) == 2) {
            while ((4 << wl) < nch) ++wl;
            e = launch_pdl(add_quantize_regs_kernel<T, 4, 1024>, dim3((unsigned)a.M), dim3(32u << wl), 0, s, a, p, wl);
        }
    } else {
        e = launch_pdl(add_quantize_kernel<T>, dim3((unsigned)a.M), dim3(256), 0, s, a, p);
    }
    return cuda_error(e, "mqd_add_quantize_q8 launch");
}

// A warp per row and up to four chunks of 256 values; the eight rows of a block are neighbours, so that a sector of the block-major
// scales serves all of them.  Bound by HBM: 8192 rows of 4096 values from q16 to f32 31 us (6.5 TB/s), from q8 to bf16 17 us (6.0 TB/s).
template <typename T, bool Q16>
__global__ void __launch_bounds__(256) dequantize_kernel(Plane p, int64_t M, int64_t K, T *y, int64_t ys, int groups) {
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nch = (int)(K / 256);
    const int64_t m = (int64_t)(blockIdx.x / groups) * 8 + warp;
    const int c0 = (int)(blockIdx.x % groups) * 4;
    if (m >= M) return;
    uint4 w16[4];
    uint2 w8[4];
    float d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (c0 + j < nch) {
            const int64_t off = m * K + (int64_t)(c0 + j) * 256 + lane * 8;
            if constexpr (Q16) w16[j] = __ldg(reinterpret_cast<const uint4 *>(p.q16 + off));
            else w8[j] = __ldg(reinterpret_cast<const uint2 *>(p.q8 + off));
            d[j] = __ldg(p.d + ((int64_t)(c0 + j) * 8 + (lane >> 2)) * M + m);
        }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (c0 + j < nch) {
            float v[8];
            if constexpr (Q16) {
                unpack8(Raw8<__half>{w16[j]}, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {                // code_value: byte + 128, minus 128
                    v[i] = code_value(w8[j].x ^ 0x80808080u, i);
                    v[4 + i] = code_value(w8[j].y ^ 0x80808080u, i);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], d[j]);
            store8_row(y + m * ys + (int64_t)(c0 + j) * 256 + lane * 8, pack8(v, T()), lane);
        }
}

template <typename T>
int dequantize_t(const Plane &p, int64_t M, int64_t K, bool q16, T *y, int64_t ys, cudaStream_t s) {
    const int groups = (int)((K / 256 + 3) / 4);
    const dim3 grid((unsigned)((M + 7) / 8 * groups));
    return cuda_error(launch_pdl(q16 ? dequantize_kernel<T, true> : dequantize_kernel<T, false>, grid, dim3(256), 0, s, p, M, K, y, ys, groups),
                      "mqd_dequantize_q8 launch");
}

}  // namespace

int launch_add_quantize(const AddQuantize &a, int dtype, const Plane &p, cudaStream_t s) {
    return dtype == MQD_F32   ? add_quantize_t<float>(a, p, s)
           : dtype == MQD_F16 ? add_quantize_t<__half>(a, p, s)
                              : add_quantize_t<__nv_bfloat16>(a, p, s);
}

int launch_dequantize(const Plane &p, int64_t M, int64_t K, bool q16, int dtype, void *y, int64_t ys, cudaStream_t s) {
    return dtype == MQD_F32   ? dequantize_t(p, M, K, q16, static_cast<float *>(y), ys, s)
           : dtype == MQD_F16 ? dequantize_t(p, M, K, q16, static_cast<__half *>(y), ys, s)
                              : dequantize_t(p, M, K, q16, static_cast<__nv_bfloat16 *>(y), ys, s);
}

}  // namespace mq

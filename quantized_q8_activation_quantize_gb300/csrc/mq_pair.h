// mq_pair.h -- f32 operations with one rounding each that no compiler contracts or reassociates, and the error-free sum (plain C++: the tests compile
// it for the host, with contraction off).
#pragma once

#include <cmath>

#ifdef __CUDACC__
#define MQ_PAIR __host__ __device__ __forceinline__
#else
#define MQ_PAIR inline
#endif

namespace mq {

#ifdef __CUDA_ARCH__
MQ_PAIR float add_rn(float a, float b) { return __fadd_rn(a, b); }
MQ_PAIR float sub_rn(float a, float b) { return __fsub_rn(a, b); }
MQ_PAIR float mul_rn(float a, float b) { return __fmul_rn(a, b); }
MQ_PAIR float div_rn(float a, float b) { return __fdiv_rn(a, b); }
MQ_PAIR float fma_rn(float a, float b, float c) { return __fmaf_rn(a, b, c); }
#else
MQ_PAIR float add_rn(float a, float b) { return a + b; }
MQ_PAIR float sub_rn(float a, float b) { return a - b; }
MQ_PAIR float mul_rn(float a, float b) { return a * b; }
MQ_PAIR float div_rn(float a, float b) { return a / b; }
MQ_PAIR float fma_rn(float a, float b, float c) { return fmaf(a, b, c); }
#endif

// Error-free sum a + b = s + e (Knuth's two-sum, branch-free, any order of magnitudes).
MQ_PAIR void two_sum(float a, float b, float &s, float &e) {
    s = add_rn(a, b);
    const float bv = sub_rn(s, a);
    e = add_rn(sub_rn(a, sub_rn(s, bv)), sub_rn(b, bv));
}

}  // namespace mq

// mqd_beam_merge.h -- what beam search's join compares, and how it merges sorted lists (plain C++: the tests compile it for the host).
#pragma once

#include <cfloat>
#include <cstdint>
#include <cstring>

#include "mq_pair.h"

namespace mq {

MQ_PAIR uint32_t float_bits(float x) {
#ifdef __CUDA_ARCH__
    return __float_as_uint(x);
#else
    uint32_t u;
    std::memcpy(&u, &x, sizeof u);
    return u;
#endif
}
MQ_PAIR float bits_float(uint32_t u) {
#ifdef __CUDA_ARCH__
    return __uint_as_float(u);
#else
    float x;
    std::memcpy(&x, &u, sizeof x);
    return x;
#endif
}

// order of f32 values (no NaN; +-0 are to be made one before) as unsigned integers, and back
MQ_PAIR uint32_t ordered(float x) {
    const uint32_t u = float_bits(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MQ_PAIR float from_ordered(uint32_t u) { return bits_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// ln(sh + sl) of a positive normal number, as a pair: 2^n f with f in [0.7, 1.42), ln f = 2 (t + t^3 / 3 + .. ) with t = (f - 1) / (f + 1) as a pair; the
// series from t^3 on, in f32, is off by 2e-9 at most.  (The f64 pipe of this GPU issues ~1.7 operations per clock per SM: log() of a double for every row, with scores in f64
// below, took ten times the rest of the join.)
MQ_PAIR void pair_log(float sh, float sl, float &h, float &l) {
    const int n = (int)((float_bits(sh) - 0x3f333333u) >> 23) - (float_bits(sh) < 0x3f333333u ? 512 : 0);
    const float scale = bits_float((uint32_t)(127 - n) << 23);
    const float fh = mul_rn(sh, scale), fl = mul_rn(sl, scale), num = sub_rn(fh, 1.0f);
    float dh, de;
    two_sum(fh, 1.0f, dh, de);
    const float t = div_rn(num, dh);
    const float r = add_rn(fma_rn(-t, dh, num), fma_rn(-t, add_rn(de, fl), fl));
    const float t1 = div_rn(r, dh), z = mul_rn(t, t);
    float p = 1.0f / 11.0f;
    p = fma_rn(p, z, 1.0f / 9.0f);
    p = fma_rn(p, z, 1.0f / 7.0f);
    p = fma_rn(p, z, 1.0f / 5.0f);
    p = fma_rn(p, z, 1.0f / 3.0f);
    const float nf = (float)n;
    two_sum(mul_rn(nf, 0.693145751953125f), mul_rn(2.0f, t), h, l);         // ln 2 in two parts, the product with the first exact
    l = add_rn(l, fma_rn(nf, 1.42860682e-6f, mul_rn(2.0f, fma_rn(mul_rn(t, z), p, t1))));
}

// A candidate's score cum + x - (lh + ll) as an f32 pair (the rounded sum, the rest: 48 bits) in the order of unsigned integers (0: none).  Nearly in the order
// of x: where x - lh passes a rounding border of f32, the rest is rounded on another grid, and of two neighbouring x the larger can get a key that is lower by
// about 2^-24 of the rest.
MQ_PAIR uint64_t score_key(float cum, float x, float lh, float ll) {
    float d, e, h, l;
    two_sum(x, -lh, d, e);                                      // (|x| and the logarithm may be far apart either way)
    e = sub_rn(e, ll);
    two_sum(cum, d, h, l);
    const bool fits = fabsf(h) <= FLT_MAX;                      // (past f32 there is no rest)
    l = fits ? add_rn(l, e) : 0.0f;
    h = fabsf(cum) <= FLT_MAX ? h : cum;                        // (+inf, a beam's own, stays beside a difference past f32)
    const float s = add_rn(h, l);
    l = fits ? sub_rn(l, sub_rn(s, h)) : 0.0f;
    return ((uint64_t)ordered(add_rn(s, 0.0f)) << 32) | ordered(add_rn(l, 0.0f));
}

// One round of merging runs of k keys in pairs (a and a ^ 1; run a begins at key a * s * k; zeros, no entry, at its end): where in the next buffer entry j of run a goes,
// -1: it is not among the pair's best k.  Of equals those of the earlier run come first.  Every run has to be in falling order: then the entries of a pair go to places
// of their own and fill its k; else two could share one and leave another unwritten.
MQ_PAIR int merge_slot(const uint64_t *key, int runs, int s, int k, int a, int j) {
    const uint64_t x = key[a * s * k + j];
    int lo = 0;
    if ((a ^ 1) < runs) {
        // before it in the other run: what is better, of an earlier run what is equal too
        const uint64_t *other = key + (a ^ 1) * s * k, bar = x - (a & 1);
        for (int hi = k - j; lo < hi;) {                        // (past k - j it is out in any case)
            const int mid = (lo + hi) >> 1;
            if (other[mid] > bar) lo = mid + 1;
            else hi = mid;
        }
    }
    return j + lo < k && (x != 0 || (a & 1) == 0) ? (a & ~1) * s * k + j + lo : -1;         // (an earlier run's room without an entry is what is left)
}

}  // namespace mq

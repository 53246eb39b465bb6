// mqd_abi.cu -- the C ABI of include/mqd.h: argument checks on the host, the turns of a rotation.
#include <cmath>
#include <cstring>

#include "mqd.cuh"

#define MQD_TRY(e)                      \
    do {                                \
        const int rc_ = (e);            \
        if (rc_ != MQ_OK) return rc_;   \
    } while (0)

namespace mq {
namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

int type_bytes(int32_t dtype) { return dtype == MQD_F32 ? 4 : dtype == MQD_F16 || dtype == MQD_BF16 ? 2 : 0; }

int check_type(const char *fn, int32_t dtype) {
    return type_bytes(dtype) ? MQ_OK : set_error(MQ_ERR_ARG, "%s: dtype=%d not one of mqd_dtype", fn, dtype);
}

// a [M][K] tensor of rows `stride` apart, in pieces of 8 values
int check_rows(const char *fn, const char *what, const void *p, int64_t stride, int64_t K) {
    if (p == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL %s", fn, what);
    if (!aligned(p, 16) || stride % 8 != 0)
        return set_error(MQ_ERR_ALIGN, "%s: %s %p not 16-byte aligned or its stride %lld no multiple of 8", fn, what, p, (long long)stride);
    if (stride < K || stride > ((int64_t)1 << 40))
        return set_error(MQ_ERR_ARG, "%s: stride %lld of %s below K=%lld or past 2^40", fn, (long long)stride, what, (long long)K);
    return MQ_OK;
}
size_t rows_span(int64_t M, int64_t K, int64_t stride, int32_t dtype) { return ((size_t)(M - 1) * (size_t)stride + (size_t)K) * type_bytes(dtype); }

int check_rot(const char *fn, int32_t rot_dim) {
    return rot_dim >= 8 && rot_dim <= 1024 && rot_dim % 8 == 0 ? MQ_OK : set_error(MQ_ERR_SHAPE, "%s: rot_dim=%d not a multiple of 8 from 8 to 1024", fn, rot_dim);
}

int check_beams(const char *fn, int64_t n_groups, int32_t n_beams, int64_t vocab, int32_t n_cand) {
    if (n_groups < 0 || vocab < 0) return set_error(MQ_ERR_ARG, "%s: negative n_groups=%lld or vocab=%lld", fn, (long long)n_groups, (long long)vocab);
    if (n_beams < 1 || n_beams > 64 || n_cand < 1 || n_cand > 64)
        return set_error(MQ_ERR_SHAPE, "%s: n_beams=%d or n_cand=%d not in 1 .. 64", fn, n_beams, n_cand);
    if (n_groups >= (1 << 24) || n_groups * n_beams >= (1 << 24) || vocab >= kMaxDim - 65536)
        return set_error(MQ_ERR_SHAPE, "%s: n_groups * n_beams = %lld * %d must be below 2^24, vocab=%lld below 2^31 - 2^16", fn, (long long)n_groups, n_beams, (long long)vocab);
    return MQ_OK;
}

}  // namespace

// whether the values of two [n][width] tensors of the given token strides are surely apart: their spans are, or both have one stride and their rows'
// places in it do not meet
bool values_apart(const void *a, size_t na, int64_t as, int64_t aw, const void *b, size_t nb, int64_t bs, int64_t bw, int64_t n, int32_t dtype) {
    if (!overlaps(a, na, b, nb)) return true;
    if (n <= 1 || as != bs || as <= 0) return false;
    const int64_t size = type_bytes(dtype), s = as * size;
    int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) % s;
    if (d < 0) d += s;
    return aw * size <= d && d + bw * size <= s;
}

int rope_plan_of(const char *fn, const mqd_rope_plan *plan, int32_t head_dim, RopePlan *out) {
    if (plan == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL plan", fn);
    MQD_TRY(check_rot(fn, plan->rot_dim));
    if (head_dim < plan->rot_dim) return set_error(MQ_ERR_SHAPE, "%s: head_dim=%d below rot_dim=%d", fn, head_dim, plan->rot_dim);
    if (!std::isfinite(plan->amplitude)) return set_error(MQ_ERR_ARG, "%s: amplitude=%g not finite", fn, (double)plan->amplitude);
    if (plan->turns == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL turns", fn);
    if (!aligned(plan->turns, 8)) return set_error(MQ_ERR_ALIGN, "%s: turns %p not 8-byte aligned", fn, (const void *)plan->turns);
    *out = RopePlan{plan->turns, plan->rot_dim / 2, plan->interleaved != 0, plan->amplitude};
    return MQ_OK;
}

int check_rope_heads(const char *fn, const char *what, const void *p, int64_t ts, int64_t hs, int32_t dtype) {
    if (p == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL %s", fn, what);
    if (!aligned(p, 4 * type_bytes(dtype)) || ts % 4 != 0 || hs % 4 != 0)
        return set_error(MQ_ERR_ALIGN, "%s: %s %p (strides %lld, %lld) not aligned to 4 elements", fn, what, p, (long long)ts, (long long)hs);
    if (ts < 0 || hs < 0 || ts > ((int64_t)1 << 31) || hs > ((int64_t)1 << 31))
        return set_error(MQ_ERR_ARG, "%s: strides %lld, %lld of %s not in 0 .. 2^31", fn, (long long)ts, (long long)hs, what);
    return MQ_OK;
}

size_t heads_span(int64_t n, int64_t heads, int64_t dim, int64_t ts, int64_t hs, int32_t dtype) {
    return n == 0 ? 0 : (size_t)((n - 1) * ts + (heads - 1) * hs + dim) * type_bytes(dtype);
}

int check_rope_out(const char *fn, const void *x, int64_t xt, int64_t xh, const void *out, int64_t ot, int64_t oh, int64_t n, int64_t heads, int64_t dim,
                   int32_t dtype) {
    const bool apart = n <= 1 && heads <= 1 ? true
                       : heads <= 1         ? ot >= dim
                       : n <= 1             ? oh >= dim
                                            : (oh >= dim && ot >= (heads - 1) * oh + dim) || (ot >= dim && oh >= (n - 1) * ot + dim);
    if (!apart) return set_error(MQ_ERR_ARG, "%s: heads of out overlap (strides %lld, %lld)", fn, (long long)ot, (long long)oh);
    if (!values_apart(out, heads_span(n, heads, dim, ot, oh, dtype), ot, (heads - 1) * oh + dim, x, heads_span(n, heads, dim, xt, xh, dtype), xt,
                      (heads - 1) * xh + dim, n, dtype) &&
        !(out == x && ot == xt && oh == xh))
        return set_error(MQ_ERR_ARG, "%s: out %p overlaps the input %p without being it", fn, out, x);
    return MQ_OK;
}

}  // namespace mq

using namespace mq;

extern "C" {

int mqd_add_quantize_q8(int32_t dtype, const void *x, int64_t x_stride, const void *res, int64_t res_stride, void *h, int64_t h_stride,
                        int64_t M, int64_t K, const float *rms_w, float eps, unsigned sections, void *plane, mq_stream_t stream) {
    const char *fn = "mqd_add_quantize_q8";
    MQD_TRY(check_type(fn, dtype));
    if (sections == 0 || sections > MQ_PLANE_ALL) return set_error(MQ_ERR_ARG, "%s: sections=0x%x not a non-empty MQ_PLANE_* mask", fn, sections);
    if (M < 0) return set_error(MQ_ERR_ARG, "%s: negative M=%lld", fn, (long long)M);
    MQD_TRY(check_k(K));
    if (M >= kMaxDim) return set_error(MQ_ERR_SHAPE, "%s: M=%lld must be below 2^31", fn, (long long)M);
    if (!(std::isfinite(eps) && eps >= 0.0f)) return set_error(MQ_ERR_ARG, "%s: eps=%g must be finite and >= 0", fn, (double)eps);
    if (M == 0) return MQ_OK;
    MQD_TRY(check_rows(fn, "res", res, res_stride, K));
    if (x != nullptr) {
        MQD_TRY(check_rows(fn, "x", x, x_stride, K));
        MQD_TRY(check_rows(fn, "h", h, h_stride, K));
    }
    if (rms_w == nullptr || plane == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL pointer (rms_w=%p plane=%p)", fn, (const void *)rms_w, plane);
    if (!aligned(rms_w, 16)) return set_error(MQ_ERR_ALIGN, "%s: rms_w %p not 16-byte aligned", fn, (const void *)rms_w);
    if (!aligned(plane, 256)) return set_error(MQ_ERR_ALIGN, "%s: plane %p not 256-byte aligned", fn, plane);
    const size_t pb = mq_q8_plane_bytes(M, K), wb = (size_t)K * 4, rb = rows_span(M, K, res_stride, dtype),
                 xb = x != nullptr ? rows_span(M, K, x_stride, dtype) : 0, hb = x != nullptr ? rows_span(M, K, h_stride, dtype) : 0;
    if (overlaps(plane, pb, x, xb) || overlaps(plane, pb, res, rb) || overlaps(plane, pb, h, hb) || overlaps(plane, pb, rms_w, wb))
        return set_error(MQ_ERR_ARG, "%s: plane %p overlaps x %p, res %p, h %p or rms_w %p", fn, plane, x, res, h, (const void *)rms_w);
    if (overlaps(h, hb, rms_w, wb) || (!values_apart(h, hb, h_stride, K, x, xb, x_stride, K, M, dtype) && !(h == x && h_stride == x_stride)) ||
        (!values_apart(h, hb, h_stride, K, res, rb, res_stride, K, M, dtype) && !(h == res && h_stride == res_stride)))
        return set_error(MQ_ERR_ARG, "%s: h %p overlaps rms_w %p, or x %p or res %p without being it", fn, h, (const void *)rms_w, x, res);
    unsigned int *err = nullptr;
    MQD_TRY(device_state(&err));
    Plane p;
    plane_from(plane, M, K, &p);
    return launch_add_quantize(AddQuantize{x, res, h, x_stride, res_stride, h_stride, M, K, rms_w, eps, sections}, dtype, p,
                               reinterpret_cast<cudaStream_t>(stream));
}

int mqd_dequantize_q8(const void *plane, int64_t M, int64_t K, unsigned sections, int32_t dtype, void *y, int64_t y_stride,
                      mq_stream_t stream) {
    const char *fn = "mqd_dequantize_q8";
    MQD_TRY(check_type(fn, dtype));
    if (sections > MQ_PLANE_ALL || (sections & (MQ_PLANE_Q16 | MQ_PLANE_Q8)) == 0)
        return set_error(MQ_ERR_ARG, "%s: sections=0x%x has no codes (MQ_PLANE_Q16 or MQ_PLANE_Q8)", fn, sections);
    if (M < 0) return set_error(MQ_ERR_ARG, "%s: negative M=%lld", fn, (long long)M);
    MQD_TRY(check_k(K));
    if (M >= kMaxDim || (M + 7) / 8 * ((K / 256 + 3) / 4) >= kMaxDim)
        return set_error(MQ_ERR_SHAPE, "%s: M=%lld, K=%lld beyond 2^31 rows or pieces", fn, (long long)M, (long long)K);
    if (M == 0) return MQ_OK;
    if (plane == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL plane", fn);
    if (!aligned(plane, 256)) return set_error(MQ_ERR_ALIGN, "%s: plane %p not 256-byte aligned", fn, plane);
    MQD_TRY(check_rows(fn, "y", y, y_stride, K));
    if (overlaps(plane, mq_q8_plane_bytes(M, K), y, rows_span(M, K, y_stride, dtype)))
        return set_error(MQ_ERR_ARG, "%s: y %p overlaps the plane %p", fn, y, plane);
    unsigned int *err = nullptr;
    MQD_TRY(device_state(&err));
    Plane p;
    plane_from(const_cast<void *>(plane), M, K, &p);
    return launch_dequantize(p, M, K, (sections & MQ_PLANE_Q16) != 0, dtype, y, y_stride, reinterpret_cast<cudaStream_t>(stream));
}

int mqd_rope_turns(int32_t rot_dim, double base, int32_t scaling, double factor, double original, double low, double high, const double *factors,
                   uint64_t *turns) {
    const char *fn = "mqd_rope_turns";
    if (turns == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL output", fn);
    MQD_TRY(check_rot(fn, rot_dim));
    if (!(std::isfinite(base) && base > 1.0)) return set_error(MQ_ERR_ARG, "%s: base=%g must be finite and above 1", fn, base);
    if (scaling < MQD_ROPE_NONE || scaling > MQD_ROPE_INDEX) return set_error(MQ_ERR_ARG, "%s: scaling=%d not one of mqd_rope_scaling", fn, scaling);
    if (!(std::isfinite(factor) && factor >= 1.0)) return set_error(MQ_ERR_ARG, "%s: factor=%g must be finite and at least 1", fn, factor);
    const bool ramp = scaling == MQD_ROPE_TURNS || scaling == MQD_ROPE_INDEX;
    if (ramp && !(std::isfinite(original) && original > 0.0 && std::isfinite(high) && low > 0.0 && low < high))
        return set_error(MQ_ERR_ARG, "%s: original=%g must be positive, and 0 < low=%g < high=%g", fn, original, low, high);
    const double two_pi = 6.283185307179586476925286766559, n = rot_dim;
    if (scaling == MQD_ROPE_BASE) base *= std::pow(factor, n / (n - 2.0));
    if (!std::isfinite(base)) return set_error(MQ_ERR_ARG, "%s: factor=%g takes the base past the range of a double", fn, factor);
    const auto pair_of = [&](double t) { return n * std::log(original / (two_pi * t)) / (2.0 * std::log(base)); };
    double i0 = 0.0, i1 = 0.0;
    if (scaling == MQD_ROPE_INDEX) {
        i0 = std::fmax(std::floor(pair_of(high)), 0.0);
        i1 = std::fmin(std::ceil(pair_of(low)), n - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / n);
        if (scaling == MQD_ROPE_LINEAR) f /= factor;
        if (ramp) {
            double w = scaling == MQD_ROPE_TURNS ? (original * f / two_pi - low) / (high - low) : 1.0 - (i - i0) / std::fmax(i1 - i0, 0.001);
            w = std::fmin(std::fmax(w, 0.0), 1.0);
            f *= w + (1.0 - w) / factor;
        }
        if (factors != nullptr) {
            if (!(std::isfinite(factors[i]) && factors[i] > 0.0)) return set_error(MQ_ERR_ARG, "%s: factors[%d]=%g must be finite and positive", fn, i, factors[i]);
            f /= factors[i];
        }
        const double t = f / two_pi;
        if (!(t < 1.0)) return set_error(MQ_ERR_ARG, "%s: pair %d would turn %g times per position, below 1 wanted", fn, i, t);
        turns[i] = (uint64_t)std::ldexp(t, 64);                 // (t has 53 bits: below 2^64)
    }
    return MQ_OK;
}

int mqd_rope(const mqd_rope_plan *plan, int32_t dtype, const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
             int64_t out_token_stride, int64_t out_head_stride, int64_t n_tokens, int32_t n_heads, int32_t head_dim, const int32_t *pos,
             mq_stream_t stream) {
    const char *fn = "mqd_rope";
    MQD_TRY(check_type(fn, dtype));
    RopePlan p;
    MQD_TRY(rope_plan_of(fn, plan, head_dim, &p));
    if (head_dim > 1024 || head_dim % 8 != 0) return set_error(MQ_ERR_SHAPE, "%s: head_dim=%d not a multiple of 8 of at most 1024", fn, head_dim);
    if (n_tokens < 0 || n_heads < 0) return set_error(MQ_ERR_ARG, "%s: negative n_tokens=%lld or n_heads=%d", fn, (long long)n_tokens, n_heads);
    if (n_tokens >= kMaxDim || n_heads > 65536)
        return set_error(MQ_ERR_SHAPE, "%s: n_tokens=%lld not below 2^31 or n_heads=%d above 65536", fn, (long long)n_tokens, n_heads);
    if (n_tokens == 0 || n_heads == 0) return MQ_OK;
    if (pos == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL pos", fn);
    if (!aligned(pos, 4)) return set_error(MQ_ERR_ALIGN, "%s: pos %p not 4-byte aligned", fn, (const void *)pos);
    MQD_TRY(check_rope_heads(fn, "x", x, x_token_stride, x_head_stride, dtype));
    MQD_TRY(check_rope_heads(fn, "out", out, out_token_stride, out_head_stride, dtype));
    MQD_TRY(check_rope_out(fn, x, x_token_stride, x_head_stride, out, out_token_stride, out_head_stride, n_tokens, n_heads, head_dim, dtype));
    const size_t ob = heads_span(n_tokens, n_heads, head_dim, out_token_stride, out_head_stride, dtype);
    if (overlaps(out, ob, pos, (size_t)n_tokens * 4) || overlaps(out, ob, plan->turns, (size_t)plan->rot_dim * 4))
        return set_error(MQ_ERR_ARG, "%s: out %p overlaps pos %p or the turns %p", fn, out, (const void *)pos, (const void *)plan->turns);
    unsigned int *err = nullptr;
    MQD_TRY(device_state(&err));
    return launch_rope(p, RopeRows{x, out, x_token_stride, x_head_stride, out_token_stride, out_head_stride, n_tokens, n_heads, head_dim, 1}, dtype, pos,
                       reinterpret_cast<cudaStream_t>(stream));
}

size_t mqd_beam_workspace_bytes(int64_t n_groups, int32_t n_beams, int64_t vocab, int32_t n_cand) {
    if (check_beams("mqd_beam_workspace_bytes", n_groups, n_beams, vocab, n_cand) != MQ_OK) return 0;
    return n_groups == 0 ? 256 : beam_ws(n_groups, n_beams, vocab, n_cand);
}

int mqd_beam_select(int32_t dtype, const void *logits, int64_t row_stride, int64_t n_groups, int32_t n_beams, int64_t vocab, const float *scores,
                    int32_t n_cand, int32_t stop, float *cand_score, int32_t *cand_row, int32_t *cand_token, float *next_score, int32_t *next_row,
                    int32_t *next_token, void *workspace, size_t workspace_bytes, mq_stream_t stream) {
    const char *fn = "mqd_beam_select";
    MQD_TRY(check_type(fn, dtype));
    MQD_TRY(check_beams(fn, n_groups, n_beams, vocab, n_cand));
    if (stop < -1) return set_error(MQ_ERR_ARG, "%s: stop=%d is neither a token nor -1", fn, stop);
    if (row_stride < vocab || row_stride > ((int64_t)1 << 38))
        return set_error(MQ_ERR_ARG, "%s: row_stride=%lld below vocab=%lld or past 2^38", fn, (long long)row_stride, (long long)vocab);
    if (n_groups == 0) return MQ_OK;
    if (vocab == 0) return set_error(MQ_ERR_SHAPE, "%s: vocab=0", fn);
    const int size = type_bytes(dtype);
    if (!logits || !scores || !cand_score || !cand_row || !cand_token)
        return set_error(MQ_ERR_ARG, "%s: NULL pointer (logits=%p scores=%p cand=%p %p %p)", fn, logits, (const void *)scores, (void *)cand_score, (void *)cand_row, (void *)cand_token);
    const bool next = next_score || next_row || next_token;
    if (next && !(next_score && next_row && next_token)) return set_error(MQ_ERR_ARG, "%s: next_score, next_row, next_token are all given or none", fn);
    if (!aligned(logits, size) || !aligned(scores, 4) || !aligned(cand_score, 4) || !aligned(cand_row, 4) || !aligned(cand_token, 4) ||
        !aligned(next_score, 4) || !aligned(next_row, 4) || !aligned(next_token, 4))
        return set_error(MQ_ERR_ALIGN, "%s: a pointer is not aligned to its elements (logits=%p)", fn, logits);
    const size_t want = mqd_beam_workspace_bytes(n_groups, n_beams, vocab, n_cand);
    if (workspace == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL workspace", fn);
    if (!aligned(workspace, 256)) return set_error(MQ_ERR_ALIGN, "%s: workspace %p not 256-byte aligned", fn, workspace);
    if (workspace_bytes < want) return set_error(MQ_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, want);
    const size_t rows = (size_t)n_groups * n_beams, lb = ((rows - 1) * (size_t)row_stride + (size_t)vocab) * size, cb = (size_t)n_groups * n_cand * 4, nb = next ? rows * 4 : 0;
    // what is written, then what is read
    const struct {
        const void *p;
        size_t n;
    } all[9] = {{cand_score, cb}, {cand_row, cb}, {cand_token, cb}, {next_score, nb}, {next_row, nb}, {next_token, nb}, {workspace, want}, {logits, lb}, {scores, rows * 4}};
    for (int i = 0; i < 7; ++i)
        for (int j = i + 1; j < 9; ++j)
            if (overlaps(all[i].p, all[i].n, all[j].p, all[j].n) && !(i == 3 && j == 8 && next_score == scores))
                return set_error(MQ_ERR_ARG, "%s: an output or the workspace (%p) overlaps another tensor of the call (%p)", fn, all[i].p, all[j].p);
    unsigned int *err = nullptr;
    MQD_TRY(device_state(&err));
    return launch_beam_select(dtype, logits, row_stride, n_groups, n_beams, vocab, scores, n_cand, stop, cand_score, cand_row, cand_token, next_score, next_row,
                              next_token, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

/*
 * mqd.h -- C ABI of what a decoder layer does between its matrix products (mq.h) and its cache (mqkv.h), and of what picks
 * the tokens at its end (GB300, sm_103a; same library):
 *   the residual's addition with RMSNorm and the Q8 plane, and a plane read back;
 *   rotary positions (with the cache's append: mqkv_append_rope in mqkv.h);
 *   beam search's selection over beams and vocabulary (the cache's rows follow with mqkv_reorder).
 *
 * Conventions: those of mq.h (device pointers owned by the caller unless stated, asynchronous on the stream, host checks
 * before any launch, mq_last_error() names the values, no fallback).  Strides are in elements.
 */
#ifndef MQD_H
#define MQD_H

#include "mq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MQD_F32 = 0, MQD_F16 = 1, MQD_BF16 = 2 } mqd_dtype;  /* the numbers of mqkv_dtype */

/* ------------------------------------------------- residual, RMSNorm, Q8 plane ---
 *
 * mqd_add_quantize_q8 -- h = x + res, and the Q8 plane of RMSNorm(h): what follows every attention and every FFN block.
 *
 *   dtype      of x, res and h
 *   x          [M][K], the block's output; NULL: nothing is added, h is not written and the norm is of res (a layer
 *              stack's first norm in 16 bits)
 *   res        [M][K], the residual stream
 *   h          [M][K] output, x + res in f32 rounded once to dtype; may be res or x itself (same pointer and stride),
 *              and otherwise may not overlap them (rows of one buffer and one stride, side by side, do not); ignored where x
 *              is NULL
 *   *_stride   of rows, at least K and multiples of 8; bases 16-byte aligned
 *   rms_w      f32 [K], 16-byte aligned
 *   eps, sections, plane   as mq_quantize_q8_ex
 *
 * The plane holds what mq_quantize_q8_ex writes for h (as it is stored, widened to f32), rms_w and eps: the same bits, but
 * for about one row in 10^7, whose r lies within the f64 sums' own rounding of an f32 border.
 * K as in mq.h (a positive multiple of 256); M below 2^31, M == 0 is an empty call.
 */
MQ_API int mqd_add_quantize_q8(int32_t dtype, const void *x, int64_t x_stride, const void *res, int64_t res_stride, void *h,
                               int64_t h_stride, int64_t M, int64_t K, const float *rms_w, float eps, unsigned sections,
                               void *plane, mq_stream_t stream);

/*
 * mqd_dequantize_q8 -- the values q * d of a plane, dense, rounded once to dtype (to f16, values past its range become
 * infinities, as in any conversion): the normed activations for what does not multiply planes (a router, an adapter, an
 * embedding's output).
 *
 *   sections   what the plane holds; its q16 is read where it has MQ_PLANE_Q16, else its q8 (one of the two is needed)
 *   y          [M][K] of dtype, y_stride at least K and a multiple of 8, base 16-byte aligned
 */
MQ_API int mqd_dequantize_q8(const void *plane, int64_t M, int64_t K, unsigned sections, int32_t dtype, void *y,
                             int64_t y_stride, mq_stream_t stream);

/* ------------------------------------------------------------ rotary positions ---
 *
 * The first rot_dim values of a head are rot_dim / 2 pairs; pair i of a token at position p is turned by the angle p f_i
 * and multiplied by the amplitude a:  (u, v) -> a (u cos - v sin, v cos + u sin).  Values past rot_dim stay as they are.
 *   interleaved = 0:  pair i is values i and i + rot_dim / 2;     1: values 2 i and 2 i + 1
 *
 * An angle matters modulo a turn only, so f_i is kept as turns per position in 64-bit fixed point, F_i = 2^64 f_i / (2 pi) (a double's 53
 * bits of it), and p F_i modulo 2^64 is exact: far positions lose nothing.
 */
typedef enum {
    MQD_ROPE_NONE = 0,    /* f_i = base^(-2 i / rot_dim) */
    MQD_ROPE_LINEAR = 1,  /* f_i / factor */
    MQD_ROPE_BASE = 2,    /* base * factor^(rot_dim / (rot_dim - 2)) in place of base */
    MQD_ROPE_TURNS = 3,   /* f_i (w + (1 - w) / factor), w = clamp((n_i - low) / (high - low), 0, 1), n_i = original f_i / (2 pi)
                             the turns of pair i over the original length */
    MQD_ROPE_INDEX = 4    /* the same with w = 1 - clamp((i - i0) / max(i1 - i0, 0.001), 0, 1), i0 = max(floor(g(high)), 0), i1 =
                             min(ceil(g(low)), rot_dim - 1), g(n) = rot_dim ln(original / (2 pi n)) / (2 ln base) the pair that turns n times */
} mqd_rope_scaling;

/* Fills turns[rot_dim / 2] (HOST memory) with F_i; the caller copies it to the device.  rot_dim: a multiple of 8 from 8 to 1024; base > 1;
 * factor >= 1; original > 0 and 0 < low < high for the last two.  factors: NULL or HOST [rot_dim / 2] > 0, by which f_i is divided at the
 * end (a model's own table).  MQ_ERR_ARG for other values, where MQD_ROPE_BASE's base passes the
 * range of a double, or where a pair would turn a whole turn or more per position.
 * Host-only. */
MQ_API int mqd_rope_turns(int32_t rot_dim, double base, int32_t scaling, double factor, double original, double low, double high,
                          const double *factors, uint64_t *turns);

typedef struct {
    const uint64_t *turns;  /* device [rot_dim / 2], 8-byte aligned (mqd_rope_turns) */
    int32_t rot_dim;        /* a multiple of 8 from 8 to 1024 */
    int32_t interleaved;
    float amplitude;        /* finite */
} mqd_rope_plan;            /* a host struct, read during the call only */

/*
 * mqd_rope -- out = x with the first rot_dim values of every head turned, in f32, rounded once to dtype.
 *
 *   x, out     [n_tokens][n_heads][head_dim] of dtype, head_dim a multiple of 8 from 8 to 1024 and at least rot_dim, values of a
 *              head contiguous, strides multiples of 4 (of x: 0 repeats), bases aligned to 4 elements; out may be x (same pointer and
 *              strides), and otherwise may not overlap it (tokens of one buffer and one stride, side by side, do not).  Fewer than
 *              2^31 tokens, up to 65536 heads
 *   pos        int32 [n_tokens], any sign (a negative one turns back)
 */
MQ_API int mqd_rope(const mqd_rope_plan *plan, int32_t dtype, const void *x, int64_t x_token_stride, int64_t x_head_stride,
                    void *out, int64_t out_token_stride, int64_t out_head_stride, int64_t n_tokens, int32_t n_heads,
                    int32_t head_dim, const int32_t *pos, mq_stream_t stream);

/* --------------------------------------------------------------- beam search ---
 *
 * mqd_beam_select -- one step of beam search.  Row r = g * n_beams + b of the logits belongs to beam b of group g; the
 * continuation of row r by token t has the score  scores[r] + logits[r][t] - ln sum_t' exp(logits[r][t']).
 *
 *   logits     [n_groups * n_beams][vocab] of dtype, rows row_stride >= vocab apart, aligned to one element.  A NaN counts as
 *              -inf, +inf as the largest finite f32
 *   scores     f32 [n_groups][n_beams], the beams' own; -inf (or a NaN): a beam that is not alive; of one of +inf every candidate has +inf
 *   n_cand     candidates per group, 1 .. 64
 *   cand_*     [n_groups][n_cand]: the best continuations of each group, the best first: score, row, token.  Of equal scores the lowest
 *              row, then the lowest token comes first; tokens of -inf and rows without a finite logit continue nothing; where there are
 *              fewer, the rest has score -inf, row -1, token -1
 *   next_*     NULL (all three), or [n_groups][n_beams]: the first n_beams candidates whose token is not `stop`, filled up in the same
 *              way (n_cand = 2 n_beams always suffices for one stop token: each beam ends at most once).  next_score may be scores
 *   stop       the token that ends a sequence, or -1
 *   workspace  mqd_beam_workspace_bytes(...) bytes, 256-byte aligned, not shared by calls in flight
 *
 * Scores are compared as f32 pairs (48 bits: two beams' continuations may differ by less than an f32 step) and returned rounded to f32; of
 * those that agree in all 48 bits, tokens of one row may come in the order of their logits, and two tokens of one row whose scores agree within 1e-9 in either
 * order.  A row's logarithm is made of f32 exponentials: off by about 1e-7 where logits differ from one another, by up to 1e-6
 * where one value fills a row below a peak (the exponentials' errors then all go the same way), and by less than 8e-6 whatever the row.
 * n_beams 1 .. 64, n_groups * n_beams < 2^24, vocab < 2^31 - 2^16.
 */
MQ_API size_t mqd_beam_workspace_bytes(int64_t n_groups, int32_t n_beams, int64_t vocab, int32_t n_cand);
MQ_API int mqd_beam_select(int32_t dtype, const void *logits, int64_t row_stride, int64_t n_groups, int32_t n_beams, int64_t vocab,
                           const float *scores, int32_t n_cand, int32_t stop, float *cand_score, int32_t *cand_row,
                           int32_t *cand_token, float *next_score, int32_t *next_row, int32_t *next_token, void *workspace,
                           size_t workspace_bytes, mq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MQD_H */

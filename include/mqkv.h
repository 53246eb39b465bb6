/*
 * mqkv.h -- C ABI of the paged 8-bit KV cache: attention over it, appending to it, reading it back,
 * and the bookkeeping and copying of its pages (GB300, sm_103a; same library as mq.h).
 *
 * A cache is a pool of pages.  A page holds page_tokens tokens (T) of every layer, and the slab of one
 * layer in a page is
 *   K codes  u8  [n_kv_heads][T][head_dim]
 *   V codes  u8  [n_kv_heads][T][head_dim]
 *   scales   f32 [2 (K, V)][n_kv_heads][T / 32]
 * padded to a multiple of 256 bytes; page p starts at pool + p * page_bytes, the slab of layer l at
 * l * layer_bytes in it (mqkv_page_layout).  A code byte is q + 128 with q in [-127, 127] and stands for
 * q * d, d the scale of its block of 32 tokens, its head and its half.  (The offset makes the byte's f16
 * value one byte permute and one subtraction.)  A scale per token block and head costs 1/8 byte per
 * token and head, and it is a factor of a whole score tile, so the products of attention run on exact
 * integers.
 *
 * A sequence names its pages in order in a row of the page table: token t lies in page
 * table[seq][t / T], slot t % T.  kv_len[seq] counts the cached tokens, those being added in this step
 * included.  A step is
 *     mqkv_extend (pages for the new tokens, kv_len grows)
 *     for every layer: mqkv_append (the last n tokens' keys and values), mqkv_attention
 * where a call's new tokens are always the LAST tokens of their sequences.
 *
 * Conventions: those of mq.h (device pointers owned by the caller unless stated, asynchronous on the
 * stream, host checks before any launch, mq_last_error() names the values, no fallback).  The two
 * descriptions mqkv_cache and mqkv_seqs are host structs, read during the call only.  What only the
 * device can see (lengths, table entries, page counts) is checked there: a bad value is never followed,
 * it sets a bit that mqkv_device_status() reports, and what it concerns is left out.  A bad length: the
 * sequence (its outputs are zeros where the call has outputs).  A bad table entry: mqkv_append skips the
 * blocks that lie in it, mqkv_read gives zeros for the tokens in it, and mqkv_attention gives zeros for all
 * rows of a sequence of which any row would read it.
 */
#ifndef MQKV_H
#define MQKV_H

#include "mq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MQKV_BLOCK 32              /* tokens that share one scale per head and half */
#define MQKV_ERR_STATE (-7)        /* mqkv_device_status: a kernel met a bad length, table entry, page or sequence */

typedef enum { MQKV_F32 = 0, MQKV_F16 = 1, MQKV_BF16 = 2 } mqkv_dtype;

typedef struct {
    void *pool;             /* n_pages pages, 256-byte aligned */
    int32_t *refs;          /* [n_pages]: how many table entries name each page (0 = free); NULL where only
                               append / read / attention are used (append then skips its check of shared pages) */
    int64_t n_pages;        /* below 2^31 */
    int32_t n_layers;
    int32_t n_kv_heads;
    int32_t head_dim;       /* 64 or 128 */
    int32_t page_tokens;    /* 32, 64, 128 or 256 */
} mqkv_cache;

typedef struct {
    int32_t *page_table;    /* [n_seqs][max_pages]; entries past a sequence's last page are not read */
    int32_t *kv_len;        /* [n_seqs] */
    int32_t n_seqs;         /* below 2^24 */
    int32_t max_pages;
} mqkv_seqs;

typedef struct {
    size_t off_v, off_scales, layer_bytes, page_bytes;
} mqkv_layout;

/* Geometry of a page; MQ_ERR_SHAPE for one that is not supported.  Host-only. */
MQ_API int mqkv_page_layout(int32_t n_layers, int32_t n_kv_heads, int32_t head_dim, int32_t page_tokens,
                            mqkv_layout *out);

/*
 * mqkv_append -- quantizes the keys and values of the last tokens of every sequence into the cache.
 *
 *   k, v       [n_tokens][n_kv_heads][head_dim] of dtype, head_dim contiguous, strides in elements and
 *              multiples of 4, bases aligned to 4 elements
 *   cu         [n_seqs + 1], from 0 to n_tokens: the rows of sequence b are cu[b] .. cu[b+1] - 1 and go to
 *              positions kv_len[b] - n_b ..; NULL: n_tokens / n_seqs rows each
 *
 * Per block of 32 slots, head and half, with f slots of earlier tokens:
 *   d  = max(amax(new values) * (1 / 127), old d if f > 0)  (f32, 1 / 127 rounded to f32; 0 below 2^-126)
 *   old codes: q' = round_half_away(q * (old d / d)) where d grew, else unchanged
 *   new codes: q = clamp(round_half_away(x * (1 / d)), -127, 127), 0 where d = 0
 * NaN is stored as 0 and an infinity as the block's largest value (amax is over finite values): one bad
 * token must not spoil the scale of the 31 others.  A token at a time or all at once give the same
 * scales; codes that were rescaled have been rounded twice.
 */
MQ_API int mqkv_append(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t layer, int32_t dtype, const void *k,
                       int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                       int64_t v_head_stride, const int32_t *cu, int64_t n_tokens, mq_stream_t stream);

/*
 * mqkv_read -- the values q * d of tokens of every sequence, dense, rounded once to dtype.
 *   k, v       outputs [n_tokens][n_kv_heads][head_dim], as in mqkv_append; either may be NULL
 *   start      [n_seqs] position of the first token of each; NULL: the last n_b tokens
 */
MQ_API int mqkv_read(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t layer, int32_t dtype, void *k,
                     int64_t k_token_stride, int64_t k_head_stride, void *v, int64_t v_token_stride,
                     int64_t v_head_stride, const int32_t *cu, const int32_t *start, int64_t n_tokens,
                     mq_stream_t stream);

/*
 * mqkv_attention -- out = softmax(scale * q K^T + mask) V over each sequence's cached tokens.
 *
 *   q, out     [n_tokens][n_q_heads][head_dim] of dtype (head_dim contiguous, strides in elements and
 *              multiples of 4, bases aligned to 4 elements); query head x reads KV head
 *              x / (n_q_heads / n_kv_heads)
 *   cu         as in mqkv_append: row i of sequence b has position p = kv_len[b] - n_b + i
 *   max_q      at least the largest n_b (rows past it are not computed, which sets an error bit)
 *   max_kv     about the largest kv_len; sizes the launch and the workspace only
 *   causal     nonzero: p sees positions <= p; window > 0: only positions > p - window
 *   scale      factor of the scores (1 / sqrt(head_dim) as a rule); finite
 *   workspace  mqkv_attention_workspace_bytes(...) bytes, 256-byte aligned, not shared by calls in flight
 *
 * A row that sees nothing (its sequence has no cached token, or every position is masked) is zero.  A row
 * whose q holds a NaN or an infinity is NaN (if it sees anything).  f32 rows keep f32 accuracy: q and the
 * softmax weights enter the tensor cores as two f16 parts each.  16-bit rows enter as one f16 part (q of
 * bf16 exactly, scaled by a power of two per row) and the softmax weights are rounded to f16.  The weights
 * are held relative to the row's largest product of weight and V scale, so a row's error is a fraction of
 * the values that it weighs itself: large values of other tokens, masked or of no weight, take nothing
 * from it, except within a block of 32 tokens, which share their scale.
 */
MQ_API int mqkv_attention(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t layer, int32_t dtype, const void *q,
                          int64_t q_token_stride, int64_t q_head_stride, void *out, int64_t out_token_stride,
                          int64_t out_head_stride, int32_t n_q_heads, const int32_t *cu, int64_t n_tokens, int64_t max_q,
                          int64_t max_kv, int32_t causal, int64_t window, float scale, void *workspace,
                          size_t workspace_bytes, mq_stream_t stream);

/* Bytes of workspace for any mqkv_attention call of these sizes (0 where the sizes are invalid).  Host-only but
 * for one query of the device's SM count. */
MQ_API size_t mqkv_attention_workspace_bytes(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t dtype,
                                             int32_t n_q_heads, int64_t n_tokens, int64_t max_q, int64_t max_kv);

/* ------------------------------------------------------------------ pages ---
 *
 * refs and page_table are the allocator's whole state: a page with refs 0 is free.  Pages are taken lowest
 * first, in the order of the sequences (or forks).  These calls run on one stream in order; they must not run
 * beside one another on the same cache.  They alone give pages back: a length that is lowered by hand past its last
 * page's beginning leaves pages that belong to no sequence.  workspace: mqkv_pages_workspace_bytes(...), 256-byte aligned.
 */
MQ_API size_t mqkv_pages_workspace_bytes(const mqkv_cache *cache, const mqkv_seqs *seqs);

/* kv_len[b] += add[b] (NULL: 1), with pages for the new tokens.  All or nothing: if the pool has too few free
 * pages, or one add is negative or does not fit its table row, no sequence changes (MQKV_ERR_STATE). */
MQ_API int mqkv_extend(const mqkv_cache *cache, const mqkv_seqs *seqs, const int32_t *add, void *workspace,
                       size_t workspace_bytes, mq_stream_t stream);

/* The n sequences ids[] give their pages back: refs fall, kv_len becomes 0, their table rows -1. */
MQ_API int mqkv_release(const mqkv_cache *cache, const mqkv_seqs *seqs, const int32_t *ids, int32_t n,
                        mq_stream_t stream);

/* Sequence child[i] (empty, each named once) becomes a copy of parent[i]: it shares the parent's full pages, and
 * the used blocks of a partly filled last page are copied to a new one.  All or nothing on free pages; a pair with
 * a bad id or a child that is not empty is left out. */
MQ_API int mqkv_fork(const mqkv_cache *cache, const mqkv_seqs *seqs, const int32_t *parent, const int32_t *child,
                     int32_t n, void *workspace, size_t workspace_bytes, mq_stream_t stream);

/* Moves live pages to the front of the pool: with L live pages, the k-th live page at or past L moves to the k-th
 * free page below L, and refs and table follow.  seqs has to be all sequences of the cache: the rows of others would
 * go on naming the places that their pages have left. */
MQ_API int mqkv_compact(const mqkv_cache *cache, const mqkv_seqs *seqs, void *workspace, size_t workspace_bytes,
                        mq_stream_t stream);

/* Copies page src[i] to page dst[i] for i < n (whole pages, no bookkeeping).  No page may be both a source and a
 * destination, or a destination twice. */
MQ_API int mqkv_copy_pages(const mqkv_cache *cache, const int32_t *src, const int32_t *dst, int32_t n,
                           mq_stream_t stream);

/* Synchronizes stream, then reads and clears this device's cache error word (one for all streams): MQ_OK, MQ_ERR_DEVICE_TIMEOUT (a
 * bounded wait ran out: the outputs of that call are undefined) or MQKV_ERR_STATE (text in mq_last_error()). */
MQ_API int mqkv_device_status(mq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MQKV_H */

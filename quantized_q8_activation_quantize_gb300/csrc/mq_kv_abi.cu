// mq_kv_abi.cu -- the C ABI of the KV cache (include/mqkv.h): argument checks on the host, the cache's error word.
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "mq_kv.cuh"

namespace mq {
namespace {

__device__ unsigned int g_kv_err_word;

// address of the current device's cache error word (after the device check of the library)
int kv_state(unsigned int **err) {
    static std::mutex mu;
    static unsigned int *word[64] = {};
    unsigned int *unused = nullptr;
    int rc = device_state(&unused);
    if (rc != MQ_OK) return rc;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    if (word[dev] == nullptr) {
        void *p = nullptr;
        const cudaError_t e = cudaGetSymbolAddress(&p, g_kv_err_word);
        if (e != cudaSuccess) return cuda_error(e, "cudaGetSymbolAddress(cache error word)");
        word[dev] = static_cast<unsigned int *>(p);
    }
    *err = word[dev];
    return MQ_OK;
}

int check_cache(const char *fn, const mqkv_cache *c, mqkv_layout *lay, bool need_refs) {
    if (c == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL cache", fn);
    const int rc = mqkv_page_layout(c->n_layers, c->n_kv_heads, c->head_dim, c->page_tokens, lay);
    if (rc != MQ_OK) return rc;
    if (c->n_pages <= 0 || c->n_pages >= INT32_MAX)
        return set_error(MQ_ERR_SHAPE, "%s: n_pages=%lld not in 1 .. 2^31 - 2", fn, (long long)c->n_pages);
    if (c->pool == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL pool", fn);
    if (!aligned(c->pool, 256)) return set_error(MQ_ERR_ALIGN, "%s: pool %p not 256-byte aligned", fn, c->pool);
    if (need_refs && c->refs == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL refs", fn);
    if (!aligned(c->refs, 4)) return set_error(MQ_ERR_ALIGN, "%s: refs %p not 4-byte aligned", fn, (void *)c->refs);
    return MQ_OK;
}

int check_seqs(const char *fn, const mqkv_seqs *s) {
    if (s == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL sequences", fn);
    if (s->n_seqs < 0 || s->max_pages < 0)
        return set_error(MQ_ERR_ARG, "%s: negative n_seqs=%d or max_pages=%d", fn, s->n_seqs, s->max_pages);
    if (s->n_seqs >= 1 << 24) return set_error(MQ_ERR_SHAPE, "%s: n_seqs=%d must be below 2^24", fn, s->n_seqs);
    if (s->n_seqs == 0) return MQ_OK;
    if (s->max_pages == 0) return set_error(MQ_ERR_SHAPE, "%s: max_pages=0", fn);
    if (s->page_table == nullptr || s->kv_len == nullptr)
        return set_error(MQ_ERR_ARG, "%s: NULL page_table %p or kv_len %p", fn, (void *)s->page_table, (void *)s->kv_len);
    if (!aligned(s->page_table, 4) || !aligned(s->kv_len, 4))
        return set_error(MQ_ERR_ALIGN, "%s: page_table %p or kv_len %p not 4-byte aligned", fn, (void *)s->page_table, (void *)s->kv_len);
    return MQ_OK;
}

int type_bytes(int32_t dtype) { return dtype == MQKV_F32 ? 4 : dtype == MQKV_F16 || dtype == MQKV_BF16 ? 2 : 0; }

// rows of a ragged batch: dtype, layer, cu and the count of rows
int check_rows(const char *fn, const mqkv_cache *c, const mqkv_seqs *s, int32_t layer, int32_t dtype, const int32_t *cu,
               int64_t n_tokens) {
    if (type_bytes(dtype) == 0) return set_error(MQ_ERR_ARG, "%s: dtype=%d not one of mqkv_dtype", fn, dtype);
    if (layer < 0 || layer >= c->n_layers) return set_error(MQ_ERR_ARG, "%s: layer=%d not in 0 .. %d", fn, layer, c->n_layers - 1);
    if (n_tokens < 0 || n_tokens >= INT32_MAX) return set_error(MQ_ERR_SHAPE, "%s: n_tokens=%lld not in 0 .. 2^31 - 2", fn, (long long)n_tokens);
    if (n_tokens > 0 && s->n_seqs == 0) return set_error(MQ_ERR_ARG, "%s: %lld tokens of no sequence", fn, (long long)n_tokens);
    if (cu == nullptr && s->n_seqs > 0 && n_tokens % s->n_seqs != 0)
        return set_error(MQ_ERR_ARG, "%s: without cu, n_tokens=%lld must be a multiple of n_seqs=%d", fn, (long long)n_tokens, s->n_seqs);
    if (!aligned(cu, 4)) return set_error(MQ_ERR_ALIGN, "%s: cu %p not 4-byte aligned", fn, (const void *)cu);
    return MQ_OK;
}

// one [n_tokens][heads][dim] tensor
int check_tensor(const char *fn, const char *what, const void *p, int64_t token_stride, int64_t head_stride, int32_t dtype) {
    if (p == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL %s", fn, what);
    if (!aligned(p, 4 * type_bytes(dtype)) || token_stride % 4 != 0 || head_stride % 4 != 0)
        return set_error(MQ_ERR_ALIGN, "%s: %s %p (strides %lld, %lld) not aligned to 4 elements", fn, what, p, (long long)token_stride,
                         (long long)head_stride);
    if (token_stride < 0 || head_stride < 0)
        return set_error(MQ_ERR_ARG, "%s: %s has a negative stride (%lld, %lld)", fn, what, (long long)token_stride, (long long)head_stride);
    return MQ_OK;
}

// bytes from the first to past the last element of such a tensor
size_t span(int64_t n, int64_t heads, int64_t dim, int64_t ts, int64_t hs, int32_t dtype) {
    return n == 0 ? 0 : (size_t)((n - 1) * ts + (heads - 1) * hs + dim) * type_bytes(dtype);
}
// an output's rows may not share bytes with one another
bool rows_apart(int64_t n, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
    if (n <= 1 && heads <= 1) return true;
    if (heads <= 1) return ts >= dim;
    if (n <= 1) return hs >= dim;
    return (hs >= dim && ts >= (heads - 1) * hs + dim) || (ts >= dim && hs >= (n - 1) * ts + dim);
}

KvView view_of(const mqkv_cache &c, const mqkv_seqs &s, const mqkv_layout &lay, int32_t layer) {
    KvView v;
    v.pool = static_cast<uint8_t *>(c.pool) + (size_t)layer * lay.layer_bytes;
    v.refs = c.refs;
    v.page_bytes = (int64_t)lay.page_bytes;
    v.n_pages = c.n_pages;
    v.table = s.page_table;
    v.len = s.kv_len;
    v.n_seqs = s.n_seqs, v.max_pages = s.max_pages;
    v.H = c.n_kv_heads, v.D = c.head_dim, v.T = c.page_tokens;
    v.tshift = c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : c.page_tokens == 128 ? 7 : 8;
    v.off_v = (int64_t)lay.off_v, v.off_s = (int64_t)lay.off_scales;
    return v;
}

KvRows rows_of(const int32_t *cu, int64_t n_tokens, int32_t n_seqs) { return KvRows{cu, n_tokens, n_tokens / n_seqs}; }

KvPages pages_of(const mqkv_cache &c, const mqkv_seqs *s, const mqkv_layout &lay) {
    KvPages p;
    p.pool = static_cast<uint8_t *>(c.pool), p.refs = c.refs;
    p.table = s ? s->page_table : nullptr, p.len = s ? s->kv_len : nullptr;
    p.page_bytes = (int64_t)lay.page_bytes, p.layer_bytes = (int64_t)lay.layer_bytes, p.off_s = (int64_t)lay.off_scales;
    p.n_pages = (int32_t)c.n_pages, p.n_seqs = s ? s->n_seqs : 0, p.max_pages = s ? s->max_pages : 0;
    p.tshift = c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : c.page_tokens == 128 ? 7 : 8;
    p.n_layers = c.n_layers, p.H = c.n_kv_heads, p.D = c.head_dim;
    return p;
}

int check_ws(const char *fn, const void *ws, size_t have, size_t want) {
    if (ws == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL workspace", fn);
    if (!aligned(ws, 256)) return set_error(MQ_ERR_ALIGN, "%s: workspace %p not 256-byte aligned", fn, ws);
    if (have < want) return set_error(MQ_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, have, want);
    return MQ_OK;
}

}  // namespace
}  // namespace mq

using namespace mq;

#define KV_TRY(e)                       \
    do {                                \
        const int rc_ = (e);            \
        if (rc_ != MQ_OK) return rc_;   \
    } while (0)

extern "C" {

int mqkv_page_layout(int32_t n_layers, int32_t n_kv_heads, int32_t head_dim, int32_t page_tokens, mqkv_layout *out) {
    if (out == nullptr) return set_error(MQ_ERR_ARG, "mqkv_page_layout: NULL output");
    if (n_layers < 1 || n_layers > 4096 || n_kv_heads < 1 || n_kv_heads > 512)
        return set_error(MQ_ERR_SHAPE, "n_layers=%d not in 1 .. 4096 or n_kv_heads=%d not in 1 .. 512", n_layers, n_kv_heads);
    if (head_dim != 64 && head_dim != 128) return set_error(MQ_ERR_SHAPE, "head_dim=%d is neither 64 nor 128", head_dim);
    if (page_tokens != 32 && page_tokens != 64 && page_tokens != 128 && page_tokens != 256)
        return set_error(MQ_ERR_SHAPE, "page_tokens=%d is none of 32, 64, 128, 256", page_tokens);
    const size_t half = (size_t)n_kv_heads * page_tokens * head_dim;
    out->off_v = half;
    out->off_scales = 2 * half;
    out->layer_bytes = (2 * half + 2 * (size_t)n_kv_heads * (page_tokens / kKB) * 4 + 255) & ~size_t(255);
    out->page_bytes = out->layer_bytes * n_layers;
    return MQ_OK;
}

int mqkv_append(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t layer, int32_t dtype, const void *k,
                int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                const int32_t *cu, int64_t n_tokens, mq_stream_t stream) {
    const char *fn = "mqkv_append";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, false));
    KV_TRY(check_seqs(fn, seqs));
    KV_TRY(check_rows(fn, cache, seqs, layer, dtype, cu, n_tokens));
    if (n_tokens == 0) return MQ_OK;
    KV_TRY(check_tensor(fn, "k", k, k_token_stride, k_head_stride, dtype));
    KV_TRY(check_tensor(fn, "v", v, v_token_stride, v_head_stride, dtype));
    const int64_t H = cache->n_kv_heads, D = cache->head_dim;
    const size_t pool = lay.page_bytes * (size_t)cache->n_pages;
    if (overlaps(cache->pool, pool, k, span(n_tokens, H, D, k_token_stride, k_head_stride, dtype)) ||
        overlaps(cache->pool, pool, v, span(n_tokens, H, D, v_token_stride, v_head_stride, dtype)))
        return set_error(MQ_ERR_ARG, "%s: the pool %p overlaps k %p or v %p", fn, cache->pool, k, v);
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_append(view_of(*cache, *seqs, lay, layer), rows_of(cu, n_tokens, seqs->n_seqs), dtype, k, k_token_stride,
                            k_head_stride, v, v_token_stride, v_head_stride, err, reinterpret_cast<cudaStream_t>(stream));
}

int mqkv_read(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t layer, int32_t dtype, void *k, int64_t k_token_stride,
              int64_t k_head_stride, void *v, int64_t v_token_stride, int64_t v_head_stride, const int32_t *cu,
              const int32_t *start, int64_t n_tokens, mq_stream_t stream) {
    const char *fn = "mqkv_read";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, false));
    KV_TRY(check_seqs(fn, seqs));
    KV_TRY(check_rows(fn, cache, seqs, layer, dtype, cu, n_tokens));
    if (!aligned(start, 4)) return set_error(MQ_ERR_ALIGN, "%s: start %p not 4-byte aligned", fn, (const void *)start);
    if (n_tokens == 0) return MQ_OK;
    if (k == nullptr && v == nullptr) return set_error(MQ_ERR_ARG, "%s: both outputs NULL", fn);
    const int64_t H = cache->n_kv_heads, D = cache->head_dim;
    const size_t pool = lay.page_bytes * (size_t)cache->n_pages;
    size_t kb = 0, vb = 0;
    if (k != nullptr) {
        KV_TRY(check_tensor(fn, "k", k, k_token_stride, k_head_stride, dtype));
        kb = span(n_tokens, H, D, k_token_stride, k_head_stride, dtype);
        if (!rows_apart(n_tokens, H, D, k_token_stride, k_head_stride))
            return set_error(MQ_ERR_ARG, "%s: rows of k overlap (strides %lld, %lld)", fn, (long long)k_token_stride, (long long)k_head_stride);
    }
    if (v != nullptr) {
        KV_TRY(check_tensor(fn, "v", v, v_token_stride, v_head_stride, dtype));
        vb = span(n_tokens, H, D, v_token_stride, v_head_stride, dtype);
        if (!rows_apart(n_tokens, H, D, v_token_stride, v_head_stride))
            return set_error(MQ_ERR_ARG, "%s: rows of v overlap (strides %lld, %lld)", fn, (long long)v_token_stride, (long long)v_head_stride);
    }
    // k and v may interleave (one buffer of both); only the pool has to stay clear of them
    if (overlaps(cache->pool, pool, k, kb) || overlaps(cache->pool, pool, v, vb))
        return set_error(MQ_ERR_ARG, "%s: k %p or v %p overlaps the pool %p", fn, k, v, cache->pool);
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_read(view_of(*cache, *seqs, lay, layer), rows_of(cu, n_tokens, seqs->n_seqs), dtype, k, k_token_stride,
                          k_head_stride, v, v_token_stride, v_head_stride, start, err, reinterpret_cast<cudaStream_t>(stream));
}

// a window that reaches past every position (they lie within 2^31 of 0), with room for the sums that the kernels make of it
static constexpr int64_t kFarWindow = (int64_t)1 << 40;

static int check_attn_sizes(const char *fn, const mqkv_cache *cache, int32_t n_q_heads, int64_t max_q, int64_t max_kv) {
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads != 0 || n_q_heads > 65536)
        return set_error(MQ_ERR_SHAPE, "%s: n_q_heads=%d must be a multiple of n_kv_heads=%d of at most 65536", fn, n_q_heads, cache->n_kv_heads);
    if (max_q < 0 || max_kv < 0 || max_q >= INT32_MAX || max_kv > INT32_MAX)
        return set_error(MQ_ERR_SHAPE, "%s: max_q=%lld or max_kv=%lld not in 0 .. 2^31 - 2", fn, (long long)max_q, (long long)max_kv);
    return MQ_OK;
}

size_t mqkv_attention_workspace_bytes(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t dtype, int32_t n_q_heads,
                                      int64_t n_tokens, int64_t max_q, int64_t max_kv) {
    const char *fn = "mqkv_attention_workspace_bytes";
    mqkv_layout lay;
    if (cache == nullptr || seqs == nullptr || type_bytes(dtype) == 0 || n_tokens < 0 || seqs->n_seqs < 0 ||
        mqkv_page_layout(cache->n_layers, cache->n_kv_heads, cache->head_dim, cache->page_tokens, &lay) != MQ_OK ||
        check_attn_sizes(fn, cache, n_q_heads, max_q, max_kv) != MQ_OK)
        return 0;
    if (n_tokens == 0 || seqs->n_seqs == 0) return 256;
    return kv_attention_ws(seqs->n_seqs, cache->n_kv_heads, cache->head_dim, dtype, n_q_heads, n_tokens, max_q, max_kv);
}

int mqkv_attention(const mqkv_cache *cache, const mqkv_seqs *seqs, int32_t layer, int32_t dtype, const void *q,
                   int64_t q_token_stride, int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride,
                   int32_t n_q_heads, const int32_t *cu, int64_t n_tokens, int64_t max_q, int64_t max_kv, int32_t causal,
                   int64_t window, float scale, void *workspace, size_t workspace_bytes, mq_stream_t stream) {
    const char *fn = "mqkv_attention";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, false));
    KV_TRY(check_seqs(fn, seqs));
    KV_TRY(check_rows(fn, cache, seqs, layer, dtype, cu, n_tokens));
    KV_TRY(check_attn_sizes(fn, cache, n_q_heads, max_q, max_kv));
    if (window < 0) return set_error(MQ_ERR_ARG, "%s: negative window=%lld", fn, (long long)window);
    if (!std::isfinite(scale)) return set_error(MQ_ERR_ARG, "%s: scale=%g not finite", fn, (double)scale);
    window = window < kFarWindow ? window : kFarWindow;
    if (n_tokens == 0) return MQ_OK;
    if (max_q == 0) return set_error(MQ_ERR_ARG, "%s: max_q=0 for %lld tokens", fn, (long long)n_tokens);
    if (cu == nullptr && max_q < n_tokens / seqs->n_seqs)
        return set_error(MQ_ERR_ARG, "%s: max_q=%lld below the %lld tokens of each sequence", fn, (long long)max_q, (long long)(n_tokens / seqs->n_seqs));
    KV_TRY(check_tensor(fn, "q", q, q_token_stride, q_head_stride, dtype));
    KV_TRY(check_tensor(fn, "out", out, out_token_stride, out_head_stride, dtype));
    const int64_t D = cache->head_dim;
    if (!rows_apart(n_tokens, n_q_heads, D, out_token_stride, out_head_stride))
        return set_error(MQ_ERR_ARG, "%s: rows of out overlap (strides %lld, %lld)", fn, (long long)out_token_stride, (long long)out_head_stride);
    const size_t want = mqkv_attention_workspace_bytes(cache, seqs, dtype, n_q_heads, n_tokens, max_q, max_kv);
    KV_TRY(check_ws(fn, workspace, workspace_bytes, want));
    const size_t pool = lay.page_bytes * (size_t)cache->n_pages, ob = span(n_tokens, n_q_heads, D, out_token_stride, out_head_stride, dtype),
                 qb = span(n_tokens, n_q_heads, D, q_token_stride, q_head_stride, dtype);
    if (overlaps(out, ob, q, qb) || overlaps(out, ob, cache->pool, pool) || overlaps(out, ob, workspace, want) ||
        overlaps(workspace, want, q, qb) || overlaps(workspace, want, cache->pool, pool))
        return set_error(MQ_ERR_ARG, "%s: out %p, q %p, the pool %p and the workspace %p must not overlap", fn, out, q, cache->pool, workspace);
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    const KvAttn a{q, out, q_token_stride, q_head_stride, out_token_stride, out_head_stride, n_q_heads, n_q_heads / cache->n_kv_heads,
                   dtype, causal != 0, n_tokens, max_q, max_kv, window, scale};
    return kv_launch_attention(*cache, lay, layer, view_of(*cache, *seqs, lay, layer), rows_of(cu, n_tokens, seqs->n_seqs), a, workspace,
                               err, reinterpret_cast<cudaStream_t>(stream));
}

size_t mqkv_pages_workspace_bytes(const mqkv_cache *cache, const mqkv_seqs *seqs) {
    if (cache == nullptr || seqs == nullptr || cache->n_pages <= 0 || cache->n_pages >= INT32_MAX || seqs->n_seqs < 0) return 0;
    return kv_pages_ws(cache->n_pages, seqs->n_seqs);
}

int mqkv_extend(const mqkv_cache *cache, const mqkv_seqs *seqs, const int32_t *add, void *workspace, size_t workspace_bytes,
                mq_stream_t stream) {
    const char *fn = "mqkv_extend";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, true));
    KV_TRY(check_seqs(fn, seqs));
    if (!aligned(add, 4)) return set_error(MQ_ERR_ALIGN, "%s: add %p not 4-byte aligned", fn, (const void *)add);
    if (seqs->n_seqs == 0) return MQ_OK;
    KV_TRY(check_ws(fn, workspace, workspace_bytes, mqkv_pages_workspace_bytes(cache, seqs)));
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_extend(pages_of(*cache, seqs, lay), add, workspace, err, reinterpret_cast<cudaStream_t>(stream));
}

static int check_ids(const char *fn, const mqkv_seqs *seqs, const int32_t *a, const int32_t *b, int32_t n) {
    if (n < 0 || n > seqs->n_seqs) return set_error(MQ_ERR_ARG, "%s: n=%d not in 0 .. n_seqs=%d", fn, n, seqs->n_seqs);
    if (n > 0 && (a == nullptr || b == nullptr)) return set_error(MQ_ERR_ARG, "%s: NULL list of sequences", fn);
    if (!aligned(a, 4) || !aligned(b, 4)) return set_error(MQ_ERR_ALIGN, "%s: a list of sequences is not 4-byte aligned", fn);
    return MQ_OK;
}

int mqkv_release(const mqkv_cache *cache, const mqkv_seqs *seqs, const int32_t *ids, int32_t n, mq_stream_t stream) {
    const char *fn = "mqkv_release";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, true));
    KV_TRY(check_seqs(fn, seqs));
    KV_TRY(check_ids(fn, seqs, ids, ids, n));
    if (n == 0) return MQ_OK;
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_release(pages_of(*cache, seqs, lay), ids, n, err, reinterpret_cast<cudaStream_t>(stream));
}

int mqkv_fork(const mqkv_cache *cache, const mqkv_seqs *seqs, const int32_t *parent, const int32_t *child, int32_t n,
              void *workspace, size_t workspace_bytes, mq_stream_t stream) {
    const char *fn = "mqkv_fork";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, true));
    KV_TRY(check_seqs(fn, seqs));
    KV_TRY(check_ids(fn, seqs, parent, child, n));
    if (n == 0) return MQ_OK;
    KV_TRY(check_ws(fn, workspace, workspace_bytes, mqkv_pages_workspace_bytes(cache, seqs)));
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_fork(pages_of(*cache, seqs, lay), parent, child, n, workspace, err, reinterpret_cast<cudaStream_t>(stream));
}

int mqkv_compact(const mqkv_cache *cache, const mqkv_seqs *seqs, void *workspace, size_t workspace_bytes, mq_stream_t stream) {
    const char *fn = "mqkv_compact";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, true));
    KV_TRY(check_seqs(fn, seqs));
    if (seqs->n_seqs == 0) return MQ_OK;
    KV_TRY(check_ws(fn, workspace, workspace_bytes, mqkv_pages_workspace_bytes(cache, seqs)));
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_compact(pages_of(*cache, seqs, lay), workspace, err, reinterpret_cast<cudaStream_t>(stream));
}

int mqkv_copy_pages(const mqkv_cache *cache, const int32_t *src, const int32_t *dst, int32_t n, mq_stream_t stream) {
    const char *fn = "mqkv_copy_pages";
    mqkv_layout lay;
    KV_TRY(check_cache(fn, cache, &lay, false));
    if (n < 0) return set_error(MQ_ERR_ARG, "%s: negative n=%d", fn, n);
    if (n == 0) return MQ_OK;
    if (src == nullptr || dst == nullptr) return set_error(MQ_ERR_ARG, "%s: NULL list of pages", fn);
    if (!aligned(src, 4) || !aligned(dst, 4)) return set_error(MQ_ERR_ALIGN, "%s: a list of pages is not 4-byte aligned", fn);
    unsigned int *err = nullptr;
    KV_TRY(kv_state(&err));
    return kv_launch_copy(pages_of(*cache, nullptr, lay), src, dst, n, err, reinterpret_cast<cudaStream_t>(stream));
}

int mqkv_device_status(mq_stream_t stream) {
    unsigned int *word = nullptr;
    KV_TRY(kv_state(&word));
    cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_error(e, "mqkv_device_status: stream synchronize");
    unsigned int v = 0;
    const unsigned int zero = 0;
    e = cudaMemcpy(&v, word, sizeof v, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v != 0) e = cudaMemcpy(word, &zero, sizeof zero, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_error(e, "mqkv_device_status: error word");
    if (v == 0) return MQ_OK;
    static const char *names[kKvErrBits] = {"page table entry outside the pool", "length outside its table row or below the new tokens",
                                            "append into a shared or free page", "too few free pages",
                                            "sequence id out of range, named twice, or a child that is not empty",
                                            "more new tokens than max_q", "bounded device wait ran out"};
    char buf[400] = "";
    for (int i = 0; i < kKvErrBits; ++i)
        if (v & (1u << i)) {
            strncat(buf, buf[0] ? "; " : " ", sizeof buf - strlen(buf) - 1);
            strncat(buf, names[i], sizeof buf - strlen(buf) - 1);
        }
    return set_error(v & KV_ERR_WAIT ? MQ_ERR_DEVICE_TIMEOUT : MQKV_ERR_STATE, "cache (code 0x%x):%s", v, buf);
}

}  // extern "C"

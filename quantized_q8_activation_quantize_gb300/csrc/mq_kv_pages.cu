// mq_kv_pages.cu -- bookkeeping and copying of the cache's pages.
//
// The allocator's state is refs[] and the page table, both on the device, so a step (or a captured graph of one) never
// waits for the host.  Each call plans in one CTA -- a scan over the sequences (or forks) for what they need and a scan
// over refs for the lowest free pages: a few thousand integers, a few microseconds of latency that more CTAs would not
// shorten -- and what has to move goes to a second kernel over all SMs, which is bound by HBM (a read and a write
// of every byte).
#include "mq_kv.cuh"

namespace mq {
namespace {

constexpr int kPlanThreads = 1024;

// what a plan leaves for the copying kernel
struct CopyPlan {
    int32_t n;          // copies
    int32_t pad[63];
    // followed by: int32 src[], dst[], blocks[] (n_pages or n each), prefix[], free list[]
};

struct Ws {
    CopyPlan *plan;
    int32_t *src, *dst, *blocks, *prefix, *list;
    __host__ __device__ static size_t items(int64_t n_pages, int64_t n_seqs) { return (size_t)((n_pages > n_seqs ? n_pages : n_seqs) + 64) & ~size_t(63); }
    __host__ __device__ Ws(void *p, int64_t n_pages, int64_t n_seqs) {
        const size_t k = items(n_pages, n_seqs);
        plan = static_cast<CopyPlan *>(p);
        src = reinterpret_cast<int32_t *>(plan + 1);
        dst = src + k, blocks = dst + k, prefix = blocks + k, list = prefix + k;
    }
};

// exclusive prefix sum over the block's values; *total gets the sum.  Two barriers, reusable at once.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *s_warp, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    T w = s_warp[lane];                         // 32 warps: one sum a lane
    T z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, z, o);
        if (lane >= o) z += y;
    }
    const T before = __shfl_sync(0xffffffffu, z - w, warp);
    *total = __shfl_sync(0xffffffffu, z, 31);
    return before + x - v;
}

// list[0 .. need) = the lowest free pages; returns whether there are as many
__device__ bool find_free(const int32_t *refs, int n_pages, int need, int32_t *list, int *s_warp) {
    int found = 0;
    for (int64_t base = 0; base < n_pages && found < need; base += 4 * kPlanThreads) {
        const int64_t i = base + 4 * threadIdx.x;
        bool f[4];
        int cnt = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = i + e < n_pages && refs[i + e] == 0;
            cnt += f[e];
        }
        int total;
        int at = found + block_scan(cnt, s_warp, &total);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (f[e]) {
                if (at < need) list[at] = (int)(i + e);
                ++at;
            }
        found += total;
    }
    __syncthreads();
    return found >= need;
}

__global__ void __launch_bounds__(kPlanThreads) kv_extend_kernel(KvPages p, const int32_t *add, Ws ws, unsigned int *err) {
    __shared__ int s_warp[32];
    __shared__ int64_t s_need[32];
    grid_dep_launch();
    grid_dep_wait();
    const int T = 1 << p.tshift;
    int64_t need = 0;                           // of all sequences: may pass 32 bits, and is refused below
    bool bad = false;
    for (int base = 0; base < p.n_seqs; base += kPlanThreads) {
        const int b = base + threadIdx.x;
        int64_t k = 0;
        if (b < p.n_seqs) {
            const int64_t len = p.len[b], a = add != nullptr ? add[b] : 1;
            const int64_t have = (len + T - 1) >> p.tshift, want = (len + a + T - 1) >> p.tshift;
            if (len < 0 || a < 0 || want > p.max_pages || len + a > INT32_MAX) bad = true;
            else k = want - have;
        }
        int64_t total;
        const int64_t at = need + block_scan(k, s_need, &total);
        if (b < p.n_seqs) ws.prefix[b] = (int)at;
        need += total;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_LEN);
        return;
    }
    if (need > p.n_pages || !find_free(p.refs, p.n_pages, (int)need, ws.list, s_warp)) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_FULL);
        return;
    }
    for (int b = threadIdx.x; b < p.n_seqs; b += kPlanThreads) {
        const int len = p.len[b], a = add != nullptr ? add[b] : 1;
        const int have = (int)(((int64_t)len + T - 1) >> p.tshift), want = (int)(((int64_t)len + a + T - 1) >> p.tshift);
        for (int s = have; s < want; ++s) {
            const int page = ws.list[ws.prefix[b] + s - have];
            p.table[(int64_t)b * p.max_pages + s] = page;
            p.refs[page] = 1;
        }
        p.len[b] = len + a;
    }
}

// one CTA per sequence that ends
__global__ void __launch_bounds__(128) kv_release_kernel(KvPages p, const int32_t *ids, unsigned int *err) {
    __shared__ int s_len;
    grid_dep_launch();
    grid_dep_wait();
    const int id = ids[blockIdx.x];
    if (id < 0 || id >= p.n_seqs) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_SEQ);
        return;
    }
    if (threadIdx.x == 0) s_len = atomicExch(&p.len[id], 0);      // a sequence named twice is released once
    __syncthreads();
    const int T = 1 << p.tshift;
    int64_t held = ((int64_t)s_len + T - 1) >> p.tshift;
    if (held < 0 || held > p.max_pages) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_LEN);
        held = held < 0 ? 0 : p.max_pages;
    }
    int32_t *row = p.table + (int64_t)id * p.max_pages;
    for (int s = threadIdx.x; s < p.max_pages; s += blockDim.x) {
        if (s < held) {
            const int page = row[s];
            if (page < 0 || page >= p.n_pages) {
                kv_error(err, KV_ERR_PAGE);
            } else if (atomicSub(&p.refs[page], 1) <= 0) {
                atomicAdd(&p.refs[page], 1);
                kv_error(err, KV_ERR_PAGE);
            }
        }
        if (held > 0) row[s] = -1;
    }
}

__global__ void __launch_bounds__(kPlanThreads) kv_fork_kernel(KvPages p, const int32_t *parent, const int32_t *child, int n, Ws ws,
                                                               unsigned int *err) {
    __shared__ int s_warp[32];
    grid_dep_launch();
    grid_dep_wait();
    const int T = 1 << p.tshift;
    // which pair names a child first: src[] holds the lowest pair of each sequence while the plan is made
    for (int b = threadIdx.x; b < p.n_seqs; b += kPlanThreads) ws.src[b] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int c = child[i];
        if (c >= 0 && c < p.n_seqs) atomicMin(&ws.src[c], i);
    }
    __syncthreads();
    // a warp per pair: its ids, its parent's length and pages; blocks[] gets the length, -1 for a pair that is left out
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int a = parent[i], c = child[i];
        int len = -1;
        if (a < 0 || a >= p.n_seqs || c < 0 || c >= p.n_seqs || ws.src[c] != i || p.len[c] != 0) {
            if (lane == 0) kv_error(err, KV_ERR_SEQ);
        } else {
            len = p.len[a];
            const int64_t held = ((int64_t)len + T - 1) >> p.tshift;
            if (len < 0 || held > p.max_pages) {
                if (lane == 0) kv_error(err, KV_ERR_LEN);
                len = -1;
            } else {
                bool bad = false;
                for (int s = lane; s < held; s += 32) {
                    const int page = p.table[(int64_t)a * p.max_pages + s];
                    bad = bad || page < 0 || page >= p.n_pages;
                }
                if (__any_sync(0xffffffffu, bad)) {
                    if (lane == 0) kv_error(err, KV_ERR_PAGE);
                    len = -1;
                }
            }
        }
        if (lane == 0) ws.blocks[i] = len;
    }
    __syncthreads();
    int need = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        const int len = i < n ? ws.blocks[i] : -1, k = len > 0 && (len & (T - 1)) != 0;
        int total;
        const int at = need + block_scan(k, s_warp, &total);
        if (i < n) ws.prefix[i] = k ? at : -1;
        need += total;
    }
    __syncthreads();
    if (!find_free(p.refs, p.n_pages, need, ws.list, s_warp)) {
        if (threadIdx.x == 0) {
            kv_error(err, KV_ERR_FULL);
            ws.plan->n = 0;
        }
        return;
    }
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int len = ws.blocks[i], at = ws.prefix[i];
        if (len <= 0) continue;
        const int a = parent[i], c = child[i], full = len >> p.tshift;
        const int32_t *from = p.table + (int64_t)a * p.max_pages;
        int32_t *to = p.table + (int64_t)c * p.max_pages;
        for (int s = lane; s < full; s += 32) {
            to[s] = from[s];
            atomicAdd(&p.refs[from[s]], 1);
        }
        if (lane == 0) {
            if (at >= 0) {
                to[full] = ws.list[at];
                p.refs[ws.list[at]] = 1;
            }
            p.len[c] = len;
        }
        __syncwarp();
    }
    __syncthreads();
    // the copies; list[] turns from a page into the used blocks of the tail page
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int len = 0, at = -1, s = 0, d = 0;
        if (i < n) {
            len = ws.blocks[i], at = ws.prefix[i];
            if (at >= 0) {
                s = p.table[(int64_t)parent[i] * p.max_pages + (len >> p.tshift)];
                d = ws.list[at];
            }
        }
        __syncthreads();
        if (at >= 0) {
            ws.src[at] = s;
            ws.dst[at] = d;
            ws.list[at] = ((len & (T - 1)) + kKB - 1) / kKB;
        }
    }
    if (threadIdx.x == 0) ws.plan->n = need;
}

__global__ void __launch_bounds__(kPlanThreads) kv_compact_kernel(KvPages p, Ws ws, unsigned int *err) {
    __shared__ int s_warp[32];
    grid_dep_launch();
    grid_dep_wait();
    int live = 0;
    for (int64_t i = threadIdx.x; i < p.n_pages; i += kPlanThreads) live += p.refs[i] > 0;
    int n_live;
    block_scan(live, s_warp, &n_live);
    int holes = 0, movers = 0;
    for (int64_t base = 0; base < p.n_pages; base += kPlanThreads) {
        const int i = (int)(base + threadIdx.x);
        const bool in = base + threadIdx.x < p.n_pages, used = in && p.refs[i] > 0;
        const bool hole = in && !used && i < n_live, mover = used && i >= n_live;
        int total;
        int at = holes + block_scan((int)hole, s_warp, &total);
        if (hole) ws.dst[at] = i;
        holes += total;
        at = movers + block_scan((int)mover, s_warp, &total);
        if (mover) ws.src[at] = i;
        movers += total;
        if (in) ws.list[i] = i;                   // where page i goes
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kPlanThreads) {
        const int s = ws.src[k], d = ws.dst[k];
        ws.list[s] = d;
        p.refs[d] = p.refs[s];
        p.refs[s] = 0;
    }
    if (threadIdx.x == 0) ws.plan->n = movers;
}

// the table row of sequence b after pages have moved
__device__ __forceinline__ void remap_row(const KvPages &p, const Ws &ws, int b, unsigned int *err) {
    const int T = 1 << p.tshift;
    const int64_t held = ((int64_t)p.len[b] + T - 1) >> p.tshift;
    if (held < 0 || held > p.max_pages) {
        if (threadIdx.x == 0) kv_error(err, KV_ERR_LEN);
        return;
    }
    int32_t *row = p.table + (int64_t)b * p.max_pages;
    for (int s = threadIdx.x; s < held; s += blockDim.x) {
        const int page = row[s];
        if (page < 0 || page >= p.n_pages) kv_error(err, KV_ERR_PAGE);
        else row[s] = ws.list[page];
    }
}

constexpr int kCopyThreads = 256, kCopyChunk = 16384;

__device__ __forceinline__ void copy_span(uint8_t *dst, const uint8_t *src, int bytes) {
    const uint4 *s = reinterpret_cast<const uint4 *>(src);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    const int n = bytes >> 4;
    for (int i = threadIdx.x; i < n; i += 4 * kCopyThreads) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e * kCopyThreads < n) v[e] = __ldcs(s + i + e * kCopyThreads);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e * kCopyThreads < n) d[i + e * kCopyThreads] = v[e];
    }
}

// whole pages in pieces of 16 KB; n < 0: a compaction's plan, whose tables it also brings up to date
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(KvPages p, const int32_t *src, const int32_t *dst, int n, Ws ws, unsigned int *err) {
    grid_dep_launch();
    grid_dep_wait();
    if (n < 0) {
        for (int b = blockIdx.x; b < p.n_seqs; b += gridDim.x) remap_row(p, ws, b, err);
        n = ws.plan->n;
    }
    const int64_t per = (p.page_bytes + kCopyChunk - 1) / kCopyChunk;
    for (int64_t u = blockIdx.x; u < n * per; u += gridDim.x) {
        const int64_t i = u / per, off = (u - i * per) * kCopyChunk;
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= p.n_pages || d < 0 || d >= p.n_pages) {
            if (threadIdx.x == 0) kv_error(err, KV_ERR_PAGE);
            continue;
        }
        if (s == d) continue;
        copy_span(p.pool + d * p.page_bytes + off, p.pool + s * p.page_bytes + off, (int)min((int64_t)kCopyChunk, p.page_bytes - off));
    }
}

// the used blocks of partly filled pages: a unit is one (page, layer) and one of its 2 H runs of codes (the first takes the scales too)
__global__ void __launch_bounds__(kCopyThreads) kv_copy_used_kernel(KvPages p, Ws ws) {
    grid_dep_launch();
    grid_dep_wait();
    const int n = ws.plan->n, T = 1 << p.tshift, runs = 2 * p.H;
    for (int64_t u = blockIdx.x; u < (int64_t)n * p.n_layers * runs; u += gridDim.x) {
        const int64_t page = u / runs;
        const int run = (int)(u - page * runs), i = (int)(page / p.n_layers), layer = (int)(page - (int64_t)i * p.n_layers);
        const uint8_t *s = p.pool + ws.src[i] * p.page_bytes + layer * p.layer_bytes;
        uint8_t *d = p.pool + ws.dst[i] * p.page_bytes + layer * p.layer_bytes;
        copy_span(d + run * T * p.D, s + run * T * p.D, ws.list[i] * kKB * p.D);
        if (run == 0)
            for (int j = threadIdx.x; j < runs * (T / kKB); j += kCopyThreads)
                reinterpret_cast<uint32_t *>(d + p.off_s)[j] = reinterpret_cast<const uint32_t *>(s + p.off_s)[j];
    }
}

}  // namespace

size_t kv_pages_ws(int64_t n_pages, int64_t n_seqs) { return sizeof(CopyPlan) + 5 * 4 * Ws::items(n_pages, n_seqs); }

int kv_launch_extend(const KvPages &p, const int32_t *add, void *ws, unsigned int *err, cudaStream_t s) {
    return cuda_error(launch_pdl(kv_extend_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, add, Ws(ws, p.n_pages, p.n_seqs), err),
                      "mqkv_extend launch");
}

int kv_launch_release(const KvPages &p, const int32_t *ids, int n, unsigned int *err, cudaStream_t s) {
    return cuda_error(launch_pdl(kv_release_kernel, dim3(n), dim3(128), 0, s, p, ids, err), "mqkv_release launch");
}

int kv_launch_fork(const KvPages &p, const int32_t *parent, const int32_t *child, int n, void *ws, unsigned int *err,
                   cudaStream_t s) {
    const Ws w(ws, p.n_pages, p.n_seqs);
    int rc = cuda_error(launch_pdl(kv_fork_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, parent, child, n, w, err), "mqkv_fork plan launch");
    if (rc != MQ_OK) return rc;
    const int64_t units = (int64_t)n * p.n_layers * 2 * p.H;
    const int grid = (int)(units < 8 * sm_count() ? units : 8 * sm_count());
    return cuda_error(launch_pdl(kv_copy_used_kernel, dim3(grid), dim3(kCopyThreads), 0, s, p, w), "mqkv_fork copy launch");
}

int kv_launch_compact(const KvPages &p, void *ws, unsigned int *err, cudaStream_t s) {
    const Ws w(ws, p.n_pages, p.n_seqs);
    int rc = cuda_error(launch_pdl(kv_compact_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, w, err), "mqkv_compact plan launch");
    if (rc != MQ_OK) return rc;
    return cuda_error(launch_pdl(kv_copy_kernel, dim3(8 * sm_count()), dim3(kCopyThreads), 0, s, p, (const int32_t *)w.src,
                                 (const int32_t *)w.dst, -1, w, err),
                      "mqkv_compact copy launch");
}

int kv_launch_copy(const KvPages &p, const int32_t *src, const int32_t *dst, int n, unsigned int *err, cudaStream_t s) {
    return cuda_error(launch_pdl(kv_copy_kernel, dim3(8 * sm_count()), dim3(kCopyThreads), 0, s, p, src, dst, n, Ws(nullptr, 0, 0), err),
                      "mqkv_copy_pages launch");
}

}  // namespace mq

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

// ---------------------------------------------------------------- reorder ---
// Row b becomes what row parent[b] was.  A block, or for large tables a cluster of them, does the bookkeeping; a second kernel copies the used blocks of the last
// pages that two rows would share.  A plan of a few thousand integers is all latency: parents, lengths and the table are read once into shared memory
// and every phase works on them there.  Each block knows all rows and takes some columns of the table; the cluster's barriers order the phases (checks, reference counts, pages
// for the copies, the table).  (4 rows of 53 pages with their copies: 9.3 us, with the table read again in every phase 14.6; 96 rows 19.4 and
// 24.3.)
constexpr int kReorderCluster = 8, kReorderCells = 32768;      // cells of the table that a block holds at a time

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// all threads of the cluster
__device__ __forceinline__ void cluster_sync(int ranks) {
    if (ranks == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the int at `p` of this block's shared memory, in block `rank` of the cluster
__device__ __forceinline__ int cluster_peer(const int *p, int rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// rows in shared memory: parent; own length; the copy's number, -1: none
struct ReorderRows {
    int *parent, *len, *copy;
    int n, tshift;
    __device__ __forceinline__ int pages(int len) const { return (int)(((int64_t)len + (1 << tshift) - 1) >> tshift); }
    __device__ __forceinline__ int held(int b) const { return pages(len[b]); }
    __device__ __forceinline__ int new_len(int b) const { return parent[b] >= 0 ? len[parent[b]] : 0; }
};

// the table's columns [c0, c0 + nc) of all rows; what lies past a row's pages is -1
__device__ __forceinline__ void reorder_load(const KvPages &p, const ReorderRows &r, int c0, int nc, int32_t *s_cells) {
    for (int i = threadIdx.x; i < r.n * nc; i += kPlanThreads) {
        const int b = i / nc, s = c0 + i - b * nc;
        s_cells[i] = s < r.held(b) ? p.table[(int64_t)b * p.max_pages + s] : -1;
    }
}

// the reference counts' change (sign -1: taken back) in these columns: pages that a row and its parent hold in the same place stay
__device__ __forceinline__ void reorder_refs(const KvPages &p, const ReorderRows &r, int c0, int nc, const int32_t *s_cells, int sign) {
    for (int i = threadIdx.x; i < r.n * nc; i += kPlanThreads) {
        const int b = i / nc, s = c0 + i - b * nc, parent = r.parent[b];
        const bool mine = r.copy[b] >= 0 && s == r.pages(r.new_len(b)) - 1;    // the last page of a row that copies is its own
        const int a = s_cells[i], c = parent >= 0 && !mine ? s_cells[parent * nc + s - c0] : -1;
        if (a == c) continue;
        if (a >= 0) atomicAdd(&p.refs[a], -sign);
        if (c >= 0) atomicAdd(&p.refs[c], sign);
    }
}

__global__ void __launch_bounds__(kPlanThreads) kv_reorder_kernel(KvPages p, const int32_t *parent, Ws ws, int cols, unsigned int *err) {
    extern __shared__ int32_t s_rows[];                        // parent, length, copy, first [n_seqs each], cells [n_seqs][cols]
    __shared__ int s_warp[32], s_bad, s_most;
    grid_dep_launch();
    grid_dep_wait();
    const int T = 1 << p.tshift, n = p.n_seqs, ranks = gridDim.x, rank = ranks == 1 ? 0 : cluster_rank();
    const ReorderRows r{s_rows, s_rows + n, s_rows + 2 * n, n, p.tshift};
    int *first = s_rows + 3 * n;                               // the lowest row that continues each row
    int32_t *s_cells = s_rows + 4 * n;
    if (threadIdx.x == 0) s_bad = 0, s_most = 0;
    for (int b = threadIdx.x; b < n; b += kPlanThreads) r.parent[b] = parent[b], r.len[b] = p.len[b], first[b] = INT32_MAX;
    __syncthreads();
    unsigned bad = 0;
    int most = 0;
    for (int b = threadIdx.x; b < n; b += kPlanThreads) {
        const int a = r.parent[b], len = r.len[b];
        if (a < -1 || a >= n) bad |= KV_ERR_SEQ, r.parent[b] = -1;
        else if (a >= 0) atomicMin(&first[a], b);
        if (len < 0 || r.pages(len) > p.max_pages) bad |= KV_ERR_LEN, r.len[b] = 0;
        most = max(most, r.held(b));
    }
    atomicMax(&s_most, most);
    __syncthreads();
    most = s_most;
    int need = 0;                                              // copies, in the order of the rows
    for (int base = 0; base < n; base += kPlanThreads) {
        const int b = base + threadIdx.x;
        const bool k = b < n && r.parent[b] >= 0 && (r.len[r.parent[b]] & (T - 1)) != 0 && first[r.parent[b]] != b;
        int total;
        const int at = need + block_scan((int)k, s_warp, &total);
        if (b < n) r.copy[b] = k ? at : -1;
        need += total;
    }
    __syncthreads();
    // this block's columns; they stay in shared memory if they fit
    const int each = (most + ranks - 1) / ranks, from = min(rank * each, most), to = min(from + each, most);
    const bool fits = to - from <= cols;
    for (int c0 = from; c0 < to; c0 += cols) {
        const int nc = min(cols, to - c0);
        if (c0 > from) __syncthreads();
        reorder_load(p, r, c0, nc, s_cells);
        __syncthreads();
        for (int i = threadIdx.x; i < n * nc; i += kPlanThreads) {
            const int b = i / nc, s = c0 + i - b * nc, page = s_cells[i];
            if (s < r.held(b) && (page < 0 || page >= p.n_pages)) bad |= KV_ERR_PAGE;
        }
    }
    if (bad) atomicOr(&s_bad, (int)bad);
    cluster_sync(ranks);
    if (ranks == 1) bad = (unsigned)s_bad;
    else
        for (int i = 0; i < ranks; ++i) bad |= (unsigned)cluster_peer(&s_bad, i);
    if (bad) {                                                 // nothing has changed
        if (rank == 0 && threadIdx.x == 0) {
            kv_error(err, bad);
            ws.plan->n = 0;
        }
        cluster_sync(ranks);                                   // (no block ends while another reads its shared memory)
        return;
    }
    auto count = [&](int sign) {
        for (int c0 = from; c0 < to; c0 += cols) {
            const int nc = min(cols, to - c0);
            if (!fits) {
                __syncthreads();
                reorder_load(p, r, c0, nc, s_cells);
                __syncthreads();
            }
            reorder_refs(p, r, c0, nc, s_cells, sign);
        }
    };
    count(1);
    __threadfence();
    cluster_sync(ranks);
    if (rank == 0) {
        const bool enough = find_free(p.refs, p.n_pages, need, ws.dst, s_warp);
        if (enough) {
            for (int b = threadIdx.x; b < n; b += kPlanThreads)
                if (r.copy[b] >= 0) {
                    p.refs[ws.dst[r.copy[b]]] = 1;
                    ws.list[r.copy[b]] = ((r.new_len(b) & (T - 1)) + kKB - 1) / kKB;
                }
        }
        if (threadIdx.x == 0) {
            ws.plan->n = enough ? need : 0;
            s_bad = !enough;
            if (!enough) kv_error(err, KV_ERR_FULL);
        }
    }
    cluster_sync(ranks);
    if (ranks == 1 ? s_bad : cluster_peer(&s_bad, 0)) {        // too few pages: the counts go back
        count(-1);
        cluster_sync(ranks);
        return;
    }
    for (int c0 = from; c0 < to; c0 += cols) {
        const int nc = min(cols, to - c0);
        if (!fits) {
            __syncthreads();
            reorder_load(p, r, c0, nc, s_cells);
            __syncthreads();
        }
        for (int i = threadIdx.x; i < n * nc; i += kPlanThreads) {
            const int b = i / nc, s = c0 + i - b * nc, up = r.parent[b], now = r.pages(r.new_len(b));
            int page = up >= 0 ? s_cells[up * nc + s - c0] : -1;
            if (s == now - 1 && r.copy[b] >= 0) {
                ws.src[r.copy[b]] = page;
                page = ws.dst[r.copy[b]];
            }
            if (page != s_cells[i] && s < max(r.held(b), now)) p.table[(int64_t)b * p.max_pages + s] = page;
        }
    }
    if (rank == 0)                                             // (all have read the lengths)
        for (int b = threadIdx.x; b < n; b += kPlanThreads) p.len[b] = r.new_len(b);
    cluster_sync(ranks);
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

// The used blocks of partly filled pages, a warp for each: a unit is a block of 32 slots of one (page, layer) and one of its 2 H runs of codes (a page's first takes the
// scales too), 2 or 4 KB that fly together.  Two warps a block: 16 rows forked into 48 and those released 34.6 us, 96 rows reordered 18.2, one row forked and released 9.1
// (four warps 34.5, 17.9, 9.7; one 37.6, 18.6, 9.1; a block of eight for a whole run 40.2, 19.9, 9.4).
constexpr int kUsedWarps = 2;
__global__ void __launch_bounds__(32 * kUsedWarps) kv_copy_used_kernel(KvPages p, Ws ws) {
    grid_dep_launch();
    grid_dep_wait();
    const int n = ws.plan->n, T = 1 << p.tshift, runs = 2 * p.H, lane = threadIdx.x & 31, shift = p.tshift - 5, pieces = p.D / 16;
    // (every unit has 2 KB of the pool to itself, so their number has 32 bits)
    const uint32_t units = ((uint32_t)n * p.n_layers * runs) << shift;
    for (uint32_t u = blockIdx.x * kUsedWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kUsedWarps) {
        const int block = u & ((1 << shift) - 1);
        const uint32_t page = (u >> shift) / runs, i = page / p.n_layers;
        const int run = (u >> shift) - page * runs, layer = page - i * p.n_layers;
        const int used = ws.list[i], from = ws.src[i], to = ws.dst[i];
        if (block >= used) continue;
        const uint8_t *s = p.pool + from * p.page_bytes + layer * p.layer_bytes;
        uint8_t *d = p.pool + to * p.page_bytes + layer * p.layer_bytes;
        const int at = (run * T + block * kKB) * p.D + lane * 16;
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < pieces) v[e] = __ldcs(reinterpret_cast<const uint4 *>(s + at + e * 512));
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < pieces) *reinterpret_cast<uint4 *>(d + at + e * 512) = v[e];
        if (run == 0 && block == 0)
            for (int j = lane; j < runs * (T / kKB); j += 32)
                reinterpret_cast<uint32_t *>(d + p.off_s)[j] = reinterpret_cast<const uint32_t *>(s + p.off_s)[j];
    }
}

// its launch, for up to n copies
int launch_copy_used(const KvPages &p, const Ws &w, int64_t n, const char *what, cudaStream_t s) {
    const int64_t blocks = (((n * p.n_layers * 2 * p.H) << (p.tshift - 5)) + kUsedWarps - 1) / kUsedWarps;
    const int grid = (int)(blocks < 32 * sm_count() ? blocks : 32 * sm_count());
    return cuda_error(launch_pdl(kv_copy_used_kernel, dim3(grid), dim3(32 * kUsedWarps), 0, s, p, w), what);
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
    return launch_copy_used(p, w, n, "mqkv_fork copy launch", s);
}

int kv_launch_reorder(const KvPages &p, const int32_t *parent, void *ws, unsigned int *err, cudaStream_t s) {
    const Ws w(ws, p.n_pages, p.n_seqs);
    const int fit = kReorderCells / p.n_seqs, cols = fit < p.max_pages ? fit : p.max_pages;     // (8 at least where there are as many)
    const int smem = (4 * p.n_seqs + cols * p.n_seqs) * 4;
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(kv_reorder_kernel), (4 * kKvReorderRows + kReorderCells) * 4, kAttrSlotReorder);
    if (rc != MQ_OK) return rc;
    // One block for a small table, a cluster where there is much to check and to move.  Both kernels in a graph, one block and eight: 256 cells 7.9 and 10.1 us, 1024 8.9 and
    // 10.7, 2048 9.9 and 10.8, 4096 12.2 and 10.3, 16384 26 and 12.
    const unsigned blocks = (int64_t)p.n_seqs * p.max_pages <= 2048 ? 1 : kReorderCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    rc = cuda_error(cudaLaunchKernelEx(&cfg, kv_reorder_kernel, p, parent, w, cols, err), "mqkv_reorder plan launch");
    if (rc != MQ_OK) return rc;
    return launch_copy_used(p, w, p.n_seqs, "mqkv_reorder copy launch", s);
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

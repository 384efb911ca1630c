// Page bookkeeping of the paged cache: fork (reorder, grow, shorten, free) and
// compaction, and the page copies that they ask for.
//
// The bookkeeping is a few passes over the tables and over one word per page,
// with a whole-table dependency between them (which pages are free is known
// when every row has said what it keeps).  One cluster of 8 thread blocks does
// them all: cluster barriers separate the passes, so one launch replaces five,
// and 4096 threads hide the latency of the scattered counter updates.  Prefix
// sums (rows -> first dealt page, pages -> rank among the free) run over
// contiguous ranges: a thread sums its range, the block and then the cluster
// scan the sums, and a second walk over the range hands out the numbers, so the
// result does not depend on the order of any atomic.
//
// The copies are bound by memory traffic: a second kernel moves whole pages of
// all ranks and layers in 16-byte words, its work list being on the device.
#include <algorithm>
#include <climits>

#include "kv4.cuh"

namespace tpk {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kAll = kCluster * kThreads;

// Workspace: counts, then per-page and per-row words.
struct PagesWs {
    int32_t* head;       // [0] number of copies
    int32_t* writers;    // [pages] rows that will write inside the page (fork)
    int32_t* first;      // [pages] the first of them (fork); new number (compact)
    int32_t* free_list;  // [pages]
    int32_t* src;        // [rows or pages] page copies
    int32_t* dst;
    int32_t* copy_at;    // [rows] 0: no copy; else 1 + its number, or -1 when no page is left (fork)
    int32_t* deal_at;    // [rows] first of its dealt pages (fork)
};

__host__ __device__ inline PagesWs carve(void* ws, int64_t rows, int64_t pages) {
    PagesWs w;
    int32_t* p = static_cast<int32_t*>(ws);
    const int64_t lists = rows > pages ? rows : pages;
    w.head = p;
    w.writers = p + 64;
    w.first = w.writers + pages;
    w.free_list = w.first + pages;
    w.src = w.free_list + pages;
    w.dst = w.src + lists;
    w.copy_at = w.dst + lists;
    w.deal_at = w.copy_at + rows;
    return w;
}

__device__ __forceinline__ void st_cluster_i32(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Exclusive prefix sums over all threads of the cluster of two counts, in
// thread order; also the totals.  Every thread of the cluster calls it.
struct Scan2 {
    int a, b, total_a, total_b;
};
__device__ Scan2 cluster_scan(int a, int b, int (*block_sums)[2], int (*warp_sums)[2]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int ia = a, ib = b;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int va = __shfl_up_sync(0xffffffffu, ia, m), vb = __shfl_up_sync(0xffffffffu, ib, m);
        if (lane >= m) ia += va, ib += vb;
    }
    if (lane == 31) warp_sums[warp][0] = ia, warp_sums[warp][1] = ib;
    __syncthreads();
    int ba = 0, bb = 0, ta = 0, tb = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        const int va = warp_sums[i][0], vb = warp_sums[i][1];
        if (i < warp) ba += va, bb += vb;
        ta += va, tb += vb;
    }
    const uint32_t rank = cluster_ctarank();
    if (tid < kCluster) {            // this block's sums into every block's list
        const uint32_t to = mapa_shared(smem_u32(&block_sums[rank][0]), tid);
        st_cluster_i32(to, ta);
        st_cluster_i32(to + 4, tb);
    }
    cluster_sync();
    Scan2 s{ba + ia - a, bb + ib - b, 0, 0};
    for (uint32_t i = 0; i < kCluster; ++i) {
        const int va = block_sums[i][0], vb = block_sums[i][1];
        if (i < rank) s.a += va, s.b += vb;
        s.total_a += va, s.total_b += vb;
    }
    cluster_sync();                  // before the lists are written again
    return s;
}

// What output row i keeps of its parent and wants.
struct RowPlan {
    int parent;          // -1: none
    int kept, want;      // entries
    int len;             // tokens of the new row
    bool writes;         // inside the last kept page
};
__device__ __forceinline__ RowPlan row_plan(const KvPagesDesc& d, int i) {
    RowPlan r{-1, 0, 0, 0, false};
    const int p = d.parents[i];
    if (p < 0 || p >= d.rows_in) return r;
    const int64_t room = d.max_blocks * d.page_size;
    const int64_t have = min(max(static_cast<int64_t>(d.lens[p]), static_cast<int64_t>(0)), room);
    const int64_t grow = d.grow != nullptr ? d.grow[i] : d.grow_all;
    const int64_t len = min(max(have + grow, static_cast<int64_t>(0)), room);
    const int64_t keep = min(have, len);
    r.parent = p;
    r.kept = static_cast<int>((keep + d.page_size - 1) / d.page_size);
    r.want = static_cast<int>((len + d.page_size - 1) / d.page_size);
    r.len = static_cast<int>(len);
    r.writes = keep % d.page_size != 0 && len > keep;
    return r;
}

__device__ __forceinline__ bool is_free(const KvPagesDesc& d, int p) {
    return __ldcg(&d.refs[p]) == 0 && (d.held == nullptr || d.held[p] == 0);
}

// The contiguous range of n things that thread `id` of the cluster walks.
struct Range {
    int lo, hi;
};
__device__ __forceinline__ Range my_range(int n, int id) {
    const int per = (n + kAll - 1) / kAll;
    const int64_t lo = static_cast<int64_t>(id) * per;
    return {static_cast<int>(min(lo, static_cast<int64_t>(n))), static_cast<int>(min(lo + per, static_cast<int64_t>(n)))};
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) kv_fork_kernel(KvPagesDesc d) {
    __shared__ int block_sums[kCluster][2];
    __shared__ int warp_sums[kThreads / 32][2];
    const PagesWs w = carve(d.ws, d.rows_out, d.pages);
    const int id = blockIdx.x * kThreads + threadIdx.x;
    pdl_wait();
    pdl_trigger();

    for (int p = id; p < d.pages; p += kAll) {
        d.refs[p] = 0;
        w.writers[p] = 0;
        w.first[p] = INT_MAX;
    }
    if (id < 4) d.info[id] = 0;
    cluster_sync();

    // every row's kept pages: count them, note who will write where; a warp per row
    const int lane = threadIdx.x & 31;
    int bad = 0;
    for (int i = id >> 5; i < d.rows_out; i += kAll / 32) {
        const RowPlan r = row_plan(d, i);
        const int32_t* from = d.table + static_cast<int64_t>(max(r.parent, 0)) * d.max_blocks;
        int32_t* to = d.table_out + static_cast<int64_t>(i) * d.max_blocks;
        for (int c = lane; c < d.max_blocks; c += 32) {
            int page = -1;
            if (c < r.kept) {
                page = from[c];
                if (page < 0 || page >= d.pages) {
                    page = -1;
                    ++bad;
                } else {
                    atomicAdd(&d.refs[page], 1);
                    if (r.writes && c == r.kept - 1) {
                        atomicAdd(&w.writers[page], 1);
                        atomicMin(&w.first[page], i);
                    }
                }
            }
            to[c] = page;
        }
        if (lane == 0) d.lens_out[i] = r.len;
    }
    if (bad) {
        atomicAdd(&d.info[3], bad);
        atomicAdd(&d.info[1], bad);
    }
    cluster_sync();

    // what is free, what every row needs; a thread walks its range of pages and of rows
    const Range pr = my_range(d.pages, id), rr = my_range(d.rows_out, id);
    int free_here = 0, need_here = 0;
    for (int p = pr.lo; p < pr.hi; ++p) free_here += is_free(d, p);
    for (int i = rr.lo; i < rr.hi; ++i) {
        const RowPlan r = row_plan(d, i);
        int copy = 0;
        if (r.writes) {
            const int page = __ldcg(&d.table_out[static_cast<int64_t>(i) * d.max_blocks + r.kept - 1]);
            // alone: all who keep the page write in it (the others will get copies), and this row is the first
            if (page >= 0)
                copy = !(__ldcg(&d.refs[page]) == __ldcg(&w.writers[page]) && __ldcg(&w.first[page]) == i &&
                         (d.held == nullptr || d.held[page] == 0));
        }
        w.copy_at[i] = copy;
        need_here += r.want - r.kept + copy;
    }
    const Scan2 sc = cluster_scan(free_here, need_here, block_sums, warp_sums);
    const int have = sc.total_a;
    if (free_here > 0) {
        int rank = sc.a;
        for (int p = pr.lo; p < pr.hi; ++p)
            if (is_free(d, p)) w.free_list[rank++] = p;
    }
    // the first deal of each row; a copy is made when its page can be had
    int copies_here = 0, k = sc.b;
    for (int i = rr.lo; i < rr.hi; ++i) {
        const RowPlan r = row_plan(d, i);
        const int copy = w.copy_at[i];
        w.deal_at[i] = k;
        copies_here += copy != 0 && k < have;
        k += r.want - r.kept + copy;
    }
    const Scan2 cc = cluster_scan(copies_here, pr.hi - pr.lo - free_here, block_sums, warp_sums);
    {
        int c = cc.a;
        for (int i = rr.lo; i < rr.hi; ++i)
            if (w.copy_at[i] != 0) w.copy_at[i] = w.deal_at[i] < have ? ++c : -1;   // 1 + its number, -1: no page
    }
    if (id == 0) {
        w.head[0] = cc.total_a;
        d.info[2] = cc.total_a;
        d.info[0] = cc.total_b + min(have, sc.total_b);
    }
    cluster_sync();

    // deal the pages out; a warp per row
    int missing = 0;
    for (int i = id >> 5; i < d.rows_out; i += kAll / 32) {
        const RowPlan r = row_plan(d, i);
        const int copy = __ldcg(&w.copy_at[i]), deal = __ldcg(&w.deal_at[i]);
        int32_t* to = d.table_out + static_cast<int64_t>(i) * d.max_blocks;
        if (lane == 0 && copy != 0) {
            const int src = __ldcg(&to[r.kept - 1]);
            const int dst = copy > 0 ? __ldcg(&w.free_list[deal]) : -1;
            if (copy > 0) {
                w.src[copy - 1] = src;
                w.dst[copy - 1] = dst;
                d.refs[dst] = 1;
            } else {
                ++missing;
            }
            atomicSub(&d.refs[src], 1);
            to[r.kept - 1] = dst;
        }
        const int fresh = deal + (copy != 0);
        for (int c = r.kept + lane; c < r.want; c += 32) {
            const int at = fresh + c - r.kept;
            const int page = at < have ? __ldcg(&w.free_list[at]) : -1;
            to[c] = page;
            if (page >= 0)
                d.refs[page] = 1;
            else
                ++missing;
        }
    }
    if (missing) atomicAdd(&d.info[1], missing);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) kv_compact_kernel(KvPagesDesc d) {
    __shared__ int block_sums[kCluster][2];
    __shared__ int warp_sums[kThreads / 32][2];
    const PagesWs w = carve(d.ws, d.rows_out, d.pages);
    const int id = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();

    for (int p = id; p < d.pages; p += kAll) {
        d.refs[p] = 0;
        w.first[p] = p;
    }
    if (id < 4) d.info[id] = 0;
    cluster_sync();

    int bad = 0;
    for (int i = id >> 5; i < d.rows_in; i += kAll / 32) {
        const int64_t len = min(max(static_cast<int64_t>(d.lens[i]), static_cast<int64_t>(0)), d.max_blocks * d.page_size);
        const int used = static_cast<int>((len + d.page_size - 1) / d.page_size);
        const int32_t* from = d.table + static_cast<int64_t>(i) * d.max_blocks;
        int32_t* to = d.table_out + static_cast<int64_t>(i) * d.max_blocks;
        for (int c = lane; c < d.max_blocks; c += 32) {
            int page = c < used ? from[c] : -1;
            if (c < used && (page < 0 || page >= d.pages)) {
                page = -1;
                ++bad;
            }
            if (page >= 0) atomicAdd(&d.refs[page], 1);
            to[c] = page;
        }
    }
    if (bad) {
        atomicAdd(&d.info[1], bad);
        atomicAdd(&d.info[3], bad);
    }
    cluster_sync();

    const Range pr = my_range(d.pages, id);
    int live_here = 0;
    for (int p = pr.lo; p < pr.hi; ++p) live_here += !is_free(d, p);
    const int live = cluster_scan(live_here, 0, block_sums, warp_sums).total_a;
    auto moves = [&](int p) { return p >= live && __ldcg(&d.refs[p]) != 0 && (d.held == nullptr || d.held[p] == 0); };
    int movers = 0, holes = 0;
    for (int p = pr.lo; p < pr.hi; ++p) {
        movers += moves(p);
        holes += p < live && is_free(d, p);
    }
    const Scan2 sc = cluster_scan(movers, holes, block_sums, warp_sums);
    int m = sc.a, h = sc.b;
    for (int p = pr.lo; p < pr.hi; ++p) {
        if (moves(p)) w.src[m++] = p;
        if (p < live && is_free(d, p)) w.free_list[h++] = p;
    }
    if (id == 0) {
        w.head[0] = sc.total_a;
        d.info[0] = live;
        d.info[2] = sc.total_a;
    }
    cluster_sync();
    // as many holes below `live` as pages in use at or above it, so every mover has one
    for (int k = id; k < sc.total_a; k += kAll) {
        const int src = __ldcg(&w.src[k]), dst = __ldcg(&w.free_list[k]);
        w.dst[k] = dst;
        w.first[src] = dst;
        d.refs[dst] = __ldcg(&d.refs[src]);
        d.refs[src] = 0;
    }
    cluster_sync();
    for (int i = id >> 5; i < d.rows_in; i += kAll / 32) {
        int32_t* to = d.table_out + static_cast<int64_t>(i) * d.max_blocks;
        for (int c = lane; c < d.max_blocks; c += 32) {
            const int page = __ldcg(&to[c]);
            if (page < 0) continue;
            const int now = __ldcg(&w.first[page]);
            if (now != page) to[c] = now;
        }
    }
}

// Page copies: one thread block per (copy, rank, layer) at a time, 16-byte words, eight in flight per thread.
constexpr int kCopyThreads = 128;
constexpr int kCopyUnroll = 8;

__global__ void __launch_bounds__(kCopyThreads) kv_copy_pages_kernel(KvPagesDesc d) {
    const PagesWs w = carve(d.ws, d.rows_out, d.pages);
    pdl_wait();
    pdl_trigger();
    const int64_t words = d.page_bytes / 16;
    const int64_t per_copy = d.t * d.layers;
    const int64_t units = w.head[0] * per_copy;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t k = u / per_copy;
        const int rest = static_cast<int>(u - k * per_copy);
        const int r = static_cast<int>(rest / d.layers);
        const int64_t layer = rest - r * d.layers;
        uint8_t* base = d.pool[r] + layer * d.pages * d.page_bytes;
        const uint4* src = reinterpret_cast<const uint4*>(base + w.src[k] * d.page_bytes);
        uint4* dst = reinterpret_cast<uint4*>(base + w.dst[k] * d.page_bytes);
        for (int64_t i = threadIdx.x; i < words; i += kCopyThreads * kCopyUnroll) {
            uint4 v[kCopyUnroll];
#pragma unroll
            for (int j = 0; j < kCopyUnroll; ++j)
                if (i + j * kCopyThreads < words) v[j] = src[i + j * kCopyThreads];
#pragma unroll
            for (int j = 0; j < kCopyUnroll; ++j)
                if (i + j * kCopyThreads < words) dst[i + j * kCopyThreads] = v[j];
        }
    }
}

template <typename Kern>
tp_status launch_pages(const KvPagesDesc& d, Kern kern, cudaStream_t stream) {
    if (launch_pdl(kern, dim3(kCluster), dim3(kThreads), 0, stream, d) != cudaSuccess) return TP_ERR_CUDA;
    if (!d.with_pool) return TP_OK;
    const int sms = device_sms();
    if (sms <= 0) return TP_ERR_CUDA;
    if (launch_pdl(kv_copy_pages_kernel, dim3(sms * 12), dim3(kCopyThreads), 0, stream, d) != cudaSuccess)
        return TP_ERR_CUDA;
    return TP_OK;
}

}  // namespace

size_t kv_pages_workspace(int64_t rows, int64_t pages) {
    const int64_t lists = std::max(rows, pages);
    return static_cast<size_t>(64 + 3 * pages + 2 * lists + 2 * rows) * 4;
}

tp_status launch_kv_fork(const KvPagesDesc& d, cudaStream_t stream) { return launch_pages(d, kv_fork_kernel, stream); }
tp_status launch_kv_compact(const KvPagesDesc& d, cudaStream_t stream) {
    return launch_pages(d, kv_compact_kernel, stream);
}

}  // namespace tpk

// Page bookkeeping of the paged cache: fork (reorder, grow, shorten, free) and
// compaction, and the page copies that they ask for.
//
// The bookkeeping is a few passes over the tables and over one word per page,
// with a whole-table dependency between them (which pages are free is known
// when every row has said what it keeps): a chain of latencies.  Small
// tables over at most 12288 pages are done by one thread block that keeps the
// pages' counters and the rows' plans in shared memory, so that only the reading
// of lengths and tables goes through global memory.  Larger ones take one cluster of 8
// thread blocks with the counters in global memory: cluster barriers separate
// the passes, and 4096 threads hide the latency of the scattered updates.
// Prefix sums (rows -> first dealt page, pages -> rank among the free) run over
// contiguous ranges: a thread sums its range, the threads scan the sums, and a
// second walk over the range hands out the numbers, so the result does not depend
// on the order of any atomic.
//
// The copies are bound by memory traffic: a second kernel moves whole pages of
// all ranks and layers in 16-byte words, its work list being on the device (6.5
// TB/s read and written together where a compaction moves 397 MB).  With both
// kernels a fork of 8 rows takes 6.8 us, of 256 rows with 128 copies of four
// layers 24 us.
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

// ------------------------------------------------------------------ one thread block, counters in shared memory

constexpr int kOne = 1024;           // threads
// What the counters fit and what one block is faster with.  It takes 6.2 us for a fork of 64 rows of 39 entries over
// 2996 pages (the cluster 11.5), 10.0 for 256 rows over 10484 (15.4), 17.3 for 512 of 60 over 12288 (19.0), and
// 26.6 for 1024 (26.4); a compaction 6.3 (10.4), 12.2 (15.3), 20.5 (17.0), and 16.7 for 512 of 40 (16.9).
constexpr int kFewPages = 12288, kFewRows = 2048, kFewFork = 32768, kFewCompact = 16384;
constexpr int kFewSmem = kFewPages * 12 + kFewRows * 24;

// Exclusive prefix sums over the block's threads, in thread order, and the totals.
__device__ __forceinline__ Scan2 block_scan(int a, int b, int (*warp_sums)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ia = a, ib = b;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int va = __shfl_up_sync(0xffffffffu, ia, m), vb = __shfl_up_sync(0xffffffffu, ib, m);
        if (lane >= m) ia += va, ib += vb;
    }
    if (lane == 31) warp_sums[warp][0] = ia, warp_sums[warp][1] = ib;
    __syncthreads();
    int wa = warp_sums[lane][0], wb = warp_sums[lane][1];        // as many warps as lanes
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int va = __shfl_up_sync(0xffffffffu, wa, m), vb = __shfl_up_sync(0xffffffffu, wb, m);
        if (lane >= m) wa += va, wb += vb;
    }
    Scan2 s;
    s.total_a = __shfl_sync(0xffffffffu, wa, 31);
    s.total_b = __shfl_sync(0xffffffffu, wb, 31);
    const int pa = __shfl_sync(0xffffffffu, wa, (warp + 31) & 31), pb = __shfl_sync(0xffffffffu, wb, (warp + 31) & 31);
    s.a = (warp ? pa : 0) + ia - a;
    s.b = (warp ? pb : 0) + ib - b;
    __syncthreads();                 // before the sums are written again
    return s;
}

__device__ __forceinline__ Range one_range(int n) {
    const int per = (n + kOne - 1) / kOne, lo = min(n, static_cast<int>(threadIdx.x) * per);
    return {lo, min(n, lo + per)};
}

// f(row, column, entry) for every place of a table of `rows` rows, the entry being at(row, column) (or what it likes
// for a place that has none); four entries of a thread are on their way at once.  e / max_blocks by a
// multiplication, exact for e < 2^16.
template <typename At, typename F>
__device__ __forceinline__ void each_entry(int rows, int max_blocks, At at, F f) {
    constexpr int BATCH = 4;
    const float inv = 1.0f / static_cast<float>(max_blocks);
    const int n = rows * max_blocks;
    for (int e0 = threadIdx.x; e0 < n; e0 += BATCH * kOne) {
        int row[BATCH], col[BATCH], got[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int e = e0 + j * kOne;
            row[j] = static_cast<int>((static_cast<float>(e) + 0.5f) * inv);
            col[j] = e - row[j] * max_blocks;
            got[j] = e < n ? at(row[j], col[j]) : -1;
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (e0 + j * kOne < n) f(row[j], col[j], got[j]);
    }
}

__global__ void __launch_bounds__(kOne) kv_fork_few_kernel(const __grid_constant__ KvPagesDesc d) {
    extern __shared__ int few[];
    __shared__ int warp_sums[32][2];
    __shared__ int s_bad, s_missing;
    const int tid = threadIdx.x, mb = static_cast<int>(d.max_blocks);
    uint32_t* counts = reinterpret_cast<uint32_t*>(few);         // [pages] rows that keep the page, << 16 those that write in it
    int* first = few + d.pages;                                  // [pages] the first of the latter
    int* list = first + d.pages;                                 // [pages] free pages
    int* kept = list + d.pages;                                  // [rows] entries kept, << 1, and whether the row writes
    int* want = kept + d.rows_out;
    int* from = want + d.rows_out;                               // parent
    int* tail = from + d.rows_out;                               // the last kept page, -1: none
    int* deal = tail + d.rows_out;                               // first dealt page
    int* copy = deal + d.rows_out;                               // 0, 1 + the copy's number, -1: no page for it
    const PagesWs w = carve(d.ws, d.rows_out, d.pages);
    pdl_wait();
    pdl_trigger();
    for (int i = tid; i < d.rows_out; i += kOne) {
        const RowPlan r = row_plan(d, i);
        kept[i] = r.kept << 1 | (r.writes ? 1 : 0);
        want[i] = r.want;
        from[i] = r.parent;
        tail[i] = -1;
        d.lens_out[i] = r.len;
    }
    for (int p = tid; p < d.pages; p += kOne) counts[p] = 0, first[p] = INT_MAX;
    if (tid == 0) s_bad = s_missing = 0;
    __syncthreads();

    int bad = 0;
    auto entry = [&](int i, int c) { return c < kept[i] >> 1 ? __ldg(d.table + static_cast<int64_t>(from[i]) * mb + c) : -1; };
    each_entry(d.rows_out, mb, entry, [&](int i, int c, int page) {
        const int k = kept[i] >> 1;
        if (c < k) {
            if (page < 0 || page >= d.pages) {
                page = -1;
                ++bad;
            } else {
                const bool writes = (kept[i] & 1) && c == k - 1;
                atomicAdd(&counts[page], writes ? 0x10001u : 1u);
                if (writes) atomicMin(&first[page], i);
                if (c == k - 1) tail[i] = page;
            }
        }
        d.table_out[static_cast<int64_t>(i) * mb + c] = page;
    });
    if (bad) atomicAdd(&s_bad, bad);
    __syncthreads();

    const Range pr = one_range(d.pages), rr = one_range(d.rows_out);
    auto held = [&](int p) { return d.held != nullptr && d.held[p] != 0; };
    auto is_free = [&](int p) { return counts[p] == 0 && !held(p); };
    int free_here = 0, need_here = 0;
    for (int p = pr.lo; p < pr.hi; ++p) free_here += is_free(p);
    for (int i = rr.lo; i < rr.hi; ++i) {
        int cp = 0;
        const int page = tail[i];
        // alone: all who keep the page write in it (the others will get copies), and this row is the first
        if ((kept[i] & 1) && page >= 0) cp = !((counts[page] & 0xffffu) == counts[page] >> 16 && first[page] == i && !held(page));
        copy[i] = cp;
        need_here += want[i] - (kept[i] >> 1) + cp;
    }
    const Scan2 sc = block_scan(free_here, need_here, warp_sums);
    const int have = sc.total_a;
    int rank = sc.a, k = sc.b, copies_here = 0;
    if (free_here > 0)
        for (int p = pr.lo; p < pr.hi; ++p)
            if (is_free(p)) list[rank++] = p;
    for (int i = rr.lo; i < rr.hi; ++i) {
        deal[i] = k;
        copies_here += copy[i] != 0 && k < have;
        k += want[i] - (kept[i] >> 1) + copy[i];
    }
    const Scan2 cc = block_scan(copies_here, 0, warp_sums);
    if (tid == 0) {
        w.head[0] = cc.total_a;
        d.info[0] = d.pages - have + min(have, sc.total_b);
        d.info[2] = cc.total_a;
        d.info[3] = s_bad;
    }
    // deal the pages out (the list and every decision are behind the scan's barriers)
    int number = cc.a, missing = 0;
    for (int i = rr.lo; i < rr.hi; ++i) {
        int32_t* to = d.table_out + static_cast<int64_t>(i) * mb;
        const int kp = kept[i] >> 1;
        int at = deal[i];
        if (copy[i] != 0) {
            const int src = tail[i], dst = at < have ? list[at] : -1;
            atomicSub(&counts[src], 1u);
            to[kp - 1] = dst;
            if (dst >= 0) {
                w.src[number] = src;
                w.dst[number++] = dst;
                counts[dst] = 1;
            } else {
                ++missing;
            }
            ++at;
        }
        for (int c = kp; c < want[i]; ++c, ++at) {
            const int page = at < have ? list[at] : -1;
            to[c] = page;
            if (page >= 0)
                counts[page] = 1;
            else
                ++missing;
        }
    }
    if (missing) atomicAdd(&s_missing, missing);
    __syncthreads();
    if (tid == 0) d.info[1] = s_bad + s_missing;
    for (int p = tid; p < d.pages; p += kOne) d.refs[p] = static_cast<int>(counts[p] & 0xffffu);
}

__global__ void __launch_bounds__(kOne) kv_compact_few_kernel(const __grid_constant__ KvPagesDesc d) {
    extern __shared__ int few[];
    __shared__ int warp_sums[32][2];
    __shared__ int s_bad;
    const int tid = threadIdx.x, mb = static_cast<int>(d.max_blocks);
    int* refs = few;                                             // [pages]
    int* to = few + d.pages;                                     // [pages] the page's new number
    int* list = to + d.pages;                                    // [pages] movers from the front, holes from the back
    int* used = list + d.pages;                                  // [rows] entries
    const PagesWs w = carve(d.ws, d.rows_out, d.pages);
    pdl_wait();
    pdl_trigger();
    for (int i = tid; i < d.rows_in; i += kOne) {
        const int64_t len = min(max(static_cast<int64_t>(d.lens[i]), static_cast<int64_t>(0)), d.max_blocks * d.page_size);
        used[i] = static_cast<int>((len + d.page_size - 1) / d.page_size);
    }
    for (int p = tid; p < d.pages; p += kOne) refs[p] = 0, to[p] = p;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    int bad = 0;
    auto entry = [&](int i, int c) { return c < used[i] ? __ldg(d.table + static_cast<int64_t>(i) * mb + c) : -1; };
    each_entry(d.rows_in, mb, entry, [&](int i, int c, int page) {
        if (c >= used[i]) return;
        if (page < 0 || page >= d.pages)
            ++bad;
        else
            atomicAdd(&refs[page], 1);
    });
    if (bad) atomicAdd(&s_bad, bad);
    __syncthreads();
    const Range pr = one_range(d.pages);
    auto held = [&](int p) { return d.held != nullptr && d.held[p] != 0; };
    int live_here = 0;
    for (int p = pr.lo; p < pr.hi; ++p) live_here += refs[p] != 0 || held(p);
    const int live = block_scan(live_here, 0, warp_sums).total_a;
    int movers = 0, holes = 0;
    for (int p = pr.lo; p < pr.hi; ++p) {
        movers += p >= live && refs[p] != 0 && !held(p);
        holes += p < live && refs[p] == 0 && !held(p);
    }
    // as many holes below `live` as pages in use at or above it, so that every mover has one
    const Scan2 sc = block_scan(movers, holes, warp_sums);
    int m = sc.a, h = sc.b;
    for (int p = pr.lo; p < pr.hi; ++p) {
        if (p >= live && refs[p] != 0 && !held(p)) list[m++] = p;
        if (p < live && refs[p] == 0 && !held(p)) list[d.pages - 1 - h++] = p;
    }
    __syncthreads();
    for (int k = tid; k < sc.total_a; k += kOne) {
        const int src = list[k], dst = list[d.pages - 1 - k];
        w.src[k] = src;
        w.dst[k] = dst;
        to[src] = dst;
        refs[dst] = refs[src];
        refs[src] = 0;
    }
    if (tid == 0) {
        w.head[0] = sc.total_a;
        d.info[0] = live;
        d.info[1] = d.info[3] = s_bad;
        d.info[2] = sc.total_a;
    }
    __syncthreads();
    each_entry(d.rows_in, mb, entry, [&](int i, int c, int page) {
        d.table_out[static_cast<int64_t>(i) * mb + c] = page < 0 || page >= d.pages ? -1 : to[page];
    });
    for (int p = tid; p < d.pages; p += kOne) d.refs[p] = refs[p];
}

bool is_few(const KvPagesDesc& d, int64_t entries) {
    return d.pages <= kFewPages && d.rows_out <= kFewRows && d.rows_out * d.max_blocks <= entries;
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

template <typename Few, typename Many>
tp_status launch_pages(const KvPagesDesc& d, int64_t entries, Few few, Many many, std::atomic<uint64_t>& smem_set, cudaStream_t stream) {
    if (is_few(d, entries)) {
        if (!smem_attribute_once(reinterpret_cast<const void*>(few), kFewSmem, smem_set)) return TP_ERR_CUDA;
        const size_t smem = (static_cast<size_t>(d.pages) * 3 + static_cast<size_t>(d.rows_out) * 6) * 4;
        if (launch_pdl(few, dim3(1), dim3(kOne), smem, stream, d) != cudaSuccess) return TP_ERR_CUDA;
    } else if (launch_pdl(many, dim3(kCluster), dim3(kThreads), 0, stream, d) != cudaSuccess) {
        return TP_ERR_CUDA;
    }
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

tp_status launch_kv_fork(const KvPagesDesc& d, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    return launch_pages(d, kFewFork, kv_fork_few_kernel, kv_fork_kernel, smem_set, stream);
}
tp_status launch_kv_compact(const KvPagesDesc& d, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    return launch_pages(d, kFewCompact, kv_compact_few_kernel, kv_compact_kernel, smem_set, stream);
}

}  // namespace tpk

// C ABI of the decode-loop operators: argument validation and descriptors.
// See include/tp.h for the contract.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "tp.h"

namespace {

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline cudaStream_t cs(tp_stream s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }
inline bool head_dim_ok(int d) { return d == 64 || d == 128; }

// Sizes that keep row, position and block numbers within 31 bits.
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kMaxKvHeads = 1024;

#define TP_CHECK(cond, code) \
    do {                     \
        if (!(cond)) return (code); \
    } while (0)

// The checks that append, load and attention share; fills seqs and pools.
tp_status check_cache(int t, int64_t n, int64_t nseq, int kv_heads, int head_dim, void* const* pool, int64_t pages,
                      int page_size, const int32_t* table, int64_t max_blocks, const int32_t* lens,
                      const int32_t* cu_rows, tpk::KvSeqs& seqs, tpk::KvPools& pools) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(n >= 0 && nseq >= 0 && kv_heads >= 1 && pages >= 1 && max_blocks >= 1, TP_ERR_INVALID_ARG);
    TP_CHECK(head_dim_ok(head_dim) && page_size_ok(page_size) && kv_heads <= kMaxKvHeads, TP_ERR_UNSUPPORTED);
    TP_CHECK(n <= kMaxRows && nseq <= kMaxRows && pages <= INT32_MAX && max_blocks <= kMaxRows / page_size,
             TP_ERR_UNSUPPORTED);
    TP_CHECK(pool != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(cu_rows != nullptr || n == nseq, TP_ERR_INVALID_ARG);
    TP_CHECK(n == 0 || nseq > 0, TP_ERR_INVALID_ARG);
    TP_CHECK(n == 0 || (table != nullptr && lens != nullptr), TP_ERR_INVALID_ARG);
    pools.t = t;
    pools.pages = pages;
    pools.kv_heads = kv_heads;
    pools.page_shift = 0;
    while ((tpk::kKvBlock << pools.page_shift) < page_size) ++pools.page_shift;
    for (int r = 0; r < t; ++r) {
        TP_CHECK(pool[r] != nullptr, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(pool[r]), TP_ERR_ALIGNMENT);
        pools.pool[r] = static_cast<uint8_t*>(pool[r]);
    }
    seqs.n = static_cast<int>(n);
    seqs.nseq = static_cast<int>(nseq);
    seqs.table = table;
    seqs.max_blocks = max_blocks;
    seqs.lens = lens;
    seqs.cu_rows = cu_rows;
    return TP_OK;
}

// A list of t row-major matrices of `width` elements of `elem` bytes, 16-byte aligned rows.
tp_status check_rows(int t, int64_t n, const void* const* x, int64_t ld, int64_t width, int elem) {
    TP_CHECK(x != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(ld >= width, TP_ERR_INVALID_ARG);
    TP_CHECK((ld * elem) % 16 == 0, TP_ERR_ALIGNMENT);
    for (int r = 0; r < t; ++r) {
        TP_CHECK(x[r] != nullptr || n == 0, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(x[r]), TP_ERR_ALIGNMENT);
    }
    return TP_OK;
}

}  // namespace

int tpk::device_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    static std::atomic<int> cache[64];
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

extern "C" {

size_t tp_kv4_page_bytes(int page_size, int kv_heads, int head_dim) {
    if (!page_size_ok(page_size) || !head_dim_ok(head_dim) || kv_heads < 1 || kv_heads > kMaxKvHeads) return 0;
    return static_cast<size_t>(kv_heads) * page_size * (head_dim + 8);
}

int64_t tp_debug_kv4_block(const int32_t* row, int64_t max_blocks, int64_t pages, int page_size, int kv_heads,
                           int head_dim, int head, int64_t position) {
    if (row == nullptr || tp_kv4_page_bytes(page_size, kv_heads, head_dim) == 0 || head < 0 || head >= kv_heads ||
        max_blocks < 0 || position < 0)
        return -1;
    int shift = 0;
    while ((tpk::kKvBlock << shift) < page_size) ++shift;
    return tpk::kv_block_offset(row, max_blocks, pages, shift, kv_heads, head, position / tpk::kKvBlock,
                                tpk::kKvBlock * (head_dim + 8));
}

tp_status tp_kv4_append(int t, int64_t n, int64_t nseq, int kv_heads, int head_dim, const void* const* k, int64_t ldk,
                        const void* const* v, int64_t ldv, void* const* pool, int64_t pages, int page_size,
                        const int32_t* table, int64_t max_blocks, const int32_t* lens, const int32_t* cu_rows,
                        tp_stream stream) {
    tpk::KvAppendDesc d;
    tp_status s = check_cache(t, n, nseq, kv_heads, head_dim, pool, pages, page_size, table, max_blocks, lens, cu_rows,
                              d.seqs, d.pools);
    TP_CHECK(s == TP_OK, s);
    const int64_t width = static_cast<int64_t>(kv_heads) * head_dim;
    s = check_rows(t, n, k, ldk, width, 2);
    TP_CHECK(s == TP_OK, s);
    s = check_rows(t, n, v, ldv, width, 2);
    TP_CHECK(s == TP_OK, s);
    if (n == 0) return TP_OK;
    for (int r = 0; r < t; ++r) {
        d.k[r] = k[r];
        d.v[r] = v[r];
    }
    d.head_dim = head_dim;
    d.ldk = ldk;
    d.ldv = ldv;
    d.seqs.status = tpk::device_status_word();
    return tpk::launch_kv4_append(d, cs(stream));
}

tp_status tp_kv4_load(int t, int64_t n, int64_t nseq, int kv_heads, int head_dim, const void* const* pool,
                      int64_t pages, int page_size, const int32_t* table, int64_t max_blocks, const int32_t* lens,
                      const int32_t* cu_rows, void* const* k, int64_t ldk, void* const* v, int64_t ldv, tp_dtype dtype,
                      tp_stream stream) {
    tpk::KvLoadDesc d;
    // the pools are only read; the descriptor is shared with the append
    tp_status s = check_cache(t, n, nseq, kv_heads, head_dim, const_cast<void* const*>(pool), pages, page_size, table,
                              max_blocks, lens, cu_rows, d.seqs, d.pools);
    TP_CHECK(s == TP_OK, s);
    TP_CHECK(dtype == TP_BF16 || dtype == TP_F32, TP_ERR_UNSUPPORTED);
    TP_CHECK(k != nullptr || v != nullptr, TP_ERR_INVALID_ARG);
    const int64_t width = static_cast<int64_t>(kv_heads) * head_dim;
    const int elem = dtype == TP_F32 ? 4 : 2;
    if (k != nullptr) {
        s = check_rows(t, n, k, ldk, width, elem);
        TP_CHECK(s == TP_OK, s);
    }
    if (v != nullptr) {
        s = check_rows(t, n, v, ldv, width, elem);
        TP_CHECK(s == TP_OK, s);
    }
    if (n == 0) return TP_OK;
    for (int r = 0; r < t; ++r) {
        d.k[r] = k != nullptr ? k[r] : nullptr;
        d.v[r] = v != nullptr ? v[r] : nullptr;
    }
    d.with_k = k != nullptr;
    d.with_v = v != nullptr;
    d.head_dim = head_dim;
    d.ldk = ldk;
    d.ldv = ldv;
    d.out_f32 = dtype == TP_F32;
    d.seqs.status = tpk::device_status_word();
    return tpk::launch_kv4_load(d, cs(stream));
}

int tp_debug_first_worker(int block, int blocks, int groups, int workers) {
    if (blocks < 1 || blocks > 4096 || block < 0 || block > blocks || groups < 1 || groups > 8 || workers < 0 ||
        workers > blocks * groups)
        return -1;
    return tpk::first_worker_of(block, blocks, groups, workers);
}

uint64_t tp_debug_part_flag(uint64_t word, uint64_t tag, int order) {
    tag |= uint64_t{1} << 63;
    auto plain = [&](uint64_t v) {
        const uint64_t old = word;
        word = v;
        return old;
    };
    // the other worker's steps all come after the first of these
    bool first = true;
    auto then_give_up = [&](uint64_t v) {
        const uint64_t old = plain(v);
        if (first) tpk::give_up_part_flag(tag, plain);
        first = false;
        return old;
    };
    auto then_raise = [&](uint64_t v) {
        const uint64_t old = plain(v);
        if (first) tpk::raise_part_flag(tag, plain);
        first = false;
        return old;
    };
    if (order == 0 || order == 1) tpk::raise_part_flag(tag, plain);
    if (order == 1 || order == 2) tpk::give_up_part_flag(tag, plain);
    if (order == 2) tpk::raise_part_flag(tag, plain);
    if (order == 3) tpk::raise_part_flag(tag, then_give_up);
    if (order == 4) tpk::give_up_part_flag(tag, then_raise);
    return word;
}

static tp_status check_heads(int heads, int kv_heads) {
    TP_CHECK(heads >= 1 && kv_heads >= 1, TP_ERR_INVALID_ARG);
    TP_CHECK(heads % kv_heads == 0, TP_ERR_NOT_DIVISIBLE);
    TP_CHECK(heads / kv_heads <= 128, TP_ERR_UNSUPPORTED);
    return TP_OK;
}

size_t tp_kv4_attention_workspace_size(int t, int64_t n, int64_t nseq, int heads, int kv_heads, int head_dim) {
    if (t < 1 || t > TP_MAX_SHARDS || n < 0 || nseq < 0 || !head_dim_ok(head_dim)) return 0;
    if (check_heads(heads, kv_heads) != TP_OK) return 0;
    return tpk::kv4_attention_workspace(t, n, nseq, heads, kv_heads, head_dim);
}

tp_status tp_kv4_attention(int t, int64_t n, int64_t nseq, int heads, int kv_heads, int head_dim, const void* const* q,
                           int64_t ldq, const void* const* pool, int64_t pages, int page_size, const int32_t* table,
                           int64_t max_blocks, const int32_t* lens, const int32_t* cu_rows, float scale, int64_t window,
                           int64_t sinks, void* workspace, size_t workspace_bytes, void* const* out, int64_t ldo,
                           tp_stream stream) {
    tpk::KvAttentionDesc d;
    tp_status s = check_cache(t, n, nseq, kv_heads, head_dim, const_cast<void* const*>(pool), pages, page_size, table,
                              max_blocks, lens, cu_rows, d.seqs, d.pools);
    TP_CHECK(s == TP_OK, s);
    s = check_heads(heads, kv_heads);
    TP_CHECK(s == TP_OK, s);
    d.group = heads / kv_heads;
    TP_CHECK(n * d.group <= kMaxRows, TP_ERR_UNSUPPORTED);
    TP_CHECK(std::isfinite(scale) && window >= 0 && sinks >= 0, TP_ERR_INVALID_ARG);
    const int64_t width = static_cast<int64_t>(heads) * head_dim;
    s = check_rows(t, n, q, ldq, width, 2);
    TP_CHECK(s == TP_OK, s);
    s = check_rows(t, n, out, ldo, width, 2);
    TP_CHECK(s == TP_OK, s);
    if (n == 0) return TP_OK;
    TP_CHECK(workspace != nullptr &&
                 workspace_bytes >= tpk::kv4_attention_workspace(t, n, nseq, heads, kv_heads, head_dim),
             TP_ERR_WORKSPACE);
    TP_CHECK((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, TP_ERR_ALIGNMENT);
    for (int r = 0; r < t; ++r) {
        d.q[r] = q[r];
        d.out[r] = out[r];
    }
    d.head_dim = head_dim;
    d.ldq = ldq;
    d.ldo = ldo;
    d.scale = scale;
    // no position reaches 2^30, so a window of that many tokens hides nothing
    d.window = window >= kMaxRows ? 0 : static_cast<int>(window);
    d.sinks = static_cast<int>(sinks < kMaxRows ? sinks : kMaxRows);
    d.ws = workspace;
    d.seqs.status = tpk::device_status_word();
    return tpk::launch_kv4_attention(d, cs(stream));
}

size_t tp_kv_pages_workspace_size(int64_t rows, int64_t pages) {
    if (rows < 0 || pages < 1 || rows > INT32_MAX || pages > INT32_MAX) return 0;
    return tpk::kv_pages_workspace(rows, pages);
}

// What fork and compact share.
static tp_status check_pages(int t, int64_t rows_in, int64_t rows_out, int64_t max_blocks, int page_size, int64_t pages,
                             const int32_t* table, const int32_t* lens, void* const* pool, int64_t layers,
                             int64_t page_bytes, int32_t* table_out, int32_t* refs, int32_t* info, void* workspace,
                             size_t workspace_bytes, tpk::KvPagesDesc& d) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(rows_in >= 0 && rows_out >= 0 && max_blocks >= 1 && pages >= 1, TP_ERR_INVALID_ARG);
    TP_CHECK(page_size_ok(page_size), TP_ERR_UNSUPPORTED);
    TP_CHECK(pages <= INT32_MAX && rows_in <= INT32_MAX && rows_out <= INT32_MAX && max_blocks <= kMaxRows / page_size,
             TP_ERR_UNSUPPORTED);
    TP_CHECK(rows_in * max_blocks <= INT32_MAX && rows_out * max_blocks <= INT32_MAX, TP_ERR_UNSUPPORTED);
    TP_CHECK((table != nullptr && lens != nullptr) || rows_in == 0, TP_ERR_INVALID_ARG);
    TP_CHECK(table_out != nullptr || rows_out == 0, TP_ERR_INVALID_ARG);
    TP_CHECK(refs != nullptr && info != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(workspace != nullptr && workspace_bytes >= tpk::kv_pages_workspace(rows_out, pages), TP_ERR_WORKSPACE);
    TP_CHECK(al16(workspace), TP_ERR_ALIGNMENT);
    if (pool != nullptr) {
        TP_CHECK(layers >= 1 && page_bytes >= 16, TP_ERR_INVALID_ARG);
        TP_CHECK(layers <= INT32_MAX / TP_MAX_SHARDS, TP_ERR_UNSUPPORTED);
        TP_CHECK(page_bytes % 16 == 0, TP_ERR_ALIGNMENT);
        for (int r = 0; r < t; ++r) {
            TP_CHECK(pool[r] != nullptr, TP_ERR_INVALID_ARG);
            TP_CHECK(al16(pool[r]), TP_ERR_ALIGNMENT);
            d.pool[r] = static_cast<uint8_t*>(pool[r]);
        }
        d.with_pool = 1;
        d.layers = layers;
        d.page_bytes = page_bytes;
    }
    d.t = t;
    d.rows_in = static_cast<int>(rows_in);
    d.rows_out = static_cast<int>(rows_out);
    d.max_blocks = max_blocks;
    d.page_size = page_size;
    d.pages = static_cast<int>(pages);
    d.table = table;
    d.lens = lens;
    d.table_out = table_out;
    d.refs = refs;
    d.info = info;
    d.ws = workspace;
    return TP_OK;
}

// Whether [a, a + na) and [b, b + nb) overlap, in 32-bit words.
static bool overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(nb) * 4 && b0 < a0 + static_cast<uintptr_t>(na) * 4;
}

tp_status tp_kv_fork(int t, int64_t rows_in, int64_t rows_out, int64_t max_blocks, int page_size, int64_t pages,
                     const int32_t* table, const int32_t* lens, const int32_t* parents, const int32_t* grow,
                     int32_t grow_all, const uint8_t* held, void* const* pool, int64_t layers, int64_t page_bytes,
                     int32_t* table_out, int32_t* lens_out, int32_t* refs, int32_t* info, void* workspace,
                     size_t workspace_bytes, tp_stream stream) {
    tpk::KvPagesDesc d;
    const tp_status s = check_pages(t, rows_in, rows_out, max_blocks, page_size, pages, table, lens, pool, layers,
                                    page_bytes, table_out, refs, info, workspace, workspace_bytes, d);
    TP_CHECK(s == TP_OK, s);
    TP_CHECK((parents != nullptr && lens_out != nullptr) || rows_out == 0, TP_ERR_INVALID_ARG);
    TP_CHECK(!overlap(table, rows_in * max_blocks, table_out, rows_out * max_blocks) &&
                 !overlap(lens, rows_in, lens_out, rows_out),
             TP_ERR_INVALID_ARG);
    d.parents = parents;
    d.grow = grow;
    d.grow_all = grow_all;
    d.held = held;
    d.lens_out = lens_out;
    return tpk::launch_kv_fork(d, cs(stream));
}

tp_status tp_kv_compact(int t, int64_t rows, int64_t max_blocks, int page_size, int64_t pages, const int32_t* table,
                        const int32_t* lens, const uint8_t* held, void* const* pool, int64_t layers, int64_t page_bytes,
                        int32_t* table_out, int32_t* refs, int32_t* info, void* workspace, size_t workspace_bytes,
                        tp_stream stream) {
    tpk::KvPagesDesc d;
    const tp_status s = check_pages(t, rows, rows, max_blocks, page_size, pages, table, lens, pool, layers, page_bytes,
                                    table_out, refs, info, workspace, workspace_bytes, d);
    TP_CHECK(s == TP_OK, s);
    TP_CHECK(!overlap(table, rows * max_blocks, table_out, rows * max_blocks), TP_ERR_INVALID_ARG);
    d.held = held;
    return tpk::launch_kv_compact(d, cs(stream));
}

size_t tp_beam_workspace_size(int64_t items, int beams, int k, int64_t vocab) {
    if (items < 0 || items > INT32_MAX || beams < 1 || beams > TP_MAX_BEAMS || k < 1 || k > TP_MAX_BEAMS || vocab < 1 ||
        vocab > INT32_MAX)
        return 0;
    return tpk::beam_workspace(items, beams, k, vocab);
}

tp_status tp_beam_select(int t, int64_t items, int beams, int k, const int64_t* cols, const void* const* logits,
                         const int64_t* ldl, tp_dtype dtype, const float* scores, const uint8_t* finished, int32_t eos,
                         float* scores_out, int32_t* rows_out, int32_t* tokens_out, void* workspace,
                         size_t workspace_bytes, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(items >= 0 && beams >= 1 && k >= 1, TP_ERR_INVALID_ARG);
    TP_CHECK(beams <= TP_MAX_BEAMS && k <= TP_MAX_BEAMS, TP_ERR_UNSUPPORTED);
    TP_CHECK(dtype == TP_BF16 || dtype == TP_F32, TP_ERR_UNSUPPORTED);
    TP_CHECK(cols != nullptr && logits != nullptr && ldl != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(items * beams <= INT32_MAX, TP_ERR_UNSUPPORTED);
    tpk::BeamDesc d;
    int64_t vocab = 0;
    const uintptr_t elem = dtype == TP_F32 ? 4 : 2;
    for (int r = 0; r < t; ++r) {
        TP_CHECK(cols[r] >= 0 && cols[r] <= INT32_MAX && ldl[r] >= cols[r], TP_ERR_INVALID_ARG);
        TP_CHECK(logits[r] != nullptr || cols[r] == 0 || items == 0, TP_ERR_INVALID_ARG);
        TP_CHECK(reinterpret_cast<uintptr_t>(logits[r]) % elem == 0, TP_ERR_ALIGNMENT);
        vocab += cols[r];
        d.cols[r] = cols[r];
        d.logits[r] = logits[r];
        d.ldl[r] = ldl[r];
    }
    TP_CHECK(vocab >= 1, TP_ERR_INVALID_ARG);
    TP_CHECK(vocab <= INT32_MAX, TP_ERR_UNSUPPORTED);
    TP_CHECK(finished == nullptr || (eos >= 0 && eos < vocab), TP_ERR_INVALID_ARG);
    // candidates of an item are counted in 32 bits
    TP_CHECK(vocab / 4096 * beams * k <= INT32_MAX / 4, TP_ERR_UNSUPPORTED);
    TP_CHECK(items == 0 || (scores != nullptr && scores_out != nullptr && rows_out != nullptr && tokens_out != nullptr),
             TP_ERR_INVALID_ARG);
    if (items == 0) return TP_OK;
    TP_CHECK(workspace != nullptr && workspace_bytes >= tpk::beam_workspace(items, beams, k, vocab), TP_ERR_WORKSPACE);
    TP_CHECK(al16(workspace), TP_ERR_ALIGNMENT);
    d.t = t;
    d.items = static_cast<int>(items);
    d.beams = beams;
    d.k = k;
    d.f32 = dtype == TP_F32;
    d.scores = scores;
    d.finished = finished;
    d.eos = eos;
    d.scores_out = scores_out;
    d.rows_out = rows_out;
    d.tokens_out = tokens_out;
    d.ws = workspace;
    return tpk::launch_beam_select(d, cs(stream));
}

}  // extern "C"

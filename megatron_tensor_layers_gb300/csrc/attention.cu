// Attention over the paged 4-bit cache for few rows per sequence (decode,
// speculation): one pass over the cached codes.  Large calls are bound by the
// instructions that turn codes into operands (243 for a block of 16 tokens and 8
// columns, at 0.46 an SM quarter and cycle) and by what two warps there wait for
// of each other's results: 64 sequences of 4100 to 8192 tokens for 8 kv heads of 128
// take 89 us, 4.7 TB/s, with neither memory (58 %) nor the issue slots full.  Small
// ones by latencies: one sequence of 4097 tokens takes 13.8 us.
//
// Mathematics.  With key j = s_j u_j + b_j (u_j the codes),
//     x_j = c (s_j (q . u_j) + b_j sum(q)),      c = scale log2(e),
// so the matrix product runs on the bare codes and step and base enter per
// (token, column) afterwards.  With value j = s'_j u'_j + b'_j,
//     out = (sum_j (p_j s'_j) u'_j + sum_j p_j b'_j) / sum_j p_j,  p_j = 2^(x_j - m).
//
// Codes to operands.  A code is four bits of an fp16 whose other bits are zero:
// the subnormal u 2^-24, exact, with no bias to subtract.  Of a 32-bit word of
// eight codes, `w & 0x000f000f` is a pair of such numbers, `w & 0x00f000f0` a
// pair scaled by 16, and w >> 8 gives the other two: five instructions for
// eight codes.  The 16 is taken back in q (keys) and in the output's scale
// (values), both exact.  q is scaled by a power of two per row so that its
// largest element is in [2^10, 2^11): a bf16 q is exact in fp16 down to 2^-23 of
// that.  p s' is scaled by 2^(7 - E), E the exponent of the largest step that the
// column has seen, and rounded to fp16 (by 2^-11 of itself, or 2^-32 of 2^E): the
// one rounding of the products.  (One E for all columns took 87.6 us instead of
// 88.9, and a large value cost the rows that do not see it their bits.)
//
// What is subtracted, m, is a column's maximum as of the last time it was
// needed: a stage first takes p under the old m, and only when a sum exceeds 2^7
// (so that p s' could leave fp16), a larger step turns up, or a column has seen
// nothing yet, are the maxima taken across the warp and everything rescaled.
//
// Split.  The unit of work is a stage of 4 cache blocks (64 tokens; 2 with 16
// columns).  All units of all (sequence, row tile, head) items form one line, cut into equal parts, one for
// each worker of 8, 2 or 1 warps (see `ws`); the warps of a worker share each
// item's part of its range and merge through shared memory.  A worker's part of an item that it
// does not hold whole goes to the workspace, and the worker that holds the
// item's end adds the parts in order, after its own range is done: it waits, with
// a limit, for the flags of the parts before its own, which are raised before
// their workers wait for anything.  A second kernel for this took 16.2 us where
// this takes 14.7 (one row, 4097 tokens, 8 heads).
// A flag is raised by writing the call's number, which nothing else in the
// workspace holds, and taken down by whoever waited for it, so that the workspace
// needs no preparation and a graph that repeats a call finds it as the call did.  Where the wait ran out, whichever of
// the two comes second takes it down.
// The cut depends on lengths the host does not know, so every thread block finds
// its own.
//
// Each warp feeds itself: a ring of 2 stages of 4 blocks (2 with 16 columns),
// filled by bulk copies (a block is one contiguous record) and read as mma.sync
// fragments without conflicts: the transposed products K q^T and V^T p^T have
// the tokens and the head dimension as their 16 rows and only 8 columns, so 8
// query heads of a group fill them.  tcgen05 would want 128 rows of them.  With
// two warps on a scheduler it is the independent work within a warp that hides
// latencies: the blocks of a full, fully visible stage run as one straight line
// (two at a time takes 5 % longer, one at a time 8 %).  Three warps there, of 168
// registers, take 100 us and more.  An item's ends, whose instructions are rarely
// in the cache, go block by block.
#include <algorithm>
#include <type_traits>

#include "attention_args.cuh"

namespace tpk {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 32;           // blocks whose addresses a warp holds, one in each lane
constexpr int kStages = 2;
constexpr int kPShift = 8;           // p s' is held times 2^(kPShift - 1 - E)
constexpr int kUnder = 14;           // what p v adds up to is held times 2^-kUnder, so that it passes fp32 only with the values
constexpr float kMost = 128.0f;      // sum of a lane's 2^(x - m) up to which the old maximum will do
constexpr int kMany = 72;            // columns for each pair of blocks from which the many-rows kernel pays (many_pays)
constexpr float kNegInf = -INFINITY;

// An item whose end a worker holds, but not its beginning.
struct Join {
    int active;
    int from, from_slot;             // the worker that holds the beginning, and which of its two parts that is
    int first_row, rows, tile, head;
};

// A part of an item: for each (16-row tile of dimensions, column tile) 32 lanes' four accumulators, then
// 32 lanes' maxima and sums of two columns.
__host__ __device__ constexpr int slot_vectors(int nt, int hd) { return nt * (hd / 16 + 1) * 32; }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A flag of 64 bits, raised with a release and awaited, with the limit of every wait here, with an acquire.
__device__ __forceinline__ uint64_t exchange_gpu64(uint64_t* p, uint64_t v) {
    uint64_t old;
    asm volatile("atom.release.gpu.global.exch.b64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
    return old;
}
__device__ __forceinline__ bool flag64_wait(const uint64_t* flag, uint64_t value, volatile int* abort, int* status) {
    const uint64_t t0 = global_ns();
    while (true) {
        uint64_t v;
        asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(flag) : "memory");
        if (v == value) return true;
        if (*abort) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            raise_status(status, TP_ERR_TIMEOUT);
            return false;
        }
        __nanosleep(32);
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// What one sequence asks for: its rows, and the blocks that any of them sees:
// [0, front) for the sinks, then [start, start + units - front).
struct Need {
    int first_row, rows, len;
    int front, start, blocks;
    int units, tiles;                // units >= 1 per item (an item that sees nothing writes zeros)
    // the blocks of unit u, `most` at most: how many, and the first of them in the order of what is seen
    __device__ __forceinline__ int unit(int u, int most, int& first) const {
        const int sunk = (front + most - 1) / most;
        first = u < sunk ? u * most : front + (u - sunk) * most;
        return max(0, min(most, (u < sunk ? front : blocks) - first));
    }
};

__device__ __forceinline__ Need seq_need(const AttnArgs& a, int s, int cols_per_tile, int most, int many) {
    Need n;
    const SeqRows r = seq_rows(a.seqs, s);
    n.first_row = r.first;
    n.rows = r.count;
    n.len = max(a.seqs.lens[s], 0);
    const int64_t cols = static_cast<int64_t>(r.count) * a.group;
    n.tiles = cols >= many ? 0 : static_cast<int>((cols + cols_per_tile - 1) / cols_per_tile);
    Spans v{0, 0, 0};
    if (n.tiles > 0) v = visible_spans(a, static_cast<int64_t>(n.len) - r.count, static_cast<int64_t>(n.len) - 1, kKvBlock);
    n.front = v.front;
    n.start = v.start;
    n.blocks = v.count;
    n.units = max((n.front + most - 1) / most + (n.blocks - n.front + most - 1) / most, 1);
    return n;
}

// The line of `total` units in `workers` <= total equal parts; the first `more` hold one unit more.
struct Parts {
    int64_t each;
    int more;
    __device__ __forceinline__ Parts(int64_t total, int workers) {
        each = quotient(total, workers);
        more = static_cast<int>(total - each * workers);
    }
    __device__ __forceinline__ int64_t begin(int b) const { return each * b + min(b, more); }
    // the part that holds unit u
    __device__ __forceinline__ int of(int64_t u) const {
        const int64_t front = (each + 1) * more;
        return static_cast<int>(u < front ? quotient(u, each + 1) : more + quotient(u - front, each));
    }
};

// A position on the line of units, walked item by item.
struct Cursor {
    int left;                        // units of the worker's range from here on
    int s, tile, head, off;          // current item and the unit in it
    Need n;
    __device__ __forceinline__ int count() const { return min(n.units - off, left); }
    __device__ __forceinline__ void next(const AttnArgs& a, int cols_per_tile, int most, int many, int heads) {
        const int c = count();
        left -= c;
        off += c;
        if (left <= 0) return;
        off = 0;                     // more of the range left: the item is done
        if (++head < heads) return;
        head = 0;
        if (++tile < n.tiles) return;
        tile = 0;
        do {
            ++s;
            if (s >= a.seqs.nseq) {
                left = 0;
                return;
            }
            n = seq_need(a, s, cols_per_tile, most, many);
        } while (n.tiles == 0);
    }
};

__host__ __device__ constexpr size_t flag_bytes(int blocks) { return (static_cast<size_t>(blocks) * kWarps * 2 * 8 + 255) / 256 * 256; }

template <int HD, int NT>
struct Cfg {
    static constexpr int COLS = 8 * NT;
    static constexpr int WARPS = kWarps;
    static constexpr int MT = HD / 16;                       // 16-row tiles of the output's dimensions
    static constexpr int BLOCKS = 4 / NT;                    // of a stage
    static constexpr int STAGE = BLOCKS * KvBlock<HD>::BYTES;
    static constexpr int RING = WARPS * kStages * STAGE;
    static constexpr int PART = slot_vectors(NT, HD);        // of a warp, in float4
    static constexpr int SMEM = RING + WARPS * PART * 16;
};

// Where a lane's dimensions of column cc of a sequence go, nullptr past the last column.
template <int HD>
__device__ __forceinline__ uint16_t* out_of(const AttnArgs& a, int head, int first_row, int rows, int cc, int lane) {
    const int r = rows == 1 ? 0 : cc / a.group, h = cc - r * a.group;
    if (r >= rows || h >= a.group) return nullptr;
    const int rank = head / a.pools.kv_heads, kvh = head - rank * a.pools.kv_heads;
    return a.out[rank] + (first_row + r) * a.ldo + (kvh * a.group + h) * HD + (lane >> 2) * (HD / 8);
}

// Vectors v .. v + NV - 1 of an item's result (see slot_vectors; of one column tile) to the output.
template <int HD, int NV>
__device__ __forceinline__ void store_vectors(const AttnArgs& a, int head, int first_row, int rows, int first_col, int lane,
                                              int v, const float4 (&o)[NV], const float2& total) {
    constexpr int MT = HD / 16;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint16_t* p = out_of<HD>(a, head, first_row, rows, first_col + v / MT * 8 + 2 * (lane & 3) + e, lane);
        if (p == nullptr) continue;
        const float sum = e ? total.y : total.x, inv = sum == 0.0f ? 0.0f : static_cast<float>(1 << kUnder) / sum;
        uint32_t w[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) w[i] = pack_bf16x2((e ? o[i].y : o[i].x) * inv, (e ? o[i].w : o[i].z) * inv);
        if constexpr (NV == 4)
            *reinterpret_cast<uint4*>(p + 2 * (v % MT)) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint32_t*>(p + 2 * (v % MT)) = w[0];
    }
}

// The sum, in order, of `count` parts at part(p): warp wi of ws gives NV vectors of the result at a
// time (see slot_vectors) to put(first vector, vectors, maxima, sums).
template <int HD, int NT, int NV, typename Part, typename Put>
__device__ __forceinline__ void join_parts(int wi, int ws, int lane, int count, Part part, Put put) {
    constexpr int MT = HD / 16;
    for (int v = wi * NV; v < NT * MT; v += ws * NV) {
        const int nt = v / MT;
        float2 top = make_float2(kNegInf, kNegInf), total = make_float2(0.0f, 0.0f);
        float4 o[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8 / NV
        for (int p = 0; p < count; ++p) {
            const float4* from = part(p) + lane;
            const float4 st = from[(NT * MT + nt) * 32];
            const float2 m = make_float2(fmaxf(top.x, st.x), fmaxf(top.y, st.y));
            const float2 b = make_float2(m.x == kNegInf ? 0.0f : m.x, m.y == kNegInf ? 0.0f : m.y);
            const float2 fa = make_float2(ex2(top.x - b.x), ex2(top.y - b.y)), fb = make_float2(ex2(st.x - b.x), ex2(st.y - b.y));
            top = m;
            total = make_float2(total.x * fa.x + st.z * fb.x, total.y * fa.y + st.w * fb.y);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 x = from[(v + i) * 32];
                o[i] = make_float4(o[i].x * fa.x + x.x * fb.x, o[i].y * fa.y + x.y * fb.y, o[i].z * fa.x + x.z * fb.x,
                                   o[i].w * fa.y + x.w * fb.y);
            }
        }
        put(v, o, top, total);
    }
}

template <int HD, int NT>
__global__ void __launch_bounds__(Cfg<HD, NT>::WARPS * 32, 1) kv4_attention_kernel(const __grid_constant__ AttnArgs a) {
    using B = KvBlock<HD>;
    using C = Cfg<HD, NT>;
    constexpr int MT = C::MT, COLS = C::COLS, WARPS = C::WARPS, THREADS = WARPS * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[WARPS * kStages];
    __shared__ int stage_mask[WARPS * kStages];
    __shared__ int64_t scan[WARPS], scan_items[WARPS];
    __shared__ Cursor s_cursor[WARPS];
    __shared__ Join s_join[WARPS];
    __shared__ int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int heads = a.pools.t * a.pools.kv_heads;

    if (tid == 0) s_abort = 0;
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars[warp * kStages + i]), 1);
    fence_barrier_init();
    pdl_wait();
    pdl_trigger();

    if (blockIdx.x == 0 && tid == 0 && a.seqs.cu_rows != nullptr &&
        (a.seqs.cu_rows[0] != 0 || a.seqs.cu_rows[a.seqs.nseq] != a.seqs.n))
        raise_status(a.seqs.status, TP_ERR_INVALID_ARG);     // rows that no sequence holds

    // ---- which sequences are this kernel's: those with fewer than `many` columns
    int many = INT32_MAX;
    if (a.many != INT32_MAX) {
        int64_t cols = 0, tiles = 0;
        for (int s = tid; s < a.seqs.nseq; s += THREADS) {
            const int64_t c = static_cast<int64_t>(seq_rows(a.seqs, s).count) * a.group;
            const int n = many_tiles(a, c);
            if (n > 0) cols += c, tiles += n;
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            cols += __shfl_xor_sync(0xffffffffu, cols, m);
            tiles += __shfl_xor_sync(0xffffffffu, tiles, m);
        }
        if (lane == 0) scan[warp] = cols, scan_items[warp] = tiles;
        __syncthreads();
        cols = tiles = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) cols += scan[i], tiles += scan_items[i];
        if (many_pays(a, cols, tiles)) many = a.many;
        __syncthreads();
    }

    // ---- the cut: total units, items, then where each of this block's workers begins
    int64_t mine = 0, items = 0;
    const int per = (a.seqs.nseq + THREADS - 1) / THREADS;
    Need need = {};                  // of this thread's last sequence: with one each, it is not asked for twice
    for (int s = tid * per; s < min(a.seqs.nseq, (tid + 1) * per); ++s) {
        need = seq_need(a, s, COLS, C::BLOCKS, many);
        mine += static_cast<int64_t>(need.units) * need.tiles * heads;
        items += static_cast<int64_t>(need.tiles) * heads;
    }
    int64_t before = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, before, m);
        if (lane >= m) before += v;
        items += __shfl_xor_sync(0xffffffffu, items, m);
    }
    if (lane == 31) scan[warp] = before, scan_items[warp] = items;
    __syncthreads();
    int64_t total = 0, base = 0, all_items = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < warp) base += scan[i];
        total += scan[i];
        all_items += scan_items[i];
    }
    before += base - mine;           // units before this thread's sequences
    if (total == 0) return;
    // Warps of a worker.  Eight share an item's latency, but meet at its end and pay for each item's
    // beginning eight times; alone a warp does neither, but a long item is then the sum of many parts.
    // Of 4097 tokens, head dimension 128, with 8, 2 and 1 warps: 8 items 16, 20, 43 us; 64: 22, 21, 38 us;
    // 256: 49, 42, 48 us; 1024: 148, 119, 118 us; 2048: 282, 224, 219 us (4 are between 8 and 2, or behind
    // both).  Each warp is to have a unit, too: 128 items of 128 tokens take 27, 15, 17 us.
    const int64_t sms = gridDim.x;
    const int ws = all_items * 4 <= sms && total >= WARPS * all_items ? WARPS
                   : all_items <= sms * WARPS && total >= 2 * all_items ? 2 : 1;
    const int groups = WARPS / ws;
    const int workers = static_cast<int>(min(sms * groups, quotient(total + ws - 1, ws)));
    const Parts parts(total, workers);
    const int worker0 = first_worker_of(blockIdx.x, gridDim.x, groups, workers);
    const int worker1 = first_worker_of(blockIdx.x + 1, gridDim.x, groups, workers);
    for (int i = 0; i < groups; ++i) {
        const int w = worker0 + i;
        if (w >= worker1) {
            if (tid == 0) s_cursor[i].left = 0;
            continue;
        }
        const int64_t begin = parts.begin(w);
        if (begin >= before && begin < before + mine) {      // one thread's sequences hold the beginning
            int64_t u = begin - before;
            int s = tid * per;
            if (per > 1)
                while (true) {
                    need = seq_need(a, s, COLS, C::BLOCKS, many);
                    const int64_t w_s = static_cast<int64_t>(need.units) * need.tiles * heads;
                    if (u < w_s) break;
                    u -= w_s;
                    ++s;
                }
            Cursor c;
            c.left = static_cast<int>(parts.begin(w + 1) - begin);
            c.s = s;
            c.n = need;
            const int item = static_cast<int>(quotient(u, need.units));
            c.off = static_cast<int>(u - static_cast<int64_t>(item) * need.units);
            c.tile = item / heads;
            c.head = item - c.tile * heads;
            s_cursor[i] = c;
            Join jn = {};
            if (c.off > 0 && c.off + c.left >= need.units) {
                const int64_t first = begin - c.off;
                jn.active = 1;
                jn.from = parts.of(first);
                jn.from_slot = parts.begin(jn.from) == first ? 0 : 1;
                jn.first_row = need.first_row;
                jn.rows = need.rows;
                jn.tile = c.tile;
                jn.head = c.head;
            }
            s_join[i] = jn;
        }
    }
    __syncthreads();

    const int grp = warp / ws, wi = warp % ws;
    const int worker = worker0 + grp;
    // two parts of each worker: the item its range begins in, and the one it ends in
    uint64_t* flags = reinterpret_cast<uint64_t*>(a.ws);
    float4* slots = reinterpret_cast<float4*>(a.ws + flag_bytes(gridDim.x));
    auto together = [&]() {          // the worker's warps
        if (ws > 1)
            asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(ws * 32) : "memory");
        else
            __syncwarp();
    };

    Cursor cur = s_cursor[grp];      // the item being computed
    if (cur.left <= 0) return;       // the whole worker
    Cursor ahead = cur;              // the item being loaded
    bool first_segment = true;

    auto row_of = [&](int rows, int col) { return rows == 1 ? 0 : col / a.group; };

    // ---- q of an item: a lane holds a quarter of the dimensions of one column of each column tile
    constexpr int D = HD / 4;
    uint32_t raw[NT][D / 2];
    auto fetch_q = [&](const Cursor& c) {
        const int rank = c.head / a.pools.kv_heads, kvh = c.head - rank * a.pools.kv_heads;
        const int cols = c.n.rows * a.group - c.tile * COLS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int ci = nt * 8 + g;
            const bool have = ci < cols;
            const int cc = c.tile * COLS + ci;
            const int r = have ? row_of(c.n.rows, cc) : 0;
            const int h = cc - r * a.group;
            const uint4* src = reinterpret_cast<const uint4*>(a.q[rank] + (c.n.first_row + r) * a.ldq +
                                                              (kvh * a.group + h) * HD + t4 * D);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint4 v = have ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                raw[nt][4 * i] = v.x, raw[nt][4 * i + 1] = v.y, raw[nt][4 * i + 2] = v.z, raw[nt][4 * i + 3] = v.w;
            }
        }
    };

    // ---- loading
    const uint32_t ring = smem_u32(smem) + warp * kStages * C::STAGE;
    const uint32_t my_bars = smem_u32(&bars[warp * kStages]);
    // this warp's share of a segment of n units
    auto share = [&](int n, int w) { return static_cast<int>(static_cast<uint32_t>(n) * static_cast<uint64_t>(w) / ws); };
    int load_u = 0, load_u0 = 0, load_end = 0;
    int64_t batch_off = -1;          // lane l holds the address of block l of the batch
    uint32_t batch_there = 0;
    int next_page = -2;              // and the page of block l of the next batch, -2: none
    constexpr int kUnits = kBatch / C::BLOCKS;
    auto block_at = [](const Need& n, int i) { return i < n.front ? i : n.start + i - n.front; };
    // the block of this lane in the batch that begins with unit u, -1: none
    auto lane_block = [&](int u) {
        u += lane / C::BLOCKS;
        int first;
        if (u >= load_end || lane % C::BLOCKS >= ahead.n.unit(u, C::BLOCKS, first)) return -1;
        return block_at(ahead.n, first + lane % C::BLOCKS);
    };
    auto fetch_page = [&](int u) {
        const int block = lane_block(u);
        return block < 0 ? -2
                         : kv_page_at(a.seqs.table + ahead.s * a.seqs.max_blocks, a.seqs.max_blocks, a.pools.page_shift, block);
    };
    auto open_segment = [&]() {
        load_u = load_u0 = ahead.off + share(ahead.count(), wi);
        load_end = ahead.off + share(ahead.count(), wi + 1);
        next_page = fetch_page(load_u);
    };
    int issued = 0;
    auto load_stage = [&]() {
        while (load_u >= load_end) {
            ahead.next(a, COLS, C::BLOCKS, many, heads);
            if (ahead.left <= 0) return;
            open_segment();
        }
        const int rank = ahead.head / a.pools.kv_heads;
        const int at = (load_u - load_u0) & (kUnits - 1);
        if (at == 0) {
            const int page = next_page;
            batch_off = kv_page_offset(page, a.pools.pages, a.pools.page_shift, a.pools.kv_heads,
                                       ahead.head - rank * a.pools.kv_heads, lane_block(load_u), B::BYTES);
            if (batch_off < 0 && page != -2) raise_status(a.seqs.status, TP_ERR_INVALID_ARG);
            batch_there = __ballot_sync(0xffffffffu, batch_off >= 0);
            next_page = fetch_page(load_u + kUnits);
        }
        const uint32_t mask = (batch_there >> (at * C::BLOCKS)) & ((1u << C::BLOCKS) - 1u);
        const int st = issued % kStages;
        const uint32_t bar = my_bars + st * 8;
        if (lane == 0) {
            stage_mask[warp * kStages + st] = static_cast<int>(mask);
            mbar_arrive_expect_tx(bar, __popc(mask) * B::BYTES);
        }
        __syncwarp();
        const uint32_t i = static_cast<uint32_t>(lane - at * C::BLOCKS); // this lane's block of the stage
        if (i < static_cast<uint32_t>(C::BLOCKS) && batch_off >= 0)
            bulk_load(ring + st * C::STAGE + i * B::BYTES, a.pools.pool[rank] + batch_off, B::BYTES, bar);
        ++issued;
        ++load_u;
    };
    open_segment();
    fetch_q(cur);
    for (int i = 0; i < kStages; ++i) load_stage();

    // ---- computing
    const int tok = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;   // token of row g of a key tile; row g + 8: tok + 8
    bool dead = false;
    int used = 0;
    while (true) {
        const int seg_off = cur.off, seg_n = cur.count();
        const int u0 = seg_off + share(seg_n, wi), u1 = seg_off + share(seg_n, wi + 1);
        const int cols = cur.n.rows * a.group - cur.tile * COLS;         // columns left from this tile on
        const int pos0 = cur.n.len - cur.n.rows;                        // position of the sequence's first row

        // q as B fragments; per-column scale of the products, and sum(q), both times scale log2(e)
        uint32_t qf[NT][HD / 16][2];
        float cmul[NT][2], cadd[NT][2];
        int cpos[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t top = 0;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 2; ++i) {
                top = __vmaxu2(top, raw[nt][i] & 0x7fff7fffu);
                sum += __uint_as_float(raw[nt][i] << 16) + __uint_as_float(raw[nt][i] & 0xffff0000u);
            }
#pragma unroll
            for (int m = 1; m < 4; m <<= 1) {
                top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
                sum += __shfl_xor_sync(0xffffffffu, sum, m);
            }
            top = max(top & 0xffffu, top >> 16);
            // 2^k with the row's largest element in [2^10, 2^11); k within the fp32 exponents
            const int k = min(10 - (static_cast<int>(top >> 7) - 127), 126);
            const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
            const float up16 = up * 0.0625f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {                            // a word of eight codes
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = __uint_as_float(raw[nt][4 * j + i] << 16);
                    x[2 * i + 1] = __uint_as_float(raw[nt][4 * j + i] & 0xffff0000u);
                }
                qf[nt][2 * j][0] = pack_f16x2(x[0] * up, x[4] * up);
                qf[nt][2 * j][1] = pack_f16x2(x[1] * up16, x[5] * up16);
                qf[nt][2 * j + 1][0] = pack_f16x2(x[2] * up, x[6] * up);
                qf[nt][2 * j + 1][1] = pack_f16x2(x[3] * up16, x[7] * up16);
            }
            // 2^(24 - k) can pass fp32 where the factor does not; k from -118 to 126
            const float mul = a.scale_log2 * 0x1p24f * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            const float add = a.scale_log2 * sum;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * t4 + e) * 4;
                cmul[nt][e] = __shfl_sync(0xffffffffu, mul, from);
                cadd[nt][e] = __shfl_sync(0xffffffffu, add, from);
                const int ce = nt * 8 + 2 * t4 + e;
                cpos[nt][e] = ce < cols ? pos0 + row_of(cur.n.rows, cur.tile * COLS + ce) : -1;
            }
        }
        const int row_lo = pos0 + row_of(cur.n.rows, cur.tile * COLS);
        const int row_hi = pos0 + row_of(cur.n.rows, cur.tile * COLS + min(cols, COLS) - 1);

        float acc[NT][MT][4];
        float mx[NT][2], sum[NT][2], corr[NT][2];
        // exponent field of the largest value step that a column has seen, at least 16 so that 2^(kPShift - E) stays
        // finite; a range that fp32 holds has a step of at most 2^124.1, field 251
        int vexp[NT][2];
        bool fresh = true;               // some column has seen nothing
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[nt][e] = kNegInf, sum[nt][e] = 0.0f, corr[nt][e] = 0.0f, vexp[nt][e] = 16;
        }

        for (int u = u0; u < u1; ++u) {
            const int st = used % kStages;
            if (!dead) dead = !mbar_wait_warp(my_bars + st * 8, (used / kStages) & 1, &s_abort, a.seqs.status);
            const uint32_t mask = dead ? 0u : static_cast<uint32_t>(stage_mask[warp * kStages + st]);
            const uint32_t buf = ring + st * C::STAGE;
            int first;
            cur.n.unit(u, C::BLOCKS, first);
            const int j0 = block_at(cur.n, first) * kKvBlock;
            const int j1 = j0 + C::BLOCKS * kKvBlock - 1;

            // `blocks` of the stage's blocks, from block `from` on; `edge`: some column does not see some token.
            auto stage = [&](auto edge, auto blocks, int from) {
                constexpr bool EDGE = decltype(edge)::value;
                constexpr int BLOCKS = decltype(blocks)::value;
                float x[BLOCKS][NT][4];
                uint32_t vp[BLOCKS][2];
                uint32_t vtop[NT][2] = {};                               // largest step that the columns see: not negative
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
                    const uint32_t rec = buf + (from + i) * B::BYTES;
                    uint32_t wa[HD / 32], wb[HD / 32];
                    const uint32_t ka = rec + B::KEYS + tok * B::ROW + t4 * (B::ROW / 4);
                    if constexpr (HD == 128) {
                        const uint4 p = lds128(ka), q = lds128(ka + 8 * B::ROW);
                        wa[0] = p.x, wa[1] = p.y, wa[2] = p.z, wa[3] = p.w;
                        wb[0] = q.x, wb[1] = q.y, wb[2] = q.z, wb[3] = q.w;
                    } else {
                        const uint2 p = lds64(ka), q = lds64(ka + 8 * B::ROW);
                        wa[0] = p.x, wa[1] = p.y;
                        wb[0] = q.x, wb[1] = q.y;
                    }
                    const uint32_t kp0 = lds32(rec + B::KPAIR + tok * 4), kp1 = lds32(rec + B::KPAIR + (tok + 8) * 4);
                    vp[i][0] = lds32(rec + B::VPAIR + tok * 4);
                    vp[i][1] = lds32(rec + B::VPAIR + (tok + 8) * 4);
                    // two chains of products: the second half of the words has its own accumulators
                    float y[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[i][nt][e] = y[nt][e] = 0.0f;
#pragma unroll
                    for (int j = 0; j < HD / 32; ++j) {
                        const uint32_t ha = wa[j] >> 8, hb = wb[j] >> 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(x[i][nt], wa[j] & 0x000f000fu, wb[j] & 0x000f000fu, wa[j] & 0x00f000f0u,
                                    wb[j] & 0x00f000f0u, qf[nt][2 * j][0], qf[nt][2 * j][1]);
                            mma_f16(y[nt], ha & 0x000f000fu, hb & 0x000f000fu, ha & 0x00f000f0u, hb & 0x00f000f0u,
                                    qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
                        }
                    }
                    const float s0 = __uint_as_float(kp0 << 16), b0 = __uint_as_float(kp0 & 0xffff0000u);
                    const float s1 = __uint_as_float(kp1 << 16), b1 = __uint_as_float(kp1 & 0xffff0000u);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[i][nt][e] = fmaf(x[i][nt][e] + y[nt][e], cmul[nt][e] * s0, cadd[nt][e] * b0);
                            x[i][nt][2 + e] = fmaf(x[i][nt][2 + e] + y[nt][2 + e], cmul[nt][e] * s1, cadd[nt][e] * b1);
                        }
                    if constexpr (EDGE) {
                        const int ja = j0 + (from + i) * kKvBlock + tok, jb = ja + 8;
                        // a pair that no column sees may hold anything
                        if (ja > row_hi || !(a.window == 0 || ja > row_lo - a.window || ja < a.sinks)) vp[i][0] = 0;
                        if (jb > row_hi || !(a.window == 0 || jb > row_lo - a.window || jb < a.sinks)) vp[i][1] = 0;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int p = cpos[nt][e];
                                const bool sa = ja <= p && (a.window == 0 || ja > p - a.window || ja < a.sinks);
                                const bool sb = jb <= p && (a.window == 0 || jb > p - a.window || jb < a.sinks);
                                if (!sa) x[i][nt][e] = kNegInf;
                                if (!sb) x[i][nt][2 + e] = kNegInf;
                                vtop[nt][e] = max(sa ? vp[i][0] & 0xffffu : 0u, sb ? vp[i][1] & 0xffffu : 0u);
                            }
                    } else {
                        vtop[0][0] = max(vtop[0][0], max(vp[i][0] & 0xffffu, vp[i][1] & 0xffffu));
                    }
                }
                static_assert(!EDGE || BLOCKS == 1, "vtop is that of one block");
                if constexpr (!EDGE) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) vtop[nt][e] = vtop[0][0];
                }

                // p s' as B fragments, and what the stage adds to the sums
                uint32_t pf[BLOCKS][NT][2];
                float psum[NT][2], pcorr[NT][2];
                auto weigh = [&]() {
                    constexpr float under = 1.0f / (1 << kUnder);
                    float m[NT][2], vscale[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            psum[nt][e] = pcorr[nt][e] = 0.0f;
                            m[nt][e] = mx[nt][e] == kNegInf ? 0.0f : mx[nt][e];
                            vscale[nt][e] = __uint_as_float(static_cast<uint32_t>(253 - vexp[nt][e]) << 23) * (1 << kPShift);
                        }
#pragma unroll
                    for (int i = 0; i < BLOCKS; ++i) {
                        const float s0 = __uint_as_float(vp[i][0] << 16), b0 = __uint_as_float(vp[i][0] & 0xffff0000u) * under;
                        const float s1 = __uint_as_float(vp[i][1] << 16), b1 = __uint_as_float(vp[i][1] & 0xffff0000u) * under;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float ps[4];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float xa = x[i][nt][e], xb = x[i][nt][2 + e];
                                const float pa = ex2(xa - m[nt][e]), pb = ex2(xb - m[nt][e]);
                                psum[nt][e] += pa + pb;
                                if constexpr (EDGE) {
                                    // a token that this column does not see may stand for NaN or infinities
                                    ps[e] = xa == kNegInf ? 0.0f : pa * (s0 * vscale[nt][e]);
                                    ps[2 + e] = xb == kNegInf ? 0.0f : pb * (s1 * vscale[nt][e]);
                                    pcorr[nt][e] += (xa == kNegInf ? 0.0f : pa * b0) + (xb == kNegInf ? 0.0f : pb * b1);
                                } else {
                                    ps[e] = pa * (s0 * vscale[nt][e]);
                                    ps[2 + e] = pb * (s1 * vscale[nt][e]);
                                    pcorr[nt][e] = fmaf(pa, b0, fmaf(pb, b1, pcorr[nt][e]));
                                }
                            }
                            pf[i][nt][0] = pack_f16x2(ps[0], ps[1]);
                            pf[i][nt][1] = pack_f16x2(ps[2], ps[3]);
                        }
                    }
                };
                bool again = fresh;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) again |= static_cast<int>(vtop[nt][e] >> 7) > vexp[nt][e];
                if (!__any_sync(0xffffffffu, again)) {                   // the old maximum may do
                    weigh();
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) again |= !(psum[nt][e] <= kMost);
                }
                if (__any_sync(0xffffffffu, again)) {
                    float cmax[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            cmax[nt][e] = kNegInf;
#pragma unroll
                            for (int i = 0; i < BLOCKS; ++i)
                                cmax[nt][e] = fmaxf(cmax[nt][e], fmaxf(x[i][nt][e], x[i][nt][2 + e]));
                        }
#pragma unroll
                    for (int m = 4; m < 32; m <<= 1) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                vtop[nt][e] = max(vtop[nt][e], __shfl_xor_sync(0xffffffffu, vtop[nt][e], m));
                                cmax[nt][e] = fmaxf(cmax[nt][e], __shfl_xor_sync(0xffffffffu, cmax[nt][e], m));
                            }
                    }
                    bool unseen = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int e_new = max(vexp[nt][e], min(static_cast<int>(vtop[nt][e] >> 7), 251));
                            const float vdown = __uint_as_float(static_cast<uint32_t>(max(127 - (e_new - vexp[nt][e]), 0)) << 23);
                            vexp[nt][e] = e_new;
                            const float m = fmaxf(mx[nt][e], cmax[nt][e]);
                            const float alpha = ex2(mx[nt][e] - (m == kNegInf ? 0.0f : m));
                            mx[nt][e] = m;
                            unseen |= m == kNegInf && nt * 8 + 2 * t4 + e < cols;
                            sum[nt][e] *= alpha;
                            corr[nt][e] *= alpha;
#pragma unroll
                            for (int i = 0; i < MT; ++i)
                                acc[nt][i][e] *= alpha * vdown, acc[nt][i][2 + e] *= alpha * vdown;
                        }
                    fresh = __any_sync(0xffffffffu, unseen);
                    weigh();
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) sum[nt][e] += psum[nt][e], corr[nt][e] += pcorr[nt][e];
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) pf[i][nt][e] = transpose8x8(pf[i][nt][e]);
                    // values: tokens t4, 4 + (t4 ^ 1) and the same + 8 are this lane's columns of k
                    const uint32_t va = buf + (from + i) * B::BYTES + B::VALS + g * (B::ROW / 8);
                    constexpr int W = HD / 64;
                    uint32_t y[4][W];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int tk = ((p & 1) ? 4 + (t4 ^ 1) : t4) + (p >> 1) * 8;
                        if constexpr (W == 2) {
                            const uint2 v = lds64(va + tk * B::ROW);
                            y[p][0] = v.x, y[p][1] = v.y;
                        } else {
                            y[p][0] = lds32(va + tk * B::ROW);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t p01 = __byte_perm(y[0][j], y[1][j], h ? 0x7632 : 0x5410);
                            uint32_t p23 = __byte_perm(y[2][j], y[3][j], h ? 0x7632 : 0x5410);
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_f16(acc[nt][j * 4 + h * 2 + b], p01 & 0x000f000fu, p01 & 0x00f000f0u,
                                            p23 & 0x000f000fu, p23 & 0x00f000f0u, pf[i][nt][0], pf[i][nt][1]);
                                p01 >>= 8, p23 >>= 8;
                            }
                        }
                }
            };
            const bool whole = mask == (1u << C::BLOCKS) - 1u && j1 <= row_lo &&
                               (a.window == 0 || j0 > row_hi - a.window || j1 < a.sinks);
            if (whole)
                stage(std::false_type{}, std::integral_constant<int, C::BLOCKS>{}, 0);
            else
                // an item's ends: block by block, in a quarter of the instructions, which are rarely in the cache
#pragma unroll 1
                for (uint32_t left = mask; left != 0; left &= left - 1)
                    stage(std::true_type{}, std::integral_constant<int, 1>{}, __ffs(left) - 1);
            __syncwarp();                                                // every lane is done with the stage
            ++used;
            if (!dead) load_stage();
        }

        // ---- the warp's result: O, maximum and sum of each column, every lane with its own dimensions
        static_assert(24 - kPShift + 251 + 1 - kUnder <= 254 && 24 - kPShift + 16 + 1 - kUnder >= 1, "a normal power of two");
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float down = __uint_as_float(static_cast<uint32_t>(24 - kPShift + vexp[nt][e] + 1 - kUnder) << 23);
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) {
                    sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], m);
                    corr[nt][e] += __shfl_xor_sync(0xffffffffu, corr[nt][e], m);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    acc[nt][i][e] = fmaf(acc[nt][i][e], down, corr[nt][e]);
                    acc[nt][i][2 + e] = fmaf(acc[nt][i][2 + e], down * 0.0625f, corr[nt][e]);
                }
            }
        const bool complete = seg_off == 0 && seg_n == cur.n.units;
        const int head = cur.head, first_row = cur.n.first_row, rows = cur.n.rows, tile = cur.tile;
        const int slot_no = worker * 2 + (first_segment ? 0 : 1);
        float4* slot = slots + static_cast<size_t>(slot_no) * C::PART;
        const bool awaited = !complete && seg_off + seg_n < cur.n.units; // by the worker that holds the end
        first_segment = false;
        cur.next(a, COLS, C::BLOCKS, many, heads);
        const bool more = cur.left > 0;
        if (more) fetch_q(cur);
        auto store = [&](int v, const auto& o, const float2& total) {    // vectors of a complete item
            store_vectors<HD>(a, head, first_row, rows, tile * COLS, lane, v, o, total);
        };
        if (ws == 1 && complete) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < MT; i += 4) {
                    const float4 o[4] = {make_float4(acc[nt][i][0], acc[nt][i][1], acc[nt][i][2], acc[nt][i][3]),
                                         make_float4(acc[nt][i + 1][0], acc[nt][i + 1][1], acc[nt][i + 1][2], acc[nt][i + 1][3]),
                                         make_float4(acc[nt][i + 2][0], acc[nt][i + 2][1], acc[nt][i + 2][2], acc[nt][i + 2][3]),
                                         make_float4(acc[nt][i + 3][0], acc[nt][i + 3][1], acc[nt][i + 3][2], acc[nt][i + 3][3])};
                    store(nt * MT + i, o, make_float2(sum[nt][0], sum[nt][1]));
                }
            if (!more) break;
            continue;
        }
        // the worker's warps together: every one leaves its part, then they share the sum of the parts
        float4* left = reinterpret_cast<float4*>(smem + C::RING) + grp * ws * C::PART;
        float4* mine_part = ws > 1 ? left + wi * C::PART : slot;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
                mine_part[(nt * MT + i) * 32 + lane] =
                    make_float4(acc[nt][i][0], acc[nt][i][1], acc[nt][i][2], acc[nt][i][3]);
            mine_part[(NT * MT + nt) * 32 + lane] = make_float4(mx[nt][0], mx[nt][1], sum[nt][0], sum[nt][1]);
        }
        together();
        if (ws > 1) {
            auto part = [&](int i) { return left + i * C::PART; };
            auto put = [&](int v, const auto& o, const float2& top, const float2& total) {
                if (complete) {
                    store(v, o, total);
                    return;
                }
#pragma unroll
                for (int i = 0; i < static_cast<int>(sizeof(o) / sizeof(o[0])); ++i) slot[(v + i) * 32 + lane] = o[i];
                if (v % MT == 0) slot[(NT * MT + v / MT) * 32 + lane] = make_float4(top.x, top.y, total.x, total.y);
            };
            if (ws > 2)
                join_parts<HD, NT, 1>(wi, ws, lane, ws, part, put);
            else
                join_parts<HD, NT, 4>(wi, ws, lane, ws, part, put);
        }
        if (more || awaited) together();
        if (awaited && wi == 0 && lane == 0) {
            raise_part_flag(a.tag, [&](uint64_t v) { return exchange_gpu64(flags + slot_no, v); });
        }
        if (!more) break;
    }
    const Join jn = s_join[grp];
    if (jn.active) {                 // this worker's own part is its first
        const int count = worker - jn.from + 1;
        auto slot_of = [&](int i) { return (jn.from + i) * 2 + (i == 0 ? jn.from_slot : 0); };
        bool have = true;
        for (int i = wi * 32 + lane; i + 1 < count; i += ws * 32)
            have = have && flag64_wait(flags + slot_of(i), a.tag, &s_abort, a.seqs.status);
        together();
        auto part = [&](int i) { return slots + static_cast<size_t>(slot_of(i)) * C::PART; };
        auto put = [&](int v, const auto& o, const float2&, const float2& total) {
            store_vectors<HD>(a, jn.head, jn.first_row, jn.rows, jn.tile * COLS, lane, v, o, total);
        };
        if (ws > 2)
            join_parts<HD, NT, 1>(wi, ws, lane, count, part, put);
        else
            join_parts<HD, NT, 4>(wi, ws, lane, count, part, put);
        for (int i = wi * 32 + lane; i + 1 < count; i += ws * 32) {
            uint64_t* flag = flags + slot_of(i);
            if (have)
                *flag = 0;
            else
                give_up_part_flag(a.tag, [&](uint64_t v) { return exchange_gpu64(flag, v); });
        }
    }
    if (dead) spin_ns(1000000);      // copies that were issued land before the block's memory is given back
}

template <int HD, int NT>
tp_status launch_few(const AttnArgs& a, int sms, cudaStream_t stream) {
    using C = Cfg<HD, NT>;
    static std::atomic<uint64_t> smem_set{0};
    auto* kern = kv4_attention_kernel<HD, NT>;
    if (!smem_attribute_once(reinterpret_cast<const void*>(kern), C::SMEM, smem_set)) return TP_ERR_CUDA;
    if (launch_pdl(kern, dim3(sms), dim3(C::WARPS * 32), C::SMEM, stream, a) != cudaSuccess) return TP_ERR_CUDA;
    return TP_OK;
}

}  // namespace

size_t kv4_attention_workspace(int t, int64_t n, int64_t nseq, int heads, int kv_heads, int head_dim) {
    (void)t, (void)n, (void)nseq, (void)heads, (void)kv_heads;
    // two parts for each of the workers that an SM can have
    const int sms = std::max(device_sms(), 160);
    return flag_bytes(sms) + static_cast<size_t>(sms) * kWarps * 2 * slot_vectors(2, head_dim) * sizeof(float4);
}

tp_status launch_kv4_attention(const KvAttentionDesc& d, cudaStream_t stream) {
    AttnArgs a;
    a.seqs = d.seqs;
    a.pools = d.pools;
    for (int r = 0; r < TP_MAX_SHARDS; ++r) {
        a.q[r] = static_cast<const uint16_t*>(d.q[r]);
        a.out[r] = static_cast<uint16_t*>(d.out[r]);
    }
    a.ldq = d.ldq;
    a.ldo = d.ldo;
    a.group = d.group;
    a.scale_log2 = d.scale * 1.44269504088896f;
    a.window = d.window;
    a.sinks = d.sinks;
    a.ws = static_cast<uint8_t*>(d.ws);
    // numbers of calls begin at one that memory does not hold by chance
    static std::atomic<uint64_t> calls{0x9e3779b97f4a7c15ull ^ static_cast<uint64_t>(reinterpret_cast<uintptr_t>(&calls))};
    a.tag = calls.fetch_add(1, std::memory_order_relaxed) | 1ull << 63;
    const int sms = device_sms();
    if (sms <= 0 || sms > 160) return TP_ERR_CUDA;   // the workspace size is asked for without a device too
    // The kernels settle by the sequences' lengths which of them takes which; there is nothing to
    // settle while all rows together are too few (and without cu_rows each sequence has one).
    a.pairs = std::max(sms / 2, 1);
    a.many = INT32_MAX;
    const int64_t columns = static_cast<int64_t>(d.seqs.n) * d.group * d.pools.t * d.pools.kv_heads;
    if (d.seqs.cu_rows != nullptr && columns >= static_cast<int64_t>(kMany) * a.pairs) {
        a.many = kMany;
        const tp_status s = launch_attention_many(a, d.head_dim, stream);
        if (s != TP_OK) return s;
    }
    // 16 columns per tile where a sequence's rows fill more than 8 and there are enough tiles for every warp even so.
    // 4096 tokens, 16 columns for each of eight heads, tiles of 16 and of 8: 64 sequences 120 and 126 us, 16 42 and 39,
    // 4 27 and 21; of 64 dimensions, which leave more registers: 87 and 100, 30 and 32, 20 and 19 us.
    const bool filled = d.group > 8 || (d.seqs.cu_rows != nullptr && d.group * (d.seqs.n / std::max(d.seqs.nseq, 1)) > 8);
    const bool wide = filled && columns >= static_cast<int64_t>(sms) * (d.head_dim == 128 ? 48 : 12);
    if (d.head_dim == 128) return wide ? launch_few<128, 2>(a, sms, stream) : launch_few<128, 1>(a, sms, stream);
    return wide ? launch_few<64, 2>(a, sms, stream) : launch_few<64, 1>(a, sms, stream);
}

}  // namespace tpk

// Beam selection over vocab-sharded logits: one pass over the logits.  256 rows of
// 151936 fp32 logits take 50 us (39 and 11 for the kernels below; 2.7 TB/s), bound by
// the instructions of the scan (60 % of the issue slots) and the barriers at a
// piece's end; four rows of bf16 take 13 us, nearly all of it latency.
//
// First kernel: the logits of all rows are one line of chunks of 4096, cut into
// equal parts, one for each thread block that fits; a block's part of a row is a
// piece.  A ninth warp brings the chunks by bulk copies into a ring of three, so
// that two are on their way while one is worked on (128 KB for an SM; loads into
// registers, one chunk ahead in blocks of one row each, took 40 us for 136 MB,
// and a thread of the eight that also issues the copies holds up all of them).
// Each warp leaves the maximum of its 512 logits of a chunk and the sum of
// exponentials under it (fp32, an exponential from ex2).  Chunks count from a
// shard's first column, not from an aligned address, and what is joined over chunks
// is joined by the second kernel, so that a row's sum is the same wherever the row
// lies and its pieces begin: equal beams tie.  (Running sums over a piece took
// 48 us and gave such beams different last bits.)  A logit and its token make one 64-bit key, larger for a larger logit
// and, among equals, for a lower token, so the k best are unique.  The k-th
// largest of 64 group maxima (a group is 4 threads) of a piece's first chunk is
// a lower bound of the k-th largest of the piece; what is not below it goes to
// shared memory, so the pass costs one comparison per thread and 16 logits (a
// warp looks at the logits of a thread that has some together, half a warp for
// each: 6 % less time for those 256 rows than when each thread compares its
// own 16).  As the piece goes on, the k best so far are found by counting and the
// bound rises to the last of them: 40 candidates instead of 145 for k = 8 in 17
// chunks.
// Where more than kRoom at once are not below the bound (many equal logits), k
// rounds of a block-wide maximum over the piece find them instead.
//
// Second kernel, one thread block per item: the log-sum-exp of each beam from
// its warps' sums (expf joins them, in fp64 from pairs on), then the k best of all beams' candidates by the fp64 sum
// score - lse + logit, the same way.  It is a chain of latencies; fp64 is slow
// here (16 cycles an instruction and warp), so a beam takes one logarithm
// in it and no exponential.
#include <algorithm>

#include "kv4.cuh"

namespace tpk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 64;
constexpr int kRoom = 512;           // candidates that are ranked by counting
static_assert(kGroups >= TP_MAX_BEAMS, "the bound needs as many groups as there are results");

// A warp's logits of a chunk.
struct __align__(8) Part {
    float top;                       // the largest, -inf: nothing but -inf (and perhaps NaN)
    float sum;                       // of e^(x - top)
};

struct BeamArgs {
    const void* logits[TP_MAX_SHARDS];
    int64_t cols[TP_MAX_SHARDS], ldl[TP_MAX_SHARDS], start[TP_MAX_SHARDS];
    int first_chunk[TP_MAX_SHARDS + 1];  // chunks of a row, by shard
    int t, items, beams, k;
    int chunks;                      // of a row
    int blocks;                      // parts of the line
    int most;                        // pieces that a row can have
    int64_t vocab;
    const float* scores;
    const uint8_t* finished;
    int eos;
    float* scores_out;
    int32_t* rows_out;
    int32_t* tokens_out;
    Part* stats;                     // [rows, chunks, kWarps]
    uint64_t* keys;                  // [rows, most, k], best first, 0 where there are fewer
    int* status;
};

// The line of rows * chunks chunks in `blocks` equal parts; the first `more` hold one more.
struct Line {
    int64_t each, more;
    __device__ __forceinline__ explicit Line(const BeamArgs& a) {
        const int64_t total = static_cast<int64_t>(a.items) * a.beams * a.chunks;
        each = quotient(total, a.blocks);
        more = total - each * a.blocks;
    }
    __device__ __forceinline__ int64_t begin(int b) const { return each * b + min(static_cast<int64_t>(b), more); }
    __device__ __forceinline__ int of(int64_t i) const {
        const int64_t front = (each + 1) * more;
        return static_cast<int>(i < front ? quotient(i, each + 1) : more + quotient(i - front, each));
    }
};

// Order-preserving map of a float (not NaN; -0 as +0) to 32 bits.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t ordered64(double x) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(__dadd_rn(x, 0.0)));
    return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered64(uint64_t o) {
    return __longlong_as_double(static_cast<int64_t>(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}

// The k-th largest (k >= 1) of the 64 group maxima in `group`, into *out, by the first 64 threads; 0 is "none".
// The block synchronises before and after.
template <typename T>
__device__ __forceinline__ void kth_of_groups(const T* group, int k, int tid, T* out) {
    if (tid >= kGroups) return;
    const T mine = group[tid];
    int before = 0;                  // ties by place
    struct alignas(16) Some {        // one 16-byte read
        T v[16 / sizeof(T)];
    };
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kGroups; i += PER) {
        const Some g = *reinterpret_cast<const Some*>(group + i);
#pragma unroll
        for (int j = 0; j < PER; ++j) before += g.v[j] > mine || (g.v[j] == mine && i + j < tid);
    }
    if (before == k - 1) *out = mine;
}

// Group maxima of the threads' values: threads 4g .. 4g + 3 are group g.
template <typename T>
__device__ __forceinline__ void group_max(T v, T* group, int tid) {
    T o = __shfl_xor_sync(0xffffffffu, v, 1);
    v = v > o ? v : o;
    o = __shfl_xor_sync(0xffffffffu, v, 2);
    v = v > o ? v : o;
    if ((tid & 3) == 0) group[tid >> 2] = v;
}

// The barrier of the kThreads threads that compute.
__device__ __forceinline__ void sync_all() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

__device__ __forceinline__ uint64_t block_max64(uint64_t v, uint64_t* tmp, int tid) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, v, m);
        v = v > o ? v : o;
    }
    sync_all();
    if ((tid & 31) == 0) tmp[tid >> 5] = v;
    sync_all();
    v = tmp[0];
    for (int i = 1; i < kWarps; ++i) v = v > tmp[i] ? v : tmp[i];
    return v;
}

constexpr int kChunk = 16;           // logits of a thread in one go
constexpr float kLog2e = 1.4426950408889634f;

// What a sum under maximum `from` is worth under `to` >= from: times this (0 for a sum of nothing).
__device__ __forceinline__ float carried(float from, float to) { return from == -INFINITY ? 0.0f : expf(from - to); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of the warp's values, NaN aside (-inf where there is nothing else).
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kAtOnce = 4;           // blocks of an SM
constexpr int kAhead = 12;           // parts of a row that a lane of the second kernel asks for at once
constexpr int kRing = 3;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <bool F32>
__global__ void __launch_bounds__(kThreads + 32, kAtOnce) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
    constexpr int VEC = F32 ? 4 : 8, NV = kChunk / VEC, ES = F32 ? 4 : 2;
    constexpr uint32_t NONE = F32 ? 0xff800000u : 0xff80ff80u;           // -inf
    constexpr int WORDS = kThreads * NV, SLOT = WORDS + 1;               // of 16 bytes
    extern __shared__ __align__(128) uint4 ring[];                       // [kRing][SLOT]
    __shared__ __align__(8) uint64_t full[kRing], empty[kRing];
    __shared__ int4 s_place[kRing];              // of Place: token, lo, hi, off
    __shared__ int s_abort;
    __shared__ uint32_t s_none[1];               // what a place without a logit reads
    __shared__ __align__(16) uint32_t s_group[kGroups];
    __shared__ uint32_t s_bound;
    __shared__ __align__(16) uint64_t s_cand[kRoom + 2];
    __shared__ uint64_t s_best[TP_MAX_BEAMS];
    __shared__ uint64_t s_tmp[kWarps];
    __shared__ int s_count;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Line line(a);
    const int64_t begin = line.begin(blockIdx.x), end = line.begin(blockIdx.x + 1);

    auto done = [&](int row) { return a.finished != nullptr && a.finished[row] != 0; };   // its logits do not matter
    // Chunk c of a row, elements first .. of its shard.  A thread's words are VEC of them each, counted from the shard's
    // first, so that a row's sums do not depend on where it lies; in memory they begin `off` elements into a 16-byte
    // word, and the ring holds the chunk's memory words (one more where off is not 0), of which lo .. hi - 1 lie in
    // the row whole.
    struct Place {
        const uint8_t* base;                     // the row
        int64_t cols, first;
        int token, lo, hi, off;
    };
    auto place = [&](int row, int c) {
        int r = 0;
        while (c >= a.first_chunk[r + 1]) ++r;
        Place p;
        p.cols = a.cols[r];
        p.base = static_cast<const uint8_t*>(a.logits[r]) + row * a.ldl[r] * ES;
        p.off = static_cast<int>((reinterpret_cast<uintptr_t>(p.base) & 15u) / ES);
        p.first = static_cast<int64_t>(c - a.first_chunk[r]) * (kThreads * kChunk);
        p.token = static_cast<int>(a.start[r] + p.first);
        const int most = p.off ? SLOT : WORDS;
        p.lo = p.first == 0 && p.off ? 1 : 0;
        p.hi = static_cast<int>(max(static_cast<int64_t>(p.lo), min(static_cast<int64_t>(most), (p.cols - p.first + p.off) / VEC)));
        return p;
    };
    // whether a thread's word lies in memory words that are in the row whole
    auto inside = [](int word, int lo, int hi, int off) { return word >= lo && word + (off ? 1 : 0) < hi; };
    // a thread's word out of the memory words from `from` on
    auto word_of = [](const uint4* from, int word, int off) {
        const uint4 x = from[word], y = from[word + 1];
        uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const int skip = off * ES / 4;           // whole 32-bit words, then, of bf16, half of one
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = skip & 2 ? v[i + 2] : v[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) v[i] = skip & 1 ? v[i + 1] : v[i];
        if constexpr (!F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], (off & 1) * 16);
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    };
    // a word that the row's edge cuts, or one outside, element by element
    auto edge_word = [&](const Place& p, int word) {
        const int64_t col = p.first + word * VEC;
        uint32_t v[4] = {NONE, NONE, NONE, NONE};
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (col + e < p.cols) {
                if constexpr (F32) {
                    v[e] = reinterpret_cast<const uint32_t*>(p.base)[col + e];
                } else {
                    const uint32_t h = reinterpret_cast<const uint16_t*>(p.base)[col + e];
                    v[e / 2] = e & 1 ? (v[e / 2] & 0xffffu) | h << 16 : (v[e / 2] & 0xffff0000u) | h;
                }
            }
        return make_uint4(v[0], v[1], v[2], v[3]);
    };
    auto values = [&](const uint4 (&w)[NV], float (&x)[kChunk]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (F32) {
                    x[j * 4 + e] = __uint_as_float(v[e]);
                } else {
                    x[j * 8 + 2 * e] = __uint_as_float(v[e] << 16);
                    x[j * 8 + 2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
                }
            }
        }
    };
    auto key = [&](int token, int i, float x) {
        return (static_cast<uint64_t>(ordered(x)) << 32) |
               (0xffffffffu - static_cast<uint32_t>(token + i / VEC * kThreads * VEC + i % VEC));
    };
    // the k best of the candidates, in order, into s_best (0 where there are fewer); up to 128 of them are counted
    // against by two threads each
    auto rank = [&](int count) {
        if (tid < 2) s_cand[count + tid] = 0;    // read in pairs
        sync_all();
        const int both = count <= kThreads / 2 ? 1 : 0, pairs = (count + 1) / 2;
        for (int i = tid >> both; i < ((count + 31) & ~31); i += kThreads >> both) {
            const uint64_t mine = i < count ? s_cand[i] : ~0ull;
            const int lo = both && (tid & 1) ? pairs / 2 : 0, hi = both && !(tid & 1) ? pairs / 2 : pairs;
            int before = 0;
#pragma unroll 8
            for (int j = lo; j < hi; ++j) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(s_cand + 2 * j);
                before += (v.x > mine) + (v.y > mine);
            }
            if (both) before += __shfl_xor_sync(0xffffffffu, before, 1);
            if (i < count && before < a.k) s_best[before] = mine;
        }
        for (int i = count + tid; i < a.k; i += kThreads) s_best[i] = 0;
        sync_all();
    };

    int row = static_cast<int>(quotient(begin, a.chunks)), c = static_cast<int>(begin - static_cast<int64_t>(row) * a.chunks);
    if (tid == 0) {
        s_abort = 0;
        s_count = 0;
        s_none[0] = NONE;
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), kWarps);
            s_place[i] = make_int4(0, 0, 0, 0);  // what is read of a slot whose copy is lost stays in the ring
        }
    }
    fence_barrier_init();
    __syncthreads();
    if (warp == kWarps) {                        // brings the chunks
        if (lane != 0) return;
        int slot = 0, phase = 1;
        for (int64_t i = begin; i < end; ++row, c = 0) {
            const int n = static_cast<int>(min(static_cast<int64_t>(a.chunks - c), end - i));
            i += n;
            if (done(row)) continue;
            for (const int last = c + n; c < last; ++c) {
                const Place p = place(row, c);
                if (!mbar_wait(smem_u32(&empty[slot]), phase, &s_abort, a.status)) {
                    spin_ns(1000000);            // copies that were issued land
                    return;
                }
                const uint32_t bar = smem_u32(&full[slot]), bytes = static_cast<uint32_t>(p.hi - p.lo) * 16;
                s_place[slot] = make_int4(p.token, p.lo, p.hi, p.off);
                mbar_arrive_expect_tx(bar, bytes);
                if (bytes)
                    bulk_load(smem_u32(ring + slot * SLOT + p.lo), p.base + (p.first - p.off + p.lo * VEC) * ES, bytes, bar);
                if (++slot == kRing) slot = 0, phase ^= 1;
            }
        }
        if (*static_cast<volatile int*>(&s_abort)) spin_ns(1000000);     // nobody waits for the last copies then
        return;
    }
    int slot = 0, phase = 0;
    bool dead = false;                           // after a lost copy the barriers are kept, the results are not right
    for (int64_t i = begin; i < end;) {
        const int c0 = c, c1 = static_cast<int>(min(static_cast<int64_t>(a.chunks), c0 + (end - i)));    // the piece
        const bool skip = done(row);
        float bound = -INFINITY;
        bool weak = true;
        Part* stats = a.stats + (static_cast<int64_t>(row) * a.chunks + c) * kWarps + warp;
        for (; c < c1; ++c, ++i) {
            if (skip) continue;
            if (!dead) dead = !mbar_wait_warp(smem_u32(&full[slot]), phase, &s_abort, a.status);
            const int4 p = s_place[slot];
            const uint4* chunk = ring + slot * SLOT;
            uint4 w[NV];
            float x[kChunk];
            if (p.w == 0) {
#pragma unroll
                for (int j = 0; j < NV; ++j) w[j] = chunk[j * kThreads + tid];
            } else {
#pragma unroll
                for (int j = 0; j < NV; ++j) w[j] = word_of(chunk, j * kThreads + tid, p.w);
            }
            const bool partial = p.y != 0 || p.z != WORDS + (p.w ? 1 : 0);
            if (partial) {
                const Place q = place(row, c);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int word = j * kThreads + tid;
                    if (!inside(word, p.y, p.z, p.w)) w[j] = edge_word(q, word);
                }
            }
            values(w, x);
            float best = -INFINITY;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) best = fmaxf(best, x[e]);
            // The warp's sum under its maximum: 2^(x log2(e) - h), h = base log2(e) rounded, is one fma a term; what
            // the rounding of h makes of all of them is taken back from their sum.
            const float top = warp_max(best), base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f, back = 1.0f;
            if (fabsf(base) < 1e37f) {
                const float h = base * kLog2e;
                const uint64_t l2 = pack2(kLog2e, kLog2e), h2 = pack2(-h, -h);
                uint64_t u0 = 0, u1 = 0;
#pragma unroll
                for (int e = 0; e < kChunk; e += 4) {                    // NaN makes it NaN
                    float p0, p1, q0, q1;
                    unpack2(fma2(pack2(x[e], x[e + 1]), l2, h2), p0, p1);
                    unpack2(fma2(pack2(x[e + 2], x[e + 3]), l2, h2), q0, q1);
                    u0 = add2(u0, pack2(ex2(p0), ex2(p1)));
                    u1 = add2(u1, pack2(ex2(q0), ex2(q1)));
                }
                float p0, p1;
                unpack2(add2(u0, u1), p0, p1);
                sum = p0 + p1;
                back = ex2(-fmaf(base, kLog2e, -h));
            } else {                                                     // past fp32 times log2(e), or +inf: NaN
#pragma unroll
                for (int e = 0; e < kChunk; ++e) sum += ex2((x[e] - base) * kLog2e);
            }
#pragma unroll
            for (int e = 16; e >= 1; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
            if (lane == 0) *stats = Part{top, sum * back};
            stats += kWarps;
            if (weak) {                          // until a whole chunk has given the bound
                group_max(best > -INFINITY ? ordered(best) : 0u, s_group, tid);
                sync_all();
                kth_of_groups(s_group, a.k, tid, &s_bound);
                sync_all();
                if (s_bound != 0) bound = fmaxf(bound, unordered(s_bound));
                weak = partial || s_bound == 0;
                sync_all();
            }
            // Lanes with a logit that is not below the bound, two at a time, half a warp for the logits of each.
            uint32_t lanes = __ballot_sync(0xffffffffu, best >= bound && best > -INFINITY);
            if (lanes != 0) {
                __syncwarp();
                while (lanes != 0) {
                    const int l0 = __ffs(lanes) - 1;
                    lanes &= lanes - 1;
                    const int l1 = lanes != 0 ? __ffs(lanes) - 1 : -1;
                    lanes &= lanes - 1;
                    const int l = lane < kChunk ? l0 : l1, e = lane % kChunk, from = warp * 32 + max(l, 0);
                    const int word = e / VEC * kThreads + from;
                    const uint8_t* at_word = reinterpret_cast<const uint8_t*>(chunk + word) + (p.w + e % VEC) * ES;
                    if (partial && !inside(word, p.y, p.z, p.w)) {       // from the row itself, where it reaches there
                        const Place q = place(row, c);
                        const int64_t col = q.first + word * VEC + e % VEC;
                        at_word = col < q.cols ? q.base + col * ES : reinterpret_cast<const uint8_t*>(s_none);
                    }
                    const float logit = F32 ? *reinterpret_cast<const float*>(at_word) : bf16_to_f32(*reinterpret_cast<const uint16_t*>(at_word));
                    const bool take = l >= 0 && logit >= bound && logit > -INFINITY;
                    const uint32_t set = __ballot_sync(0xffffffffu, take);
                    int at = 0;
                    if (lane == 0) at = atomicAdd(&s_count, __popc(set));
                    at = __shfl_sync(0xffffffffu, at, 0) + __popc(set & ((1u << lane) - 1u));
                    if (take && at < kRoom) s_cand[at] = key(p.x + from * VEC, e, logit);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
            if (++slot == kRing) slot = 0, phase ^= 1;
            // after the piece's chunks 2, 4, 8 .. (and 1, where one chunk's candidates could fill half of the
            // room): the bound rises to the k-th best so far, so that each chunk lets about k / (its number) pass
            const int nth = c - c0;
            if ((nth & (nth + 1)) != 0 || (nth == 0 && a.k <= 16) || c + 1 == c1) continue;
            sync_all();
            const int count = s_count;
            if (count <= kRoom && count >= a.k) {
                rank(count);
                if (tid < a.k) s_cand[tid] = s_best[tid];
                bound = unordered(static_cast<uint32_t>(s_best[a.k - 1] >> 32));
                if (tid == 0) s_count = a.k;
            }
            sync_all();
        }
        if (!skip) {
            sync_all();                          // the candidates are in
            const int64_t out = static_cast<int64_t>(row) * a.most + (blockIdx.x - line.of(static_cast<int64_t>(row) * a.chunks));
            uint64_t* keys = a.keys + out * a.k;
            if (s_count <= kRoom) {
                rank(s_count);
                if (tid < a.k) keys[tid] = s_best[tid];
            } else {
                uint64_t last = ~0ull;
                for (int n = 0; n < a.k; ++n) {
                    uint64_t mine = 0;
                    for (int cc = c0; cc < c1; ++cc) {
                        const Place p = place(row, cc);
                        const int token = p.token + tid * VEC;
                        uint4 w[NV];
                        float x[kChunk];
#pragma unroll
                        for (int j = 0; j < NV; ++j) {
                            const int word = j * kThreads + tid;
                            const uint4* from = reinterpret_cast<const uint4*>(p.base + (p.first - p.off) * ES);
                            w[j] = !inside(word, p.lo, p.hi, p.off) ? edge_word(p, word)
                                   : p.off == 0                     ? from[word]
                                                                    : word_of(from, word, p.off);
                        }
                        values(w, x);
#pragma unroll
                        for (int e = 0; e < kChunk; ++e)
                            if (x[e] > -INFINITY) {
                                const uint64_t v = key(token, e, x[e]);
                                if (v < last && v > mine) mine = v;
                            }
                    }
                    last = block_max64(mine, s_tmp, tid);
                    if (tid == 0) keys[n] = last;
                }
            }
            if (tid == 0) s_count = 0;
            sync_all();
        }
        if (c == a.chunks) c = 0, ++row;
    }
}

// A continuation: its score (ordered64 of it, 0: none) and its place, beam in the upper half, token in the lower.
struct Cand {
    uint64_t score, place;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
    return a.score > b.score || (a.score == b.score && a.place < b.place);
}

// log of x >= 2^-1000 to about 1e-14 (x itself is good to about 2^-22): exponent and the series
// 2 (z + z^3/3 + ...) of log f, z = (f - 1) / (f + 1), for f in [3/4, 3/2).  A third of the library's fp64 instructions, which are what the second kernel waits for.
__device__ __forceinline__ double log_of_sum(double x) {
    const long long bits = __double_as_longlong(x);
    int e = static_cast<int>(bits >> 52) - 1023;
    double f = __longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll);
    if (f >= 1.5) f *= 0.5, ++e;
    const double d = f + 1.0;
    double r = static_cast<double>(1.0f / static_cast<float>(d));
    r = fma(r, fma(-d, r, 1.0), r);              // the reciprocal, by Newton's step
    const double z = (f - 1.0) * r, w = z * z;
    double p = 1.0 / 17;
    p = fma(p, w, 1.0 / 15);
    p = fma(p, w, 1.0 / 13);
    p = fma(p, w, 1.0 / 11);
    p = fma(p, w, 1.0 / 9);
    p = fma(p, w, 1.0 / 7);
    p = fma(p, w, 1.0 / 5);
    p = fma(p, w, 1.0 / 3);
    p = fma(p, w, 1.0);
    return fma(static_cast<double>(e), 0.693147180559945309417, 2.0 * z * p);
}

__global__ void __launch_bounds__(kThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ double s_add[TP_MAX_BEAMS];       // score - lse; NaN: no continuations
    __shared__ __align__(16) uint64_t s_group[kGroups];
    __shared__ uint64_t s_bound;
    __shared__ Cand s_cand[kRoom];
    __shared__ Cand s_best[kWarps];
    __shared__ int s_count;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = blockIdx.x;
    const int64_t row0 = static_cast<int64_t>(item) * a.beams;
    if (tid == 0) s_count = 0;
    // A warp takes every kWarps-th beam: f(continuation) for this lane's keys of each; a finished beam has
    // one.  With `first` it finds score - lse before.
    const Line line(a);
    auto each = [&](bool first, auto f) {
        for (int b = warp; b < a.beams; b += kWarps) {
            const bool done = a.finished != nullptr && a.finished[row0 + b] != 0;
            const int64_t begin = (row0 + b) * a.chunks;
            const int pieces = line.of(begin + a.chunks - 1) - line.of(begin) + 1, per_beam = pieces * a.k;
            const uint64_t* keys = a.keys + (row0 + b) * a.most * a.k;
            uint64_t key = !done && lane < per_beam ? keys[lane] : 0;
            if (first) {
                const float score = a.scores[row0 + b];
                double add = __longlong_as_double(0x7ff8000000000000ll);
                if (done) {
                    if (score > -INFINITY) add = score;
                } else {
                    // the sums of all chunks and warps, joined in an order that a row's sizes give
                    const Part* st = a.stats + (row0 + b) * a.chunks * kWarps;
                    const int parts = a.chunks * kWarps;
                    float top = -INFINITY;
                    double sum = 0.0;
                    for (int i0 = 0; i0 < parts; i0 += 32 * kAhead) {
                        Part part[kAhead];
                        float up = top;
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const int at = i0 + 32 * i + lane;
                            part[i] = at < parts ? st[at] : Part{-INFINITY, 0.0f};
                            up = fmaxf(up, part[i].top);
                        }
                        up = warp_max(up);
                        if (i0 != 0) sum *= carried(top, up);
                        top = up;
#pragma unroll
                        for (int i = 0; i < kAhead; i += 2)
                            if (i0 + 32 * i < parts)
                                sum += static_cast<double>(part[i].sum * carried(part[i].top, top) +
                                                           part[i + 1].sum * carried(part[i + 1].top, top));
                    }
#pragma unroll
                    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                    // a finite maximum's sum is at least 1, unless NaN is in it
                    if (score > -INFINITY && top > -INFINITY && top < INFINITY && sum >= 0.5)
                        add = score - (top + log_of_sum(sum));
                }
                if (lane == 0) s_add[b] = add;
                __syncwarp();
            }
            const double add = s_add[b];
            if (!(add == add)) continue;
            const uint64_t place = static_cast<uint64_t>(b) << 32;
            if (done) {
                if (lane == 0) f(Cand{ordered64(add), place | static_cast<uint32_t>(a.eos)});
                continue;
            }
            for (int i = lane; i < per_beam; i += 32) {
                if (key != 0)
                    f(Cand{ordered64(add + static_cast<double>(unordered(static_cast<uint32_t>(key >> 32)))),
                           place | (0xffffffffu - static_cast<uint32_t>(key))});
                if (i + 32 < per_beam) key = keys[i + 32];
            }
        }
    };
    uint64_t best = 0;
    each(true, [&](const Cand& c) { best = best > c.score ? best : c.score; });
    group_max(best, s_group, tid);
    __syncthreads();
    kth_of_groups(s_group, a.k, tid, &s_bound);
    __syncthreads();
    const uint64_t bound = s_bound > 1 ? s_bound : 1;
    each(false, [&](const Cand& c) {
        if (c.score >= bound) {
            const int at = atomicAdd(&s_count, 1);
            if (at < kRoom) s_cand[at] = c;
        }
    });
    __syncthreads();
    const int count = s_count;
    const int64_t out = static_cast<int64_t>(item) * a.k;
    auto put = [&](int at, const Cand& c) {
        a.scores_out[out + at] = c.score ? static_cast<float>(unordered64(c.score)) : -INFINITY;
        a.rows_out[out + at] = c.score ? static_cast<int32_t>(row0 + (c.place >> 32)) : -1;
        a.tokens_out[out + at] = c.score ? static_cast<int32_t>(c.place) : -1;
    };
    if (count <= kRoom) {
        for (int i = tid; i < count; i += kThreads) {
            const Cand mine = s_cand[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) rank += before(s_cand[j], mine);
            if (rank < a.k) put(rank, mine);
        }
        for (int i = count + tid; i < a.k; i += kThreads) put(i, Cand{0, 0});
        return;
    }
    Cand last{~0ull, 0};
    for (int m = 0; m < a.k; ++m) {
        Cand mine{0, ~0ull};
        each(false, [&](const Cand& c) {
            if (before(last, c) && before(c, mine)) mine = c;
        });
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) {
            const Cand o{__shfl_xor_sync(0xffffffffu, mine.score, s), __shfl_xor_sync(0xffffffffu, mine.place, s)};
            if (before(o, mine)) mine = o;
        }
        __syncthreads();
        if (lane == 0) s_best[warp] = mine;
        __syncthreads();
        last = s_best[0];
        for (int i = 1; i < kWarps; ++i)
            if (before(s_best[i], last)) last = s_best[i];
        if (tid == 0) put(m, last);
        if (last.score == 0) last = Cand{0, ~0ull};
    }
}

constexpr int kChunkLogits = kThreads * kChunk;

}  // namespace

size_t beam_workspace(int64_t items, int beams, int k, int64_t vocab) {
    // a row has at most as many pieces as chunks, and never more chunks than this
    const int64_t most = (vocab + kChunkLogits - 1) / kChunkLogits + TP_MAX_SHARDS;
    const int64_t rows = items * beams;
    return static_cast<size_t>(rows) * most * (kWarps * sizeof(Part) + static_cast<size_t>(k) * 8);
}

tp_status launch_beam_select(const BeamDesc& d, cudaStream_t stream) {
    BeamArgs a = {};
    const int64_t rows = static_cast<int64_t>(d.items) * d.beams;
    int64_t vocab = 0;
    for (int r = 0; r < d.t; ++r) {
        a.logits[r] = d.logits[r];
        a.cols[r] = d.cols[r];
        a.ldl[r] = d.ldl[r];
        a.start[r] = vocab;
        vocab += d.cols[r];
    }
    const int sms = device_sms();
    if (sms <= 0) return TP_ERR_CUDA;
    for (int r = 0; r < TP_MAX_SHARDS; ++r) {
        a.first_chunk[r] = a.chunks;
        if (r < d.t) a.chunks += static_cast<int>((d.cols[r] + kChunkLogits - 1) / kChunkLogits);
    }
    a.first_chunk[TP_MAX_SHARDS] = a.chunks;
    const int64_t total = rows * a.chunks;
    a.blocks = static_cast<int>(std::min<int64_t>(total, static_cast<int64_t>(sms) * kAtOnce));
    // a part holds at least `each` chunks, so a row lies in at most this many
    const int64_t each = total / a.blocks;
    a.most = static_cast<int>(std::min<int64_t>(a.chunks, (a.chunks - 1) / each + 2));
    a.t = d.t;
    a.items = d.items;
    a.beams = d.beams;
    a.k = d.k;
    a.vocab = vocab;
    a.scores = d.scores;
    a.finished = d.finished;
    a.eos = d.eos;
    a.scores_out = d.scores_out;
    a.rows_out = d.rows_out;
    a.tokens_out = d.tokens_out;
    a.stats = static_cast<Part*>(d.ws);
    a.keys = reinterpret_cast<uint64_t*>(a.stats + rows * a.chunks * kWarps);
    const dim3 grid(a.blocks), block(kThreads + 32);
    a.status = device_status_word();
    constexpr int kSmem = kRing * (kThreads * kChunk * 4 + 16), kSmem16 = kRing * (kThreads * kChunk * 2 + 16);
    static std::atomic<uint64_t> smem_f32{0}, smem_bf16{0};
    if (!smem_attribute_once(d.f32 ? reinterpret_cast<const void*>(beam_scan_kernel<true>)
                                   : reinterpret_cast<const void*>(beam_scan_kernel<false>),
                             kSmem, d.f32 ? smem_f32 : smem_bf16))
        return TP_ERR_CUDA;
    const cudaError_t e = d.f32 ? launch_pdl(beam_scan_kernel<true>, grid, block, kSmem, stream, a)
                                : launch_pdl(beam_scan_kernel<false>, grid, block, kSmem16, stream, a);
    if (e != cudaSuccess) return TP_ERR_CUDA;
    return launch_pdl(beam_pick_kernel, dim3(d.items), dim3(kThreads), 0, stream, a) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace tpk

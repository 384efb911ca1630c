// Beam selection over vocab-sharded logits: one pass over the logits, bound by
// reading them.
//
// First kernel, one thread block per (row, slice of a shard), which walks its
// slice 4096 logits at a time, the next ones already on their way.  Each thread
// keeps a running maximum and the sum of exponentials under it (fp32, an
// exponential from ex2; what joins sums under different maxima is expf, so that
// errors do not pile up; the threads' sums are added in fp64).  A logit and its token make one 64-bit key,
// larger for a larger logit and, among equals, for a lower token, so the k best
// are unique.  The k-th largest of 64 group maxima (a group is 4 threads) of the
// first 4096 is a lower bound of the k-th largest of the slice; what is not
// below it goes to shared memory, a few logits in a hundred threads' worth, so
// the pass costs one comparison per thread and 16 logits.  When the room fills
// up, the k best are found by counting and the bound rises to the last of them.
// Where more than kRoom at once are not below the bound (many equal logits), k
// rounds of a block-wide maximum over the slice find them instead.
//
// Second kernel, one thread block per item: the log-sum-exp of each beam from
// its slices, then the k best of all beams' candidates by the fp64 sum
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

struct Slice {
    double sum;                      // of e^(x - top)
    float top;                       // -inf: nothing but -inf (and perhaps NaN)
    int pad;
};

struct BeamArgs {
    const void* logits[TP_MAX_SHARDS];
    int64_t cols[TP_MAX_SHARDS], ldl[TP_MAX_SHARDS], start[TP_MAX_SHARDS];
    int first_slice[TP_MAX_SHARDS + 1];  // slices of a row, by shard
    int t, items, beams, k, slices, chunks;
    int64_t vocab;
    const float* scores;
    const uint8_t* finished;
    int eos;
    float* scores_out;
    int32_t* rows_out;
    int32_t* tokens_out;
    Slice* stats;                    // [rows, slices]
    uint64_t* keys;                  // [rows, slices, k], best first, 0 where there are fewer
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
#pragma unroll 16
    for (int i = 0; i < kGroups; ++i) before += group[i] > mine || (group[i] == mine && i < tid);
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

__device__ __forceinline__ uint64_t block_max64(uint64_t v, uint64_t* tmp, int tid) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, v, m);
        v = v > o ? v : o;
    }
    __syncthreads();
    if ((tid & 31) == 0) tmp[tid >> 5] = v;
    __syncthreads();
    v = tmp[0];
    for (int i = 1; i < kWarps; ++i) v = v > tmp[i] ? v : tmp[i];
    return v;
}

constexpr int kChunk = 16;           // logits of a thread in one go
constexpr float kLog2e = 1.4426950408889634f;

// What a sum under maximum `from` is worth under `to` >= from: times this (0 for a sum of nothing).
__device__ __forceinline__ float carried(float from, float to) { return from == -INFINITY ? 0.0f : expf(from - to); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) beam_slice_kernel(const __grid_constant__ BeamArgs a) {
    constexpr int VEC = F32 ? 4 : 8, NV = kChunk / VEC, ES = F32 ? 4 : 2;
    constexpr uint32_t NONE = F32 ? 0xff800000u : 0xff80ff80u;           // -inf
    __shared__ float s_top[kWarps];
    __shared__ double s_sum[kWarps];
    __shared__ uint32_t s_group[kGroups], s_bound;
    __shared__ uint64_t s_cand[kRoom], s_best[TP_MAX_BEAMS];
    __shared__ uint64_t s_tmp[kWarps];
    __shared__ int s_count;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / a.slices, slice = blockIdx.x - row * a.slices;
    if (a.finished != nullptr && a.finished[row] != 0) return;   // its logits do not matter
    int r = 0;
    while (slice >= a.first_slice[r + 1]) ++r;
    const int64_t cols = a.cols[r];
    const uint8_t* base = static_cast<const uint8_t*>(a.logits[r]) + row * a.ldl[r] * ES;
    // 16-byte words counted from the one that holds the row's first element
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / ES);
    const int64_t word0 = static_cast<int64_t>(slice - a.first_slice[r]) * a.chunks * (kThreads * NV);
    const int64_t words = (off + cols + VEC - 1) / VEC - word0;  // of the row from this slice on
    const int chunks = static_cast<int>(min(static_cast<int64_t>(a.chunks), (words + kThreads * NV - 1) / (kThreads * NV)));
    // column of the first element of this thread's word j of a chunk
    auto column = [&](int chunk, int j) { return (word0 + static_cast<int64_t>(chunk * NV + j) * kThreads + tid) * VEC - off; };
    auto load = [&](int chunk, uint4 (&w)[NV]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = column(chunk, j);
            if (c >= 0 && c + VEC <= cols) {
                w[j] = __ldg(reinterpret_cast<const uint4*>(base + c * ES));
            } else {                             // a word that the row's edge cuts, or one outside
                uint32_t v[4] = {NONE, NONE, NONE, NONE};
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (c + e >= 0 && c + e < cols) {
                        if constexpr (F32) {
                            v[e] = reinterpret_cast<const uint32_t*>(base)[c + e];
                        } else {
                            const uint32_t h = reinterpret_cast<const uint16_t*>(base)[c + e];
                            v[e / 2] = e & 1 ? (v[e / 2] & 0xffffu) | h << 16 : (v[e / 2] & 0xffff0000u) | h;
                        }
                    }
                w[j] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
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
    auto key = [&](int chunk, int i, float x) {
        return (static_cast<uint64_t>(ordered(x)) << 32) |
               (0xffffffffu - static_cast<uint32_t>(a.start[r] + column(chunk, i / VEC) + i % VEC));
    };
    // the k best of the candidates, in order, into s_best (0 where there are fewer)
    auto rank = [&](int count) {
        for (int i = tid; i < count; i += kThreads) {
            const uint64_t mine = s_cand[i];
            int before = 0;
            for (int j = 0; j < count; ++j) before += s_cand[j] > mine;
            if (before < a.k) s_best[before] = mine;
        }
        for (int i = count + tid; i < a.k; i += kThreads) s_best[i] = 0;
        __syncthreads();
    };
    if (tid == 0) s_count = 0;
    uint4 next[NV];
    load(0, next);
    float m = -INFINITY, s = 0.0f;
    float bound = -INFINITY;
    bool over = false;
    for (int c = 0; c < chunks; ++c) {
        float x[kChunk];
        values(next, x);
        if (c + 1 < chunks) load(c + 1, next);
        float best = x[0];
#pragma unroll
        for (int i = 1; i < kChunk; ++i) best = fmaxf(best, x[i]);
        if (best > m) {
            s *= m == -INFINITY ? 1.0f : expf(m - best);                 // a sum of nothing is 0, or NaN
            m = best;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kChunk; i += 2) {                            // NaN and +inf make it NaN
            s += ex2((x[i] - base) * kLog2e);
            s1 += ex2((x[i + 1] - base) * kLog2e);
        }
        s += s1;
        if (c == 0) {
            group_max(best > -INFINITY ? ordered(best) : 0u, s_group, tid);
            __syncthreads();
            kth_of_groups(s_group, a.k, tid, &s_bound);
            __syncthreads();
            bound = s_bound == 0 ? -INFINITY : unordered(s_bound);
        }
        if (best >= bound) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (x[i] >= bound && x[i] > -INFINITY) {
                    const int at = atomicAdd(&s_count, 1);
                    if (at < kRoom) s_cand[at] = key(c, i, x[i]);
                }
        }
        __syncthreads();
        const int count = s_count;
        __syncthreads();                         // nobody adds before everybody has read
        over = count > kRoom;
        if (over) {                              // the sum goes on, the candidates are found below
            bound = INFINITY;
            if (tid == 0) s_count = kRoom + 1;
        } else if (count > kRoom / 2 && c + 1 < chunks) {
            rank(count);
            if (tid < a.k) s_cand[tid] = s_best[tid];
            bound = unordered(static_cast<uint32_t>(s_best[a.k - 1] >> 32));
            if (tid == 0) s_count = a.k;
            __syncthreads();
        }
    }
    // the slice's maximum and sum
    float top = m;
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    top = s_top[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) top = fmaxf(top, s_top[i]);
    double sum = s * carried(m, top);            // NaN stays
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    if (lane == 0) s_sum[warp] = sum;
    const int64_t out = static_cast<int64_t>(row) * a.slices + slice;
    uint64_t* keys = a.keys + out * a.k;
    if (!over) {
        rank(s_count);
        if (tid < a.k) keys[tid] = s_best[tid];
    } else {
        uint64_t last = ~0ull;
        for (int n = 0; n < a.k; ++n) {
            uint64_t mine = 0;
            for (int c = 0; c < chunks; ++c) {
                uint4 w[NV];
                float x[kChunk];
                load(c, w);
                values(w, x);
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    if (x[i] > -INFINITY) {
                        const uint64_t v = key(c, i, x[i]);
                        if (v < last && v > mine) mine = v;
                    }
            }
            last = block_max64(mine, s_tmp, tid);
            if (tid == 0) keys[n] = last;
        }
    }
    if (tid == 0) {
        Slice st;
        st.top = top;
        st.pad = 0;
        st.sum = 0.0;
        for (int i = 0; i < kWarps; ++i) st.sum += s_sum[i];
        a.stats[out] = st;
    }
}

// A continuation: its score (ordered64 of it, 0: none) and its place beam * vocab + token.
struct Cand {
    uint64_t score, flat;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
    return a.score > b.score || (a.score == b.score && a.flat < b.flat);
}

__global__ void __launch_bounds__(kThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ double s_add[TP_MAX_BEAMS];       // score - lse; NaN: no continuations
    __shared__ uint64_t s_group[kGroups], s_bound;
    __shared__ Cand s_cand[kRoom];
    __shared__ Cand s_best[kWarps];
    __shared__ float s_top[TP_MAX_BEAMS];
    __shared__ int s_count;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = blockIdx.x;
    const int64_t row0 = static_cast<int64_t>(item) * a.beams;
    auto done = [&](int b) { return a.finished != nullptr && a.finished[row0 + b] != 0; };
    if (tid == 0) s_count = 0;
    // this thread's candidates, the first few of which it keeps: a key of a beam's slice each; a finished
    // beam has its first alone
    const int per_beam = a.slices * a.k, n = a.beams * per_beam;
    constexpr int KEEP = 8;
    uint64_t key[KEEP];
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const int i = tid + j * kThreads;
        key[j] = i < n ? a.keys[row0 * per_beam + i] : 0;
    }
    for (int b = warp; b < a.beams; b += kWarps) {
        if (done(b)) continue;
        const Slice* st = a.stats + (row0 + b) * a.slices;
        Slice mine{0.0, -INFINITY, 0};
        if (lane < a.slices) mine = st[lane];
        for (int i = lane + 32; i < a.slices; i += 32) {
            const Slice o = st[i];
            const float up = fmaxf(mine.top, o.top);
            mine.sum = mine.sum * carried(mine.top, up) + o.sum * carried(o.top, up);
            mine.top = up;
        }
        float top = mine.top;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        double sum = mine.sum * carried(mine.top, top);
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane == 0) s_add[b] = sum, s_top[b] = top;
    }
    __syncthreads();
    for (int b = tid; b < a.beams; b += kThreads) {
        const float score = a.scores[row0 + b];
        double add = __longlong_as_double(0x7ff8000000000000ll);
        if (done(b)) {
            if (score > -INFINITY) add = score;
        } else if (score > -INFINITY) {
            const double lse = s_top[b] + log(s_add[b]);
            if (lse > -INFINITY && lse < INFINITY) add = score - lse;
        }
        s_add[b] = add;
    }
    __syncthreads();
    auto cand = [&](int i, uint64_t k64) {
        Cand c{0, 0};
        const uint32_t b = static_cast<uint32_t>(i) / static_cast<uint32_t>(per_beam);
        const double add = s_add[b];
        if (!(add == add)) return c;
        if (done(b)) {
            if (i != static_cast<int>(b) * per_beam) return c;
            c.score = ordered64(add);
            c.flat = static_cast<uint64_t>(b) * a.vocab + static_cast<uint32_t>(a.eos);
            return c;
        }
        if (k64 == 0) return c;
        c.score = ordered64(add + static_cast<double>(unordered(static_cast<uint32_t>(k64 >> 32))));
        c.flat = static_cast<uint64_t>(b) * a.vocab + (0xffffffffu - static_cast<uint32_t>(k64));
        return c;
    };
    // f(candidate) for all of this thread's
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < KEEP; ++j)
            if (tid + j * kThreads < n) f(cand(tid + j * kThreads, key[j]));
        for (int i = tid + KEEP * kThreads; i < n; i += kThreads) f(cand(i, a.keys[row0 * per_beam + i]));
    };
    uint64_t best = 0;
    each([&](const Cand& c) { best = best > c.score ? best : c.score; });
    group_max(best, s_group, tid);
    __syncthreads();
    kth_of_groups(s_group, a.k, tid, &s_bound);
    __syncthreads();
    const uint64_t bound = s_bound > 1 ? s_bound : 1;
    if (best >= bound)
        each([&](const Cand& c) {
            if (c.score >= bound) {
                const int at = atomicAdd(&s_count, 1);
                if (at < kRoom) s_cand[at] = c;
            }
        });
    __syncthreads();
    const int count = s_count;
    const int64_t out = static_cast<int64_t>(item) * a.k;
    auto put = [&](int at, const Cand& c) {
        const int b = c.score ? static_cast<int>(c.flat / a.vocab) : 0;
        a.scores_out[out + at] = c.score ? static_cast<float>(unordered64(c.score)) : -INFINITY;
        a.rows_out[out + at] = c.score ? static_cast<int32_t>(row0 + b) : -1;
        a.tokens_out[out + at] = c.score ? static_cast<int32_t>(c.flat - static_cast<uint64_t>(b) * a.vocab) : -1;
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
        each([&](const Cand& c) {
            if (c.score != 0 && before(last, c) && before(c, mine)) mine = c;
        });
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) {
            const Cand o{__shfl_xor_sync(0xffffffffu, mine.score, s), __shfl_xor_sync(0xffffffffu, mine.flat, s)};
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

// Chunks of a slice: as many as leave six blocks for each SM (the registers allow five to run at once),
// at most 16.
int pick_chunks(int64_t rows, int64_t vocab, int sms) {
    const int64_t all = rows * ((vocab + kChunkLogits - 1) / kChunkLogits);
    return static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, all / (6 * sms))));
}

// Slices of a shard: its 16-byte words, one more for a row that begins inside a word.
int64_t slices_of(int64_t cols, int vec, int chunks) {
    if (cols == 0) return 0;
    const int64_t words = (cols + 2 * vec - 2) / vec, per = static_cast<int64_t>(kChunkLogits / vec) * chunks;
    return (words + per - 1) / per;
}

}  // namespace

size_t beam_workspace(int64_t items, int beams, int k, int64_t vocab) {
    // the most slices any cut of the vocabulary gives
    const int64_t slices = (vocab + kChunkLogits - 1) / kChunkLogits + 2 * TP_MAX_SHARDS;
    const int64_t rows = items * beams;
    return static_cast<size_t>(rows) * slices * (sizeof(Slice) + static_cast<size_t>(k) * 8);
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
    a.chunks = pick_chunks(rows, vocab, sms);
    int64_t slices = 0;
    for (int r = 0; r < TP_MAX_SHARDS; ++r) {
        a.first_slice[r] = static_cast<int>(slices);
        if (r < d.t) slices += slices_of(d.cols[r], d.f32 ? 4 : 8, a.chunks);
    }
    a.first_slice[TP_MAX_SHARDS] = static_cast<int>(slices);
    a.t = d.t;
    a.items = d.items;
    a.beams = d.beams;
    a.k = d.k;
    a.slices = static_cast<int>(slices);
    a.vocab = vocab;
    a.scores = d.scores;
    a.finished = d.finished;
    a.eos = d.eos;
    a.scores_out = d.scores_out;
    a.rows_out = d.rows_out;
    a.tokens_out = d.tokens_out;
    a.stats = static_cast<Slice*>(d.ws);
    a.keys = reinterpret_cast<uint64_t*>(a.stats + rows * slices);
    if (slices * rows > INT32_MAX) return TP_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(slices * rows)), block(kThreads);
    const cudaError_t e = d.f32 ? launch_pdl(beam_slice_kernel<true>, grid, block, 0, stream, a)
                                : launch_pdl(beam_slice_kernel<false>, grid, block, 0, stream, a);
    if (e != cudaSuccess) return TP_ERR_CUDA;
    return launch_pdl(beam_pick_kernel, dim3(d.items), block, 0, stream, a) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace tpk

// Beam selection over vocab-sharded logits: one pass over the logits, bound by
// reading them.
//
// First kernel, one thread block per (row, slice of a shard): the slice stays in
// registers; its maximum and the sum of exponentials under it (each term fp32,
// the terms of a thread added in fp32, the threads in fp64), and its k best
// logits.  A logit and its token make one 64-bit key, larger for a larger logit
// and, among equals, for a lower token, so the k best are unique.  The k-th
// largest of 64 group maxima (a group is 4 threads) is a lower bound of the k-th
// largest of the slice; what is not below it, a few more than k elements, goes
// to shared memory and is ranked by counting.  Where more than kRoom elements
// are not below the bound (many equal logits), k rounds of a block-wide
// maximum find them instead.
//
// Second kernel, one thread block per item: the log-sum-exp of each beam from
// its slices, then the k best of all beams' candidates by the fp64 sum
// score - lse + logit, the same way.
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
    double sum;
    float top;
    int pad;
};

struct BeamArgs {
    const void* logits[TP_MAX_SHARDS];
    int64_t cols[TP_MAX_SHARDS], ldl[TP_MAX_SHARDS], start[TP_MAX_SHARDS];
    int first_slice[TP_MAX_SHARDS + 1];  // slices of a row, by shard
    int t, items, beams, k, slices;
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

// The k-th largest (k >= 1) of the 64 group maxima in `group`, for every thread of a warp; 0 is "none".
template <typename T>
__device__ __forceinline__ T kth_of_groups(const T* group, int k, int lane) {
    const T a = group[lane], b = group[lane + 32];
    int ra = 0, rb = 0;              // how many are before it (ties by place)
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        const T u = __shfl_sync(0xffffffffu, a, i), v = __shfl_sync(0xffffffffu, b, i);
        ra += (u > a || (u == a && i < lane)) + (v > a);
        rb += (u >= b) + (v > b || (v == b && i < lane));
    }
    const uint32_t ha = __ballot_sync(0xffffffffu, ra == k - 1), hb = __ballot_sync(0xffffffffu, rb == k - 1);
    return ha ? __shfl_sync(0xffffffffu, a, __ffs(ha) - 1) : __shfl_sync(0xffffffffu, b, __ffs(hb) - 1);
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

// EPT elements per thread, VEC of them per 16-byte load.
template <int EPT, bool F32>
__global__ void __launch_bounds__(kThreads) beam_slice_kernel(const __grid_constant__ BeamArgs a) {
    constexpr int VEC = F32 ? 4 : 8, NV = EPT / VEC;
    __shared__ float s_top[kWarps];
    __shared__ double s_sum[kWarps];
    __shared__ uint32_t s_group[kGroups];
    __shared__ uint64_t s_cand[kRoom];
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
    constexpr int ES = F32 ? 4 : 2;
    const uint8_t* base = static_cast<const uint8_t*>(a.logits[r]) + row * a.ldl[r] * ES;
    // 16-byte words counted from the one that holds the row's first element
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / ES);
    const int64_t word0 = static_cast<int64_t>(slice - a.first_slice[r]) * (kThreads * NV);
    float x[EPT];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (word0 + j * kThreads + tid) * VEC - off;      // column of the word's first element
        if (c >= 0 && c + VEC <= cols) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(base + c * ES));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (F32) {
                    x[j * VEC + e] = __uint_as_float(w[e]);
                } else {
                    x[j * VEC + 2 * e] = __uint_as_float(w[e] << 16);
                    x[j * VEC + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float v = -INFINITY;
                if (c + e >= 0 && c + e < cols) {
                    if constexpr (F32)
                        v = reinterpret_cast<const float*>(base)[c + e];
                    else
                        v = bf16_to_f32(reinterpret_cast<const uint16_t*>(base)[c + e]);
                }
                x[j * VEC + e] = v;
            }
        }
    }
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPT; ++i) best = fmaxf(best, x[i]);
    float top = best;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (lane == 0) s_top[warp] = top;
    group_max(best == -INFINITY ? 0u : ordered(best), s_group, tid);
    if (tid == 0) s_count = 0;
    __syncthreads();
    top = s_top[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) top = fmaxf(top, s_top[i]);
    float part = 0.0f;
    if (top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) part += expf(x[i] - top);          // NaN and +inf make it NaN
    } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i) part += x[i] == x[i] ? 0.0f : x[i];
    }
    double sum = part;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == 0) s_sum[warp] = sum;

    const uint32_t bound = max(kth_of_groups(s_group, a.k, lane), 1u);
    auto key = [&](int i) {
        const int64_t c = (word0 + (i / VEC) * kThreads + tid) * VEC - off + i % VEC;
        return (static_cast<uint64_t>(ordered(x[i])) << 32) | (0xffffffffu - static_cast<uint32_t>(a.start[r] + c));
    };
    if (best > -INFINITY && ordered(best) >= bound) {
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            if (x[i] > -INFINITY && ordered(x[i]) >= bound) {
                const int at = atomicAdd(&s_count, 1);
                if (at < kRoom) s_cand[at] = key(i);
            }
    }
    __syncthreads();
    const int64_t out = static_cast<int64_t>(row) * a.slices + slice;
    if (tid == 0) {
        Slice s;
        s.top = top;
        s.pad = 0;
        s.sum = 0.0;
        for (int i = 0; i < kWarps; ++i) s.sum += s_sum[i];
        a.stats[out] = s;
    }
    uint64_t* keys = a.keys + out * a.k;
    const int count = s_count;
    if (count <= kRoom) {
        for (int i = tid; i < count; i += kThreads) {
            const uint64_t mine = s_cand[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) rank += s_cand[j] > mine;
            if (rank < a.k) keys[rank] = mine;
        }
        for (int i = count + tid; i < a.k; i += kThreads) keys[i] = 0;
    } else {
        uint64_t last = ~0ull;
        for (int n = 0; n < a.k; ++n) {
            uint64_t mine = 0;
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (x[i] > -INFINITY) {
                    const uint64_t v = key(i);
                    if (v < last && v > mine) mine = v;
                }
            last = block_max64(mine, s_tmp, tid);
            if (tid == 0) keys[n] = last;
        }
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
    __shared__ uint64_t s_group[kGroups];
    __shared__ Cand s_cand[kRoom];
    __shared__ Cand s_best[kWarps];
    __shared__ int s_count;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = blockIdx.x;
    const int64_t row0 = static_cast<int64_t>(item) * a.beams;
    if (tid == 0) s_count = 0;
    for (int b = warp; b < a.beams; b += kWarps) {
        const float score = a.scores[row0 + b];
        double add = __longlong_as_double(0x7ff8000000000000ll);
        if (a.finished != nullptr && a.finished[row0 + b] != 0) {
            if (score > -INFINITY) add = score;
        } else {
            const Slice* st = a.stats + (row0 + b) * a.slices;
            float top = -INFINITY;
            for (int i = lane; i < a.slices; i += 32) top = fmaxf(top, st[i].top);
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            double sum = 0.0;
            for (int i = lane; i < a.slices; i += 32) {
                const Slice s = st[i];
                if (s.top > -INFINITY)
                    sum += s.sum * exp(static_cast<double>(s.top) - top);
                else
                    sum += s.sum;                // 0, or NaN
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            const double lse = top + log(sum);
            if (score > -INFINITY && lse > -INFINITY && lse < INFINITY) add = score - lse;
        }
        if (lane == 0) s_add[b] = add;
    }
    __syncthreads();
    const int per_beam = a.slices * a.k;
    const int64_t n = static_cast<int64_t>(a.beams) * per_beam;
    // candidate i of the item: a key of a beam's slice; a finished beam has its first alone
    auto cand = [&](int64_t i) {
        Cand c{0, 0};
        const int b = static_cast<int>(i / per_beam), j = static_cast<int>(i - static_cast<int64_t>(b) * per_beam);
        const double add = s_add[b];
        if (!(add == add)) return c;
        if (a.finished != nullptr && a.finished[row0 + b] != 0) {
            if (j != 0) return c;
            c.score = ordered64(add);
            c.flat = static_cast<uint64_t>(b) * a.vocab + static_cast<uint32_t>(a.eos);
            return c;
        }
        const uint64_t key = a.keys[(row0 + b) * per_beam + j];
        if (key == 0) return c;
        c.score = ordered64(add + static_cast<double>(unordered(static_cast<uint32_t>(key >> 32))));
        c.flat = static_cast<uint64_t>(b) * a.vocab + (0xffffffffu - static_cast<uint32_t>(key));
        return c;
    };
    uint64_t best = 0;
    for (int64_t i = tid; i < n; i += kThreads) {
        const uint64_t s = cand(i).score;
        best = best > s ? best : s;
    }
    group_max(best, s_group, tid);
    __syncthreads();
    const uint64_t kth = kth_of_groups(s_group, a.k, lane), bound = kth > 1 ? kth : 1;
    if (best >= bound)
        for (int64_t i = tid; i < n; i += kThreads) {
            const Cand c = cand(i);
            if (c.score >= bound) {
                const int at = atomicAdd(&s_count, 1);
                if (at < kRoom) s_cand[at] = c;
            }
        }
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
        for (int64_t i = tid; i < n; i += kThreads) {
            const Cand c = cand(i);
            if (c.score != 0 && before(last, c) && before(c, mine)) mine = c;
        }
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

// Elements per thread of a slice: 32, or fewer while the slices would not fill the GPU twice.
int pick_ept(int64_t rows, int64_t vocab, int sms) {
    for (int e = 32; e > 8; e >>= 1)
        if (rows * ((vocab + kThreads * e - 1) / (kThreads * e)) >= 2 * sms) return e;
    return 8;
}

// Slices of a shard: its 16-byte words, one more for a row that begins inside a word.
int64_t slices_of(int64_t cols, int vec, int ept) {
    if (cols == 0) return 0;
    const int64_t words = (cols + 2 * vec - 2) / vec, per = static_cast<int64_t>(kThreads) * (ept / vec);
    return (words + per - 1) / per;
}

}  // namespace

size_t beam_workspace(int64_t items, int beams, int k, int64_t vocab) {
    // the most slices any cut of the vocabulary gives (8 elements per thread, 8 shards)
    const int64_t slices = (vocab + kThreads * 8 - 1) / (kThreads * 8) + 2 * TP_MAX_SHARDS;
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
    const int ept = pick_ept(rows, vocab, sms);
    int64_t slices = 0;
    for (int r = 0; r < TP_MAX_SHARDS; ++r) {
        a.first_slice[r] = static_cast<int>(slices);
        if (r < d.t) slices += slices_of(d.cols[r], d.f32 ? 4 : 8, ept);
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
    cudaError_t e;
    if (d.f32)
        e = ept == 32   ? launch_pdl(beam_slice_kernel<32, true>, grid, block, 0, stream, a)
            : ept == 16 ? launch_pdl(beam_slice_kernel<16, true>, grid, block, 0, stream, a)
                        : launch_pdl(beam_slice_kernel<8, true>, grid, block, 0, stream, a);
    else
        e = ept == 32   ? launch_pdl(beam_slice_kernel<32, false>, grid, block, 0, stream, a)
            : ept == 16 ? launch_pdl(beam_slice_kernel<16, false>, grid, block, 0, stream, a)
                        : launch_pdl(beam_slice_kernel<8, false>, grid, block, 0, stream, a);
    if (e != cudaSuccess) return TP_ERR_CUDA;
    return launch_pdl(beam_pick_kernel, dim3(d.items), block, 0, stream, a) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace tpk

// What the two attention kernels share: arguments, which blocks of its cache a
// run of rows sees, and which of the kernels takes a sequence.
#pragma once

#include "kv4.cuh"

namespace tpk {

struct AttnArgs {
    KvSeqs seqs;
    KvPools pools;
    const uint16_t* q[TP_MAX_SHARDS];
    uint16_t* out[TP_MAX_SHARDS];
    int64_t ldq, ldo;
    int group;                       // query heads per kv head
    float scale_log2;                // scale * log2(e)
    int window, sinks;
    int many;                        // columns (rows * group) from which a sequence may go to the many-rows kernel
    int pairs;                       // pairs of thread blocks that the device runs at once
    uint8_t* ws;
    uint64_t tag;                    // number of the call, never 0
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Spans of `span` tokens that rows at positions first .. last see: [0, front)
// for the sinks, then [start, start + count - front).
struct Spans {
    int front, start, count;
};
__device__ __forceinline__ Spans visible_spans(const AttnArgs& a, int64_t first, int64_t last, int span) {
    Spans v;
    const int64_t low = a.window > 0 ? first - a.window + 1 : 0;
    const int lo = low > 0 ? static_cast<int>(low) : 0;
    // tokens past the table are not there
    const int64_t most = a.seqs.max_blocks << a.pools.page_shift;
    int64_t end = (last + 1 + kKvBlock - 1) / kKvBlock;
    if (last < 0) end = 0;
    if (end > most) {
        raise_status(a.seqs.status, TP_ERR_INVALID_ARG);
        end = most;
    }
    const int per = span / kKvBlock;
    const int stop = static_cast<int>((end + per - 1) / per);
    v.front = lo > 0 ? min((min(a.sinks, lo) + span - 1) / span, stop) : 0;
    v.start = max(lo / span, v.front);
    v.count = v.front + max(0, stop - v.start);
    return v;
}

constexpr int kManyCols = 512;       // columns of a pair of thread blocks of the many-rows kernel

// Which kernel takes a sequence.  The few-rows kernel's time grows with the
// columns, the many-rows kernel's with the waves of pairs of blocks, however few
// columns they hold: over 4096 cached tokens of head dimension 128 the first takes
// 64 us for 4096 columns, 84 for 5504 and 111 for 8192, the second 77 to 78 us
// (dimension 64: 46, 59 and 80 us against 64 to 66; over 512 tokens, 128: 23, 26
// and 39 us against 32 to 33).  From 72 columns for each pair of each wave (5472 here),
// counted over the sequences that have 72 by themselves (a shorter one would leave
// a pair to fewer), the second is taken.  That is where they cross over 4096 tokens
// of dimension 128; with dimension 64 or short contexts, whose crossing is at 6000
// to 7000 columns, the second is up to a quarter slower between the two.  `cols`
// columns of such sequences for each of the heads make `tiles` tiles; both kernels
// come to the same answer.
__device__ __forceinline__ int many_tiles(const AttnArgs& a, int64_t cols) {
    return cols < a.many ? 0 : static_cast<int>((cols + kManyCols - 1) / kManyCols);
}
__device__ __forceinline__ bool many_pays(const AttnArgs& a, int64_t cols, int64_t tiles) {
    const int heads = a.pools.t * a.pools.kv_heads;
    const int64_t waves = quotient(tiles * heads + a.pairs - 1, a.pairs);
    return tiles > 0 && cols * heads >= waves * a.pairs * a.many;
}

tp_status launch_attention_many(const AttnArgs& a, int head_dim, cudaStream_t stream);

}  // namespace tpk

// The paged 4-bit KV cache: the layout of a block, where a token's block is,
// and which row belongs to which sequence.  See include/tp.h for the format.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "kernels.h"

namespace tpk {

// A block of 16 tokens of one kv head: key codes, value codes, key pairs, value pairs.
template <int HD>
struct KvBlock {
    static constexpr int ROW = HD / 2;                  // code bytes of one token
    static constexpr int KEYS = 0;
    static constexpr int VALS = kKvBlock * ROW;
    static constexpr int KPAIR = 2 * kKvBlock * ROW;    // (step, base) bf16 of each key
    static constexpr int VPAIR = KPAIR + 4 * kKvBlock;
    static constexpr int BYTES = VPAIR + 4 * kKvBlock;
    static_assert(BYTES == kKvBlock * (HD + 8), "block size of the format");
};

// a / b for a >= 0, b > 0: 32-bit division where it will do (a 64-bit one takes a hundred instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A page table or row offset outside its range (or a lost wait) is recorded
// once; an earlier error stays.
__device__ __forceinline__ void raise_status(int* status, tp_status code) {
    if (status != nullptr) atomicCAS(status, 0, static_cast<int>(code));
}

// Rows [first, first + count) of sequence s, count 0 when the offsets are out of order or range.
struct SeqRows {
    int first, count;
};
__device__ __forceinline__ SeqRows seq_rows(const KvSeqs& q, int s) {
    if (q.cu_rows == nullptr) return {s, 1};
    const int a = q.cu_rows[s], b = q.cu_rows[s + 1];
    if (a < 0 || b < a || b > q.n) {
        raise_status(q.status, TP_ERR_INVALID_ARG);
        return {0, 0};
    }
    return {a, b - a};
}

}  // namespace tpk

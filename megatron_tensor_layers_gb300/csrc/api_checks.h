// Argument checks that the C ABI's files share.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "tp.h"

namespace {

inline bool al2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int esize(tp_dtype d) { return d == TP_F32 ? 4 : 2; }
inline bool dtype_ok(int d) { return d == TP_BF16 || d == TP_F32; }
inline bool ld_ok(int64_t ld, int64_t minimum, int elem) { return ld >= minimum && (ld * elem) % 16 == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline cudaStream_t cs(tp_stream s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

#define TP_CHECK(cond, code) \
    do {                     \
        if (!(cond)) return (code); \
    } while (0)

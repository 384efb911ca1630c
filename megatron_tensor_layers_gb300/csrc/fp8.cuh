// Device helpers of the 8-bit floating-point operators: e4m3 codes with one
// fp32 scale for each group of 128.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace tpk {

constexpr float kFp8Max = 448.0f;                 // largest e4m3 value
constexpr float kFp8LeastAmax = 7.8886090522101181e-31f;   // 2^-100: a group's largest value counts as at least this,
                                                  // so that a scale and its quotients stay normal fp32 numbers

// The larger of two, NaN if one is: a group with a NaN gets a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float fp8_scale(float amax) { return __fdiv_rn(max_nan(amax, kFp8LeastAmax), kFp8Max); }

// Codes of four values (the first in the low byte), rounded to nearest even;
// values past the range give +-448, NaN gives NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Codes of x / scale: the quotient rounded to fp32, then to e4m3.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, float scale) {
    return e4m3x4(__fdiv_rn(a, scale), __fdiv_rn(b, scale), __fdiv_rn(c, scale), __fdiv_rn(d, scale));
}

// Largest |x| of eight values.
__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float m = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
    return m;
}

// Eight consecutive bf16 (one 16-byte load) or fp32 values (two).
template <bool F32>
struct Vec8 {
    uint4 q[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, int64_t element) {
        const char* p = static_cast<const char*>(base) + element * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) q[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (F32) {
            const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
};

// Largest of the 16 lanes of a half warp, in all of them.
__device__ __forceinline__ float max16(float m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

__device__ __forceinline__ uint2 fp8_codes8(const float (&x)[8], float scale) {
    return make_uint2(fp8_codes4(x[0], x[1], x[2], x[3], scale), fp8_codes4(x[4], x[5], x[6], x[7], scale));
}

}  // namespace tpk

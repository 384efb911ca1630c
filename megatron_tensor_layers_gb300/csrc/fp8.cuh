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

// amax / 448 rounded to nearest: the quotient of a constant, as Fp8Quotient's below (amax is at least 2^-100, so no
// remainder is subnormal); an infinity's remainder would be NaN and is left out.
__device__ __forceinline__ float fp8_scale(float amax) {
    constexpr float r = 1.0f / kFp8Max;
    const float a = max_nan(amax, kFp8LeastAmax);
    const float q0 = a * r;
    const float q1 = fmaf(fmaf(-q0, kFp8Max, a), r, q0);
    const float q2 = fmaf(fmaf(-q1, kFp8Max, a), r, q1);
    return a == __int_as_float(0x7f800000) ? a : q2;
}

// Codes of four values (the first in the low byte), rounded to nearest even;
// values past the range give +-448, NaN gives NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Pairs of fp32 values in one register pair, and two multiply-adds in one
// instruction.  The sums stay packed over the whole loop and a block's factor is packed
// once: packed in each multiply-add anew, 128 of them took a warp 220 cycles
// instead of 153.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 d, f32x2 s, f32x2 a) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(d), "l"(s), "l"(a));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Quotients x / scale rounded to nearest as a division's: with r = 1 / s
// rounded to nearest, q0 = x r is within 1.5 units of the last place, one
// correction q1 = q0 + (x - q0 s) r (the remainder is exact in an fma) brings it
// within one, and by Markstein's theorem a second then rounds correctly.  Two
// at a time, six packed operations instead of a reciprocal and steps for each.
// Scales below 2^-60 and their values are taken times 2^64, so that no
// remainder is subnormal.  An infinite scale's quotients are 0 (NaN of an
// infinity): there the remainders are taken with 0 in place of the scale.  Values
// and remainders are carried negated, so that a quotient of -0 stays one.
struct Fp8Quotient {
    f32x2 nf, s, nr;
    __device__ __forceinline__ explicit Fp8Quotient(float scale) {
        const float f = scale < 8.6736173798840355e-19f ? 1.8446744073709552e19f : 1.0f;   // 2^-60, 2^64
        const float sf = scale * f, r = __frcp_rn(sf);
        const float sr = sf == __int_as_float(0x7f800000) ? 0.0f : sf;
        nf = pack2(-f, -f);
        s = pack2(sr, sr);
        nr = pack2(-r, -r);
    }
    __device__ __forceinline__ f32x2 operator()(f32x2 x) const {
        const f32x2 nx = mul2(x, nf);
        const f32x2 q0 = mul2(nx, nr);
        const f32x2 q1 = fma2(fma2(q0, s, nx), nr, q0);
        return fma2(fma2(q1, s, nx), nr, q1);
    }
};

// Codes of four values.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, const Fp8Quotient& q) {
    float x, y, z, w;
    unpack2(q(pack2(a, b)), x, y);
    unpack2(q(pack2(c, d)), z, w);
    return e4m3x4(x, y, z, w);
}
__device__ __forceinline__ uint32_t fp8_codes4(f32x2 ab, f32x2 cd, const Fp8Quotient& q) {
    float x, y, z, w;
    unpack2(q(ab), x, y);
    unpack2(q(cd), z, w);
    return e4m3x4(x, y, z, w);
}

// act(g) of a gated block as g / (1 + exp(-z)): SiLU has z = g, and GeLU-tanh's
// 0.5 g (1 + tanh(u)) is z = 2 u with u = sqrt(2/pi) (g + 0.044715 g^3).  With
// coefficients in place of a branch, exp as 2^(g (a + b g^2)), and the hardware's
// 2^x and reciprocal (2^-22 and 1 ulp); two values at a time.
struct GateAct {
    f32x2 a, b;
    __device__ __forceinline__ explicit GateAct(int act) {
        constexpr float log2e = 1.4426950408889634f, k = 2.0f * 0.7978845608028654f;
        const bool gelu = act == TP_ACT_GELU_TANH_MUL;
        const float fa = gelu ? -k * log2e : -log2e, fb = gelu ? -k * 0.044715f * log2e : 0.0f;
        a = pack2(fa, fa);
        b = pack2(fb, fb);
    }
    __device__ __forceinline__ f32x2 operator()(f32x2 g) const {
        float s0, s1, e0, e1;
        unpack2(mul2(g, g), s0, s1);
        const f32x2 g2 = pack2(fminf(s0, 3.0e38f), fminf(s1, 3.0e38f));       // finite: b may be 0
        unpack2(mul2(g, fma2(b, g2, a)), s0, s1);
        asm("ex2.approx.f32 %0, %1;" : "=f"(e0) : "f"(s0));
        asm("ex2.approx.f32 %0, %1;" : "=f"(e1) : "f"(s1));
        asm("rcp.approx.f32 %0, %1;" : "=f"(s0) : "f"(1.0f + e0));
        asm("rcp.approx.f32 %0, %1;" : "=f"(s1) : "f"(1.0f + e1));
        return mul2(g, pack2(s0, s1));
    }
};

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
    const Fp8Quotient q(scale);
    return make_uint2(fp8_codes4(x[0], x[1], x[2], x[3], q), fp8_codes4(x[4], x[5], x[6], x[7], q));
}

}  // namespace tpk

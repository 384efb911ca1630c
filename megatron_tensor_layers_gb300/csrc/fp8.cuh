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

// The largest magnitude of three values; NaN if one of them is NaN.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The larger magnitudes of two pairs of bf16, with signs that mean nothing.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// amax / 448 rounded to nearest: q0 = a r with r = 1 / 448 rounded, and one
// correction by the exact remainder, which gives the rounded quotient for every
// 24-bit a (all of them were compared; amax is at least 2^-100, so no remainder is
// subnormal).  An infinity's remainder would be NaN and is left out.
__device__ __forceinline__ float fp8_scale(float amax) {
    constexpr float r = 1.0f / kFp8Max;
    const float a = max_nan(amax, kFp8LeastAmax);
    const float q0 = a * r;
    const float q1 = fmaf(fmaf(-q0, kFp8Max, a), r, q0);
    return a == __int_as_float(0x7f800000) ? a : q1;
}

// Codes of four values (the first in the low byte), rounded to nearest even;
// values past the range give +-448, NaN gives NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Quotients x / scale, of values given negated, as close as codes need: with r =
// 1 / s rounded to nearest, q0 = x r is within 1.5 units of the last place, and one
// correction q1 = q0 + (x - q0 s) r (the remainder is exact in an fma) leaves
// less than a unit.  A code goes by the side of the ties between codes (values of
// up to five significant bits) that the quotient lies on, and q1 lies on, or not
// on, the side of every tie as the rounded quotient does: compared for all 2^23
// significands of s, every tie t and the x next to s t.  Two at a time, three packed
// operations instead of a reciprocal and steps for each.  An infinite scale's
// quotients are 0 (NaN of an infinity): there the remainders are taken with 0 in
// place of the scale.  Carried negated, values and remainders leave a quotient of -0
// one.  Where `tiny`, s is below 2^-60, and it and the values are taken times 2^64
// first, so that no remainder is subnormal.
struct Fp8Quotient {
    f32x2 s, nr;
    bool tiny;
    __device__ __forceinline__ explicit Fp8Quotient(float scale) {
        tiny = scale < 8.6736173798840355e-19f;             // 2^-60
        const float sf = tiny ? scale * 1.8446744073709552e19f : scale;
        const float sr = sf == __int_as_float(0x7f800000) ? 0.0f : sf;
        const float r = __frcp_rn(sf);
        s = pack2(sr, sr);
        nr = pack2(-r, -r);
    }
    // Asked of the whole warp, for it is rare.
    __device__ __forceinline__ bool any_tiny() const { return __any_sync(0xffffffffu, tiny); }
    __device__ __forceinline__ f32x2 scaled(f32x2 nx) const {
        const float f = tiny ? 1.8446744073709552e19f : 1.0f;   // 2^64
        return mul2(nx, pack2(f, f));
    }
    __device__ __forceinline__ f32x2 operator()(f32x2 nx) const {
        const f32x2 q0 = mul2(nx, nr);
        return fma2(fma2(q0, s, nx), nr, q0);
    }
};

// Codes of 4 PAIRS / 2 values given negated, four a word; all lanes of the warp.
template <int PAIRS>
__device__ __forceinline__ void fp8_codes(f32x2 (&nx)[PAIRS], float scale, uint32_t (&out)[PAIRS / 2]) {
    const Fp8Quotient q(scale);
    if (q.any_tiny()) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) nx[i] = q.scaled(nx[i]);
    }
#pragma unroll
    for (int i = 0; i < PAIRS; i += 2) {
        float x, y, z, w;
        unpack2(q(nx[i]), x, y);
        unpack2(q(nx[i + 1]), z, w);
        out[i / 2] = e4m3x4(x, y, z, w);
    }
}

// Largest magnitude of pairs.
template <int PAIRS>
__device__ __forceinline__ float amax_pairs(const f32x2 (&x)[PAIRS]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float lo, hi;
        unpack2(x[i], lo, hi);
        m = max_abs(m, lo, hi);
    }
    return m;
}

// act(g) of a gated block as g s, s = 1 / (1 + exp(-z)): SiLU has z = g, and
// GeLU-tanh's 0.5 g (1 + tanh(u)) is z = 2 u with u = sqrt(2/pi) (g + 0.044715
// g^3).  Two values at a time, with the hardware's 2^x (2 ulp) and reciprocal (1 ulp).  The
// exponential of t = -z log2(e) alone would carry t's rounding, which grows with |g| (57 units of
// 2^-24 at g = -60, 148 for GeLU at -9), so what t's rounding left, times ln 2, goes along as m and
// moves s by its derivative, -s (1 - s) m (3876 rows of 4 x 5440 columns, K of 688: 170 us without,
// 183 with it; K of 8192: no difference that the clock does not hide).  act(g) times up is then within 10
// units of 2^-24: four of 2^x, one of the sum, two of the reciprocal, one each of the
// correction and the two products; where 2^t passes fp32's range act(g) is 0.  `negated`
// gives -act(g), with the same magnitude, as the codes' quotients take it.
template <int ACT>
struct GateAct {
    f32x2 sign;
    __device__ __forceinline__ explicit GateAct(bool negated) : sign(negated ? 0ull : 0x8000000080000000ull) {}
    // |g| past this has s of 0 or 1, and t and its rounding stay finite
    static constexpr float kLimit = ACT == TP_ACT_GELU_TANH_MUL ? 32.0f : 1.0e30f;
    // v where |v| is within the limit, else the limit with v's sign (of NaN either)
    static __device__ __forceinline__ float limited(float v) {
        float d;
        asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(v), "f"(kLimit));
        return d;
    }
    // -t, and -m
    static __device__ __forceinline__ f32x2 exponent(f32x2 g, f32x2& m) {
        constexpr double log2e = 1.4426950408889634074, k = 2.0 * 0.79788456080286535588, c = 0.044715;
        constexpr float ln2 = 0.69314718055994531f;
        if constexpr (ACT == TP_ACT_GELU_TANH_MUL) {
            // -t = h q, h = p g and q = 1 + c g^2, each with what its rounding left; 1 - q is exact below 2^24
            constexpr float p = static_cast<float>(k * log2e), pl = static_cast<float>(k * log2e - static_cast<double>(p));
            constexpr float ch = static_cast<float>(c), cl = static_cast<float>(c - static_cast<double>(ch));
            const f32x2 w = mul2(g, g), wl = fma2(g, g, neg2(w));
            const f32x2 q = fma2(w, both(ch), both(1.0f));
            f32x2 ql = fma2(w, both(ch), fma2(q, both(-1.0f), both(1.0f)));
            ql = fma2(w, both(cl), ql);
            ql = fma2(wl, both(ch), ql);
            const f32x2 h = mul2(g, both(p)), hl = fma2(g, both(pl), fma2(g, both(p), neg2(h)));
            const f32x2 nt = mul2(h, q);
            f32x2 r = fma2(h, q, neg2(nt));
            r = fma2(hl, q, r);
            r = fma2(h, ql, r);
            m = mul2(r, both(ln2));
            return nt;
        } else {
            constexpr float p = static_cast<float>(log2e), pl = static_cast<float>(log2e - static_cast<double>(p));
            const f32x2 nt = mul2(g, both(p));
            const f32x2 r = fma2(g, both(-p), nt);               // t's rounding, but for p's own
            m = mul2(fma2(g, both(-pl), r), both(-ln2));
            return nt;
        }
    }
    __device__ __forceinline__ f32x2 operator()(f32x2 g) const {
        float x0, x1, e0, e1;
        unpack2(g, x0, x1);
        f32x2 m;
        unpack2(exponent(pack2(limited(x0), limited(x1)), m), x0, x1);
        asm("ex2.approx.f32 %0, %1;" : "=f"(e0) : "f"(-x0));
        asm("ex2.approx.f32 %0, %1;" : "=f"(e1) : "f"(-x1));
        unpack2(fma2(pack2(e0, e1), both(-1.0f), both(-1.0f)), e0, e1);
        asm("rcp.approx.f32 %0, %1;" : "=f"(x0) : "f"(e0));
        asm("rcp.approx.f32 %0, %1;" : "=f"(x1) : "f"(e1));
        const f32x2 ns = pack2(x0, x1);                          // -s; with ns^2 + ns = -s (1 - s)
        return mul2(g ^ sign, fma2(m, fma2(ns, ns, ns), ns));
    }
};

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
    // the largest magnitude
    __device__ __forceinline__ float amax() const {
        if constexpr (F32) {
            const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) m = max_abs(m, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
            return m;
        } else {
            const uint32_t m = max_abs_bf16x2(max_abs_bf16x2(q[0].x, q[0].y), max_abs_bf16x2(q[0].z, q[0].w));
            return max_abs(0.0f, __uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        }
    }
    // the eight values negated, in pairs
    __device__ __forceinline__ void negated(f32x2 (&x)[4]) const {
        if constexpr (F32) {
            const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = pack2(-__uint_as_float(w[2 * i]), -__uint_as_float(w[2 * i + 1]));
        } else {
            const uint32_t w[4] = {q[0].x ^ 0x80008000u, q[0].y ^ 0x80008000u, q[0].z ^ 0x80008000u, q[0].w ^ 0x80008000u};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
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

}  // namespace tpk

// Rows and weights brought to 8 bits (e4m3 codes, one fp32 scale for each
// group of 128 columns of a row or each 128 x 128 block of a weight), and the
// norm between two layers with its rows in 8 bits.
//
//   scale = max(amax of the group, 2^-100) / 448,  code = e4m3(x / scale)
//
// Every operation is rounded to fp32, so codes and scales are those of the
// same formulas anywhere.  A group with a NaN or an infinity stands for NaN
// in every element (its scale is NaN or infinite).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8.cuh"
#include "kernels.h"

namespace tpk {

struct Fp8QuantArgs {
    const void* x[TP_MAX_SHARDS];
    uint8_t* codes[TP_MAX_SHARDS];
    float* scales[TP_MAX_SHARDS];
    int64_t n, k, ldx, ldc, lds, half;
    int groups;          // groups of a row
    int blocks_half;     // weight: blocks of the first part's rows
};

// ------------------------------------------------------------------ rows
//
// Sixteen lanes hold a group (eight elements each); a thread issues the loads
// of kQuantUnits groups before it uses the first.
constexpr int kQuantThreads = 256;
constexpr int kQuantUnits = 4;

template <bool F32>
__global__ void __launch_bounds__(kQuantThreads) fp8_quant_rows_kernel(const __grid_constant__ Fp8QuantArgs a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int r = blockIdx.y;
    const int lane16 = threadIdx.x & 15;
    const int64_t units = a.n * a.groups;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 16 * kQuantUnits) + (threadIdx.x >> 4);
    Vec8<F32> v[kQuantUnits];
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u) {
        const int64_t unit = first + u * (kQuantThreads / 16);
        const int64_t row = unit / a.groups;
        const int64_t col = (unit - row * a.groups) * kFp8Group + lane16 * 8;
        if (unit < units && col < a.k)
            v[u].load(a.x[r], row * a.ldx + col);
        else
            v[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kQuantUnits; ++u) {
        const int64_t unit = first + u * (kQuantThreads / 16);
        const int64_t row = unit / a.groups;
        const int64_t g = unit - row * a.groups;
        const int64_t col = g * kFp8Group + lane16 * 8;
        float x[8];
        v[u].get(x);
        const float s = fp8_scale(max16(amax8(x)));
        if (unit < units && col < a.k) {
            *reinterpret_cast<uint2*>(a.codes[r] + row * a.ldc + col) = fp8_codes8(x, s);
            if (lane16 == 0) a.scales[r][g * a.lds + row] = s;
        }
    }
}

// ------------------------------------------------------------------ weights
//
// One thread block per 128 x 128 block, held in registers between its largest
// value and its codes.
constexpr int kWeightRowsPerPass = kQuantThreads / 16;
constexpr int kWeightPasses = kFp8Group / kWeightRowsPerPass;

template <bool F32>
__global__ void __launch_bounds__(kQuantThreads) fp8_quant_weight_kernel(const __grid_constant__ Fp8QuantArgs a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    __shared__ float warp_max[kQuantThreads / 32];
    const int r = blockIdx.z;
    const int lane16 = threadIdx.x & 15;
    // rows [row0, row_end): a block ends with its part
    const int64_t nb = blockIdx.y;
    const bool second = a.half > 0 && nb >= a.blocks_half;
    const int64_t row0 = second ? a.half + (nb - a.blocks_half) * kFp8Group : nb * kFp8Group;
    const int64_t row_end = a.half > 0 && !second ? a.half : a.n;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kFp8Group + lane16 * 8;
    Vec8<F32> v[kWeightPasses];
#pragma unroll
    for (int i = 0; i < kWeightPasses; ++i) {
        const int64_t row = row0 + i * kWeightRowsPerPass + (threadIdx.x >> 4);
        if (row < row_end && col < a.k)
            v[i].load(a.x[r], row * a.ldx + col);
        else
            v[i].zero();
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kWeightPasses; ++i) {
        float x[8];
        v[i].get(x);
        m = max_nan(m, amax8(x));
    }
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
    m = max16(m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = max_nan(m, warp_max[w]);
    const float s = fp8_scale(m);
#pragma unroll
    for (int i = 0; i < kWeightPasses; ++i) {
        const int64_t row = row0 + i * kWeightRowsPerPass + (threadIdx.x >> 4);
        float x[8];
        v[i].get(x);
        if (row < row_end && col < a.k) *reinterpret_cast<uint2*>(a.codes[r] + row * a.ldc + col) = fp8_codes8(x, s);
    }
    if (threadIdx.x == 0) a.scales[r][nb * a.lds + blockIdx.x] = s;
}

tp_status launch_fp8_quant(const Fp8QuantDesc& d, cudaStream_t stream) {
    if (d.n == 0) return TP_OK;
    Fp8QuantArgs a = {};
    for (int r = 0; r < d.t; ++r) {
        a.x[r] = d.x[r];
        a.codes[r] = static_cast<uint8_t*>(d.codes[r]);
        a.scales[r] = d.scales[r];
    }
    a.n = d.n;
    a.k = d.k;
    a.ldx = d.ldx;
    a.ldc = d.ldc;
    a.lds = d.lds;
    a.half = d.half;
    a.groups = static_cast<int>(fp8_groups(d.k));
    cudaError_t e;
    if (d.weight) {
        a.blocks_half = static_cast<int>(fp8_groups(d.half));
        const int64_t blocks = d.half > 0 ? a.blocks_half + fp8_groups(d.n - d.half) : fp8_groups(d.n);
        if (blocks > 65535) return TP_ERR_UNSUPPORTED;
        const dim3 grid(static_cast<unsigned>(a.groups), static_cast<unsigned>(blocks), static_cast<unsigned>(d.t));
        e = d.in_f32 ? launch_pdl(fp8_quant_weight_kernel<true>, grid, dim3(kQuantThreads), 0, stream, a)
                     : launch_pdl(fp8_quant_weight_kernel<false>, grid, dim3(kQuantThreads), 0, stream, a);
    } else {
        const int64_t per = kQuantThreads / 16 * kQuantUnits;
        const int64_t blocks = (d.n * a.groups + per - 1) / per;
        if (blocks > INT32_MAX) return TP_ERR_UNSUPPORTED;
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(d.t), 1);
        e = d.in_f32 ? launch_pdl(fp8_quant_rows_kernel<true>, grid, dim3(kQuantThreads), 0, stream, a)
                     : launch_pdl(fp8_quant_rows_kernel<false>, grid, dim3(kQuantThreads), 0, stream, a);
    }
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

// ------------------------------------------------------------------ norm
//
// One thread block per row, which stays in its registers: the t partials are
// folded in fp32 in the reduce-scatter's order, the residual is added (and
// stored, rounded once), the squares are summed over the block, and the
// normed values go from fp32 to 8 bits without a rounding between.  Eight
// elements a thread and vector, so that a group is a half warp's.
struct Fp8NormArgs {
    const void* p[TP_MAX_SHARDS];
    const uint16_t* residual;
    const uint16_t* weight;
    uint16_t* residual_out;
    uint8_t* codes;
    float* scales;
    int64_t n, h, rows_per, ldc, lds;
    float eps;
    int t, ring;
};

template <bool F32, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) fp8_norm_kernel(const __grid_constant__ Fp8NormArgs a) {
    __shared__ float warp_sums[THREADS / 32];
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int64_t row = blockIdx.x;
    const int owner = static_cast<int>(row / a.rows_per);
    const int start = a.ring ? (owner + 1) % a.t : 0;
    const int64_t base = row * a.h;
    float x[VPT][8];
    Vec8<false> res[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t col = (static_cast<int64_t>(v) * THREADS + threadIdx.x) * 8;
        if (a.residual != nullptr && col < a.h)
            res[v].load(a.residual, base + col);
        else
            res[v].zero();
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t col = (static_cast<int64_t>(v) * THREADS + threadIdx.x) * 8;
        Vec8<F32> q[TP_MAX_SHARDS];
#pragma unroll
        for (int j = 0; j < TP_MAX_SHARDS; ++j) {
            if (j < a.t && col < a.h) {
                int r = start + j;
                if (r >= a.t) r -= a.t;
                q[j].load(a.p[r], base + col);
            } else {
                q[j].zero();
            }
        }
        q[0].get(x[v]);
#pragma unroll
        for (int j = 1; j < TP_MAX_SHARDS; ++j) {
            if (j < a.t) {
                float y[8];
                q[j].get(y);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[v][i] += y[i];
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (a.residual != nullptr) {
            float y[8];
            res[v].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[v][i] = y[i] + x[v][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[v][i] * x[v][i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = ss;
    __syncthreads();
    float tot = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) tot += warp_sums[w];
    const float rstd = rsqrtf(tot / static_cast<float>(a.h) + a.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t col = (static_cast<int64_t>(v) * THREADS + threadIdx.x) * 8;
        const bool in = col < a.h;
        if (in && a.residual_out != nullptr)
            *reinterpret_cast<uint4*>(a.residual_out + base + col) =
                make_uint4(pack_bf16x2(x[v][0], x[v][1]), pack_bf16x2(x[v][2], x[v][3]), pack_bf16x2(x[v][4], x[v][5]),
                           pack_bf16x2(x[v][6], x[v][7]));
        float w[8];
        Vec8<false> q;
        if (in)
            q.q[0] = *reinterpret_cast<const uint4*>(a.weight + col);
        else
            q.zero();
        q.get(w);
        // beyond the row: exact zeros, whatever the row's scale is
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = in ? x[v][i] * rstd * w[i] : 0.0f;
        const float s = fp8_scale(max16(amax8(w)));
        if (in) {
            *reinterpret_cast<uint2*>(a.codes + row * a.ldc + col) = fp8_codes8(w, s);
            if ((threadIdx.x & 15) == 0) a.scales[(col / kFp8Group) * a.lds + row] = s;
        }
    }
}

template <bool F32>
static cudaError_t launch_norm_sized(const Fp8NormArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.n));
    const int64_t vecs = (a.h + 7) / 8;
    if (vecs <= 128) return launch_pdl(fp8_norm_kernel<F32, 1, 128>, grid, dim3(128), 0, stream, a);
    if (vecs <= 256) return launch_pdl(fp8_norm_kernel<F32, 1, 256>, grid, dim3(256), 0, stream, a);
    if (vecs <= 512) return launch_pdl(fp8_norm_kernel<F32, 2, 256>, grid, dim3(256), 0, stream, a);
    if (vecs <= 1024) return launch_pdl(fp8_norm_kernel<F32, 2, 512>, grid, dim3(512), 0, stream, a);
    if (vecs <= 2048) return launch_pdl(fp8_norm_kernel<F32, 4, 512>, grid, dim3(512), 0, stream, a);
    return launch_pdl(fp8_norm_kernel<F32, 4, 1024>, grid, dim3(1024), 0, stream, a);
}

tp_status launch_fp8_norm(const Fp8NormDesc& d, cudaStream_t stream) {
    if (d.n == 0) return TP_OK;
    Fp8NormArgs a = {};
    for (int r = 0; r < d.t; ++r) a.p[r] = d.p[r];
    a.residual = static_cast<const uint16_t*>(d.residual);
    a.weight = static_cast<const uint16_t*>(d.weight);
    a.residual_out = static_cast<uint16_t*>(d.residual_out);
    a.codes = static_cast<uint8_t*>(d.codes);
    a.scales = d.scales;
    a.n = d.n;
    a.h = d.h;
    a.rows_per = (d.n + d.t - 1) / d.t;
    a.ldc = d.ldc;
    a.lds = d.lds;
    a.eps = d.eps;
    a.t = d.t;
    a.ring = d.ring;
    const cudaError_t e = d.in_bf16 ? launch_norm_sized<false>(a, stream) : launch_norm_sized<true>(a, stream);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace tpk

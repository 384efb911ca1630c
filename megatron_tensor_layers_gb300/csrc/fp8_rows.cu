// Rows and weights brought to 8 bits (e4m3 codes, one fp32 scale for each
// group of 128 columns of a row or each 128 x 128 block of a weight), and the
// norm between two layers with its rows in 8 bits.
//
//   scale = max(amax of the group, 2^-100) / 448,  code = e4m3(x / scale)
//
// The quantisers round every operation to fp32, so their codes and scales are those of the
// same formulas anywhere.  The norm's values take the hardware's reciprocal root (2 ulp) and two
// products on the way: within 6 units of 2^-24 beside the sum of squares' (a root, a division and a product: 3), most of which a
// group's scale shares (a rounded root and a product rounded once took 1 us more for 8192 rows and changed no code).  A group with a NaN or an infinity stands for NaN
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
    int blocks_half;     // weight: blocks of the first part's rows
};

// ------------------------------------------------------------------ rows
//
// A thread has eight columns of ROWS consecutive rows, whose loads it issues
// before it uses the first; sixteen neighbouring lanes hold a group.  Blocks are
// as wide as the rows up to 1024 columns.  Four matrices of 8192 x 2048: 32.1 us, 6.3
// TB/s (quotients with a second correction 32.6 us, the largest magnitude taken
// from fp32 values 34.2 us, values scaled and negated one by one 38 us).
constexpr int kRowThreads = 128;

template <bool F32, int ROWS>
__global__ void __launch_bounds__(kRowThreads) fp8_quant_rows_kernel(const __grid_constant__ Fp8QuantArgs a) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
    const int r = blockIdx.z;
    const int64_t col = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * 8;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS;
    const int rows = col < a.k ? static_cast<int>(min(static_cast<int64_t>(ROWS), a.n - row0)) : 0;   // of this thread's columns
    const char* from = static_cast<const char*>(a.x[r]) + (row0 * a.ldx + col) * (F32 ? 4 : 2);
    Vec8<F32> v[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        if (u < rows)
            v[u].load(from, 0);
        else
            v[u].zero();
        from += a.ldx * (F32 ? 4 : 2);
    }
    uint8_t* to = a.codes[r] + row0 * a.ldc + col;
    float* scale = a.scales[r] + (col / kFp8Group) * a.lds + row0;
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        f32x2 x[4];
        uint32_t code[2];
        const float s = fp8_scale(max16(v[u].amax()));
        v[u].negated(x);
        fp8_codes(x, s, code);
        if (u < rows) {
            *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
            if ((threadIdx.x & 15) == 0) scale[u] = s;
        }
        to += a.ldc;
    }
}

// ------------------------------------------------------------------ weights
//
// One thread block per 128 x 128 block, held in registers between its largest
// value and its codes.  What it takes beside the memory is arithmetic, which other
// thread blocks' loads cover: 14336 x 8192 with four an SM 52.7 us, 6.7 TB/s (with
// quotients of a second correction 55 us, three an SM 61, five 72, two or three of
// 512 threads 76 and 65).
constexpr int kQuantThreads = 256;
constexpr int kWeightRowsPerPass = kQuantThreads / 16;
constexpr int kWeightPasses = kFp8Group / kWeightRowsPerPass;

template <bool F32>
__global__ void __launch_bounds__(kQuantThreads, F32 ? 2 : 4) fp8_quant_weight_kernel(const __grid_constant__ Fp8QuantArgs a) {
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
    const int64_t first = row0 + (threadIdx.x >> 4);     // this thread's rows: every 16th from here
    const int64_t left = col < a.k ? min(static_cast<int64_t>(kFp8Group), row_end - first) : 0;
    const int rows = static_cast<int>((left + kWeightRowsPerPass - 1) / kWeightRowsPerPass);
    const char* from = static_cast<const char*>(a.x[r]) + (first * a.ldx + col) * (F32 ? 4 : 2);
    Vec8<F32> v[kWeightPasses];
#pragma unroll
    for (int i = 0; i < kWeightPasses; ++i) {
        if (i < rows)
            v[i].load(from, 0);
        else
            v[i].zero();
        from += a.ldx * (kWeightRowsPerPass * (F32 ? 4 : 2));
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kWeightPasses; ++i) m = max_nan(m, v[i].amax());
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
    m = max16(m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = max_nan(m, warp_max[w]);
    const float s = fp8_scale(m);
    uint8_t* to = a.codes[r] + first * a.ldc + col;
#pragma unroll
    for (int i = 0; i < kWeightPasses; ++i) {
        f32x2 x[4];
        uint32_t code[2];
        v[i].negated(x);
        fp8_codes(x, s, code);
        if (i < rows) *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
        to += a.ldc * kWeightRowsPerPass;
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
    cudaError_t e;
    if (d.weight) {
        a.blocks_half = static_cast<int>(fp8_groups(d.half));
        const int64_t blocks = d.half > 0 ? a.blocks_half + fp8_groups(d.n - d.half) : fp8_groups(d.n);
        if (blocks > 65535) return TP_ERR_UNSUPPORTED;
        const dim3 grid(static_cast<unsigned>(fp8_groups(d.k)), static_cast<unsigned>(blocks), static_cast<unsigned>(d.t));
        e = d.in_f32 ? launch_pdl(fp8_quant_weight_kernel<true>, grid, dim3(kQuantThreads), 0, stream, a)
                     : launch_pdl(fp8_quant_weight_kernel<false>, grid, dim3(kQuantThreads), 0, stream, a);
    } else {
        const int64_t vecs = d.k / 8;
        const int threads = static_cast<int>(std::min<int64_t>(kRowThreads, (vecs + 31) / 32 * 32));
        const int64_t across = (vecs + threads - 1) / threads;
        if (across > 65535) return TP_ERR_UNSUPPORTED;
        // four rows a thread where that still leaves every SM several blocks
        const bool many = across * d.t * ((d.n + 3) / 4) >= 4 * std::max(1, device_sms());
        const int rows = many ? 4 : 1;
        const dim3 grid(static_cast<unsigned>((d.n + rows - 1) / rows), static_cast<unsigned>(across), static_cast<unsigned>(d.t));
        const dim3 block(threads);
        if (many)
            e = d.in_f32 ? launch_pdl(fp8_quant_rows_kernel<true, 4>, grid, block, 0, stream, a)
                         : launch_pdl(fp8_quant_rows_kernel<false, 4>, grid, block, 0, stream, a);
        else
            e = d.in_f32 ? launch_pdl(fp8_quant_rows_kernel<true, 1>, grid, block, 0, stream, a)
                         : launch_pdl(fp8_quant_rows_kernel<false, 1>, grid, block, 0, stream, a);
    }
    return e == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

// ------------------------------------------------------------------ norm
//
// One thread block per row, which stays in its registers (from 16385 columns on the
// 64 registers a thread do not hold the loads in flight too, and some spill): the t partials are
// folded in fp32 in the reduce-scatter's order, the residual is added (and
// stored, rounded once), the squares are summed over the block, and the
// normed values go from fp32 to 8 bits without a rounding between.  Eight
// elements a thread and vector, so that a group is a half warp's.  8192 rows of
// 8192 from four bf16 shards: 136 us, 6.4 TB/s; 2048 rows of 16384 and 32768 96 and
// 179 us, 4.6 and 4.9 TB/s, of 32768 from eight shards 456 us, 3.1.
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

template <bool F32, int MAXT, int VPT, int THREADS>
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
    // up to eight 16-byte loads of the shards are issued before the first vector is folded (8192 rows of 8192, four bf16
    // shards: 136 us with eight, 165 with the compiler's order; sixteen cost occupancy, 152)
    constexpr int LOADS = MAXT * (F32 ? 2 : 1);
    constexpr int FRONT = LOADS >= 8 ? 1 : (8 / LOADS < VPT ? 8 / LOADS : VPT);
#pragma unroll
    for (int v0 = 0; v0 < VPT; v0 += FRONT) {
        Vec8<F32> q[FRONT][MAXT];
#pragma unroll
        for (int u = 0; u < FRONT; ++u) {
            const int64_t col = (static_cast<int64_t>(v0 + u) * THREADS + threadIdx.x) * 8;
#pragma unroll
            for (int j = 0; j < MAXT; ++j) {
                if ((j == 0 || j < a.t) && col < a.h) {
                    int r = start + j;
                    if (r >= a.t) r -= a.t;
                    q[u][j].load(a.p[MAXT == 1 ? 0 : r], base + col);
                } else {
                    q[u][j].zero();
                }
            }
            if (a.residual != nullptr && col < a.h)
                res[v0 + u].load(a.residual, base + col);
            else
                res[v0 + u].zero();
        }
#pragma unroll
        for (int u = 0; u < FRONT; ++u) {
            q[u][0].get(x[v0 + u]);
#pragma unroll
            for (int j = 1; j < MAXT; ++j) {
                if (j < a.t) {
                    float y[8];
                    q[u][j].get(y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[v0 + u][i] += y[i];
                }
            }
        }
    }
    float sq[4] = {};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (a.residual != nullptr) {
            float y[8];
            res[v].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[v][i] = y[i] + x[v][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[i & 3] += x[v][i] * x[v][i];
    }
    float ss = (sq[0] + sq[1]) + (sq[2] + sq[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = ss;
    __syncthreads();
    float part[THREADS / 32];                            // in pairs: an addition's rounding is not carried along
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) part[w] = warp_sums[w];
#pragma unroll
    for (int d = THREADS / 64; d > 0; d >>= 1)
#pragma unroll
        for (int w = 0; w < d; ++w) part[w] += part[w + d];
    const float nrstd = -rsqrtf(part[0] / static_cast<float>(a.h) + a.eps);
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
        // the normed values, negated; beyond the row exact zeros, whatever the row's scale is
        f32x2 y[4];
        uint32_t code[2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = in ? pack2(x[v][2 * i] * nrstd * w[2 * i], x[v][2 * i + 1] * nrstd * w[2 * i + 1]) : 0;
        const float s = fp8_scale(max16(amax_pairs(y)));
        fp8_codes(y, s, code);
        if (in) {
            *reinterpret_cast<uint2*>(a.codes + row * a.ldc + col) = make_uint2(code[0], code[1]);
            if ((threadIdx.x & 15) == 0) a.scales[(col / kFp8Group) * a.lds + row] = s;
        }
    }
}

template <bool F32, int MAXT, int VPT, int THREADS>
static cudaError_t launch_norm_cfg(const Fp8NormArgs& a, cudaStream_t stream) {
    return launch_pdl(fp8_norm_kernel<F32, MAXT, VPT, THREADS>, dim3(static_cast<unsigned>(a.n)), dim3(THREADS), 0, stream, a);
}

// Rows of up to 8192 columns: with no more rows than SMs one vector a thread (one row of 8192: 3.2 us instead of 3.7 with
// two), else two vectors and half the threads (8192 rows: 136 us instead of 139, and 59 instead of 94 with 8 shards).
template <bool F32, int MAXT>
static cudaError_t launch_norm_sized(const Fp8NormArgs& a, cudaStream_t stream) {
    const int64_t vecs = (a.h + 7) / 8;
    const bool few = a.n <= device_sms();
    if (vecs <= 128) return launch_norm_cfg<F32, MAXT, 1, 128>(a, stream);
    if (vecs <= 256) return launch_norm_cfg<F32, MAXT, 1, 256>(a, stream);
    if (vecs <= 512) return few ? launch_norm_cfg<F32, MAXT, 1, 512>(a, stream) : launch_norm_cfg<F32, MAXT, 2, 256>(a, stream);
    if (vecs <= 1024) return few ? launch_norm_cfg<F32, MAXT, 1, 1024>(a, stream) : launch_norm_cfg<F32, MAXT, 2, 512>(a, stream);
    if (vecs <= 2048) return launch_norm_cfg<F32, MAXT, 4, 512>(a, stream);
    return launch_norm_cfg<F32, MAXT, 4, 1024>(a, stream);
}

template <bool F32>
static cudaError_t launch_norm_typed(const Fp8NormArgs& a, cudaStream_t stream) {
    if (a.t == 1) return launch_norm_sized<F32, 1>(a, stream);
    if (a.t == 2) return launch_norm_sized<F32, 2>(a, stream);
    if (a.t <= 4) return launch_norm_sized<F32, 4>(a, stream);
    return launch_norm_sized<F32, 8>(a, stream);
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
    const cudaError_t e = d.in_bf16 ? launch_norm_typed<false>(a, stream) : launch_norm_typed<true>(a, stream);
    return e == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace tpk

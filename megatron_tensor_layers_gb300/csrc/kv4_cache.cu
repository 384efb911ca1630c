// Writing to and reading from the paged 4-bit KV cache.
//
// Both kernels are elementwise over rows of head_dim elements and bound by the
// memory traffic of large calls (append: 2 bytes in and about 0.53 out per
// element) and by the chain of dependent loads (row -> sequence -> page) of
// small ones.  HD / 8 lanes hold one row, eight elements each: a 16-byte load,
// a 4-byte store of eight codes.
#include "kv4.cuh"

namespace tpk {
namespace {

constexpr int kThreads = 256;

// min, max and "all finite" of a row held by LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ void row_range(const float (&x)[8], float& lo, float& hi, bool& finite) {
    lo = hi = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad |= !(fabsf(x[i]) <= 3.402823466e38f);
    }
    uint32_t b = bad;
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
        b |= __shfl_xor_sync(0xffffffffu, b, m);
    }
    finite = b == 0;
}

// One warp per (row, rank, group of sub-rows); a sub-row is one kv head's key or value.
template <int HD>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(KvAppendDesc d) {
    using B = KvBlock<HD>;
    constexpr int LANES = HD / 8, SUB = 32 / LANES;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int subs = 2 * d.pools.kv_heads, groups = (subs + SUB - 1) / SUB;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t per_row = static_cast<int64_t>(d.pools.t) * groups;
    if (warp >= d.seqs.n * per_row) return;
    const int row = static_cast<int>(warp / per_row);
    const int rest = static_cast<int>(warp - row * per_row);
    const int r = rest / groups, sub = (rest - r * groups) * SUB + lane / LANES;
    const int part = lane % LANES;
    const bool active = sub < subs;
    const int head = active ? sub >> 1 : 0;
    const bool val = sub & 1;

    uint4 raw = make_uint4(0, 0, 0, 0);
    if (active) {
        const uint16_t* src = static_cast<const uint16_t*>(val ? d.v[r] : d.k[r]) +
                              row * (val ? d.ldv : d.ldk) + head * HD + part * 8;
        raw = __ldg(reinterpret_cast<const uint4*>(src));
    }
    int seq, pos;
    const bool found = row_place(d.seqs, row, lane, seq, pos);
    if (!found) raise_status(d.seqs.status, TP_ERR_INVALID_ARG);
    if (!found || pos < 0) return;
    const int64_t off = kv_block_offset(d.seqs.table + seq * d.seqs.max_blocks, d.seqs.max_blocks, d.pools.pages,
                                        d.pools.page_shift, d.pools.kv_heads, head, pos / kKvBlock, B::BYTES);
    if (off < 0) {
        raise_status(d.seqs.status, TP_ERR_INVALID_ARG);
        return;                                   // page and position are the same for the whole warp
    }
    float x[8];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    float lo, hi;
    bool finite;
    row_range<LANES>(x, lo, hi, finite);
    // fp32 throughout; the base is a bf16 already (an element of the row), the step is rounded to bf16
    // once and the codes are taken with the rounded step, so that they are the nearest to it.
    lo = __fadd_rn(lo, 0.0f);                     // -0 becomes +0
    const float range = __fadd_rn(__fsub_rn(hi, lo), 0.0f);   // a step is never -0: attention compares its bits
    finite = finite && range <= 3.402823466e38f;
    const uint16_t step16 = finite ? f32_to_bf16(__fmul_rn(range, 1.0f / 15.0f)) : 0;
    const float step = bf16_to_f32(step16);
    uint32_t code = 0;
    if (step > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = rintf(__fdiv_rn(__fsub_rn(x[i], lo), step));
            code |= static_cast<uint32_t>(fminf(fmaxf(u, 0.0f), 15.0f)) << (4 * i);
        }
    }
    if (!active) return;
    const int slot = pos % kKvBlock;
    uint8_t* block = d.pools.pool[r] + off;
    *reinterpret_cast<uint32_t*>(block + (val ? B::VALS : B::KEYS) + slot * B::ROW + part * 4) = code;
    if (part == 0) {
        const uint32_t base16 = finite ? __float_as_uint(lo) >> 16 : 0x7fc0u;
        *reinterpret_cast<uint32_t*>(block + (val ? B::VPAIR : B::KPAIR) + slot * 4) = step16 | (base16 << 16);
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(KvLoadDesc d) {
    using B = KvBlock<HD>;
    constexpr int LANES = HD / 8, SUB = 32 / LANES;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int subs = 2 * d.pools.kv_heads, groups = (subs + SUB - 1) / SUB;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t per_row = static_cast<int64_t>(d.pools.t) * groups;
    if (warp >= d.seqs.n * per_row) return;
    const int row = static_cast<int>(warp / per_row);
    const int rest = static_cast<int>(warp - row * per_row);
    const int r = rest / groups, sub = (rest - r * groups) * SUB + lane / LANES;
    const int part = lane % LANES;
    const int head = sub >> 1;
    const bool val = sub & 1;

    int seq, pos;
    const bool found = row_place(d.seqs, row, lane, seq, pos);
    if (!found) raise_status(d.seqs.status, TP_ERR_INVALID_ARG);
    if (sub >= subs || !(val ? d.with_v : d.with_k)) return;
    int64_t off = -1;
    if (found && pos >= 0) {
        off = kv_block_offset(d.seqs.table + seq * d.seqs.max_blocks, d.seqs.max_blocks, d.pools.pages,
                              d.pools.page_shift, d.pools.kv_heads, head, pos / kKvBlock, B::BYTES);
        if (off < 0) raise_status(d.seqs.status, TP_ERR_INVALID_ARG);
    }
    float y[8] = {};
    if (off >= 0) {
        const int slot = pos % kKvBlock;
        const uint8_t* block = d.pools.pool[r] + off;
        const uint32_t code =
            *reinterpret_cast<const uint32_t*>(block + (val ? B::VALS : B::KEYS) + slot * B::ROW + part * 4);
        const uint32_t pair = *reinterpret_cast<const uint32_t*>(block + (val ? B::VPAIR : B::KPAIR) + slot * 4);
        const float step = __uint_as_float(pair << 16), base = __uint_as_float(pair & 0xffff0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(step, static_cast<float>((code >> (4 * i)) & 15u), base);
    }
    const int64_t at = row * (val ? d.ldv : d.ldk) + head * HD + part * 8;
    void* out = val ? d.v[r] : d.k[r];
    if (d.out_f32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        p[0] = make_float4(y[0], y[1], y[2], y[3]);
        p[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
}

int64_t warps_of(int64_t n, const KvPools& p, int head_dim) {
    const int sub = 32 / (head_dim / 8);
    return n * p.t * ((2 * p.kv_heads + sub - 1) / sub);
}

template <typename Desc, typename K128, typename K64>
tp_status launch_rows(const Desc& d, K128 k128, K64 k64, cudaStream_t stream) {
    const int64_t warps = warps_of(d.seqs.n, d.pools, d.head_dim);
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return TP_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    const cudaError_t e = d.head_dim == 128 ? launch_pdl(k128, grid, dim3(kThreads), 0, stream, d)
                                            : launch_pdl(k64, grid, dim3(kThreads), 0, stream, d);
    return e == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace

tp_status launch_kv4_append(const KvAppendDesc& d, cudaStream_t stream) {
    return launch_rows(d, kv4_append_kernel<128>, kv4_append_kernel<64>, stream);
}

tp_status launch_kv4_load(const KvLoadDesc& d, cudaStream_t stream) {
    return launch_rows(d, kv4_load_kernel<128>, kv4_load_kernel<64>, stream);
}

}  // namespace tpk

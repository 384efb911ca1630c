// Writing to and reading from the paged 4-bit KV cache.
//
// Both kernels are elementwise over rows of head_dim elements.  Large calls are
// bound by memory traffic (append: 2 bytes in and about 0.53 out per element) and
// by the instructions of an element: 8192 rows of 8 heads of 128, keys and values,
// append 23 us with inputs that are not in L2 and 18 with such that are (three
// quarters of the issue slots), load 11 us.  Small ones are bound by the chain of dependent loads (row ->
// sequence -> page): append and load of 64 rows 5.9 us.  HD / 8
// lanes hold one sub-row (a kv head's key or value of a row), eight elements
// each: a 16-byte load, a 4-byte store of eight codes.
//
// A warp takes kRows rows of one group of sub-rows (those that its 32 lanes
// hold).  Lane r looks up the place of row r, so that one chain of loads serves
// all of them, and the rows' data are on their way before it.  Few rows to
// append take one a warp, so that they spread over the GPU.  Half as many lanes
// a sub-row, with sixteen elements each, take fewer instructions but leave fewer
// loads in flight: 43 us where append and load of 8192 rows take 36.
#include "kv4.cuh"

namespace tpk {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Smallest and largest of a row of bf16 held by LANES neighbouring lanes, eight elements each; NaN when one is.
template <int LANES>
__device__ __forceinline__ void row_range(const uint4& w, float& lo, float& hi) {
    uint32_t a = min2(min2(w.x, w.y), min2(w.z, w.w)), b = max2(max2(w.x, w.y), max2(w.z, w.w));
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) {
        a = min2(a, __shfl_xor_sync(0xffffffffu, a, m));
        b = max2(b, __shfl_xor_sync(0xffffffffu, b, m));
    }
    a = min2(a, a >> 16);                        // the lower half; the upper is not looked at
    b = max2(b, b >> 16);
    lo = __uint_as_float(a << 16);
    hi = __uint_as_float(b << 16);
}

__device__ __forceinline__ void store8(float* p, const float (&y)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(y[0]), "f"(y[1]), "f"(y[2]),
                 "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                 : "memory");
}

// The place in its rank's pool of row `row` (offset of its block for kv head 0, and its slot), by one lane:
// block -1 when it is at a negative position, -2 when it has no place.
struct RowAt {
    int64_t block;
    int slot;
};
template <int HD>
__device__ __forceinline__ RowAt row_at(const KvSeqs& q, const KvPools& p, int row) {
    int seq = row, pos;
    if (q.cu_rows == nullptr) {
        pos = max(q.lens[row], 0) - 1;
    } else {
        int lo = 0, hi = q.nseq;                 // the last sequence that begins at or before the row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (q.cu_rows[mid] <= row)
                lo = mid;
            else
                hi = mid;
        }
        const int a = q.cu_rows[lo], b = q.cu_rows[lo + 1];
        if (a < 0 || a > row || row >= b || b > q.n) return {-2, 0};
        // 64 bits: a length of any value minus any row count stays in range
        const int64_t at = static_cast<int64_t>(q.lens[lo]) - (static_cast<int64_t>(b) - row);
        seq = lo;
        pos = at < 0 ? -1 : static_cast<int>(at);
    }
    if (pos < 0) return {-1, 0};
    const int64_t off = kv_block_offset(q.table + seq * q.max_blocks, q.max_blocks, p.pages, p.page_shift, p.kv_heads, 0,
                                        pos / kKvBlock, KvBlock<HD>::BYTES);
    return {off < 0 ? -2 : off, pos % kKvBlock};
}

// What a warp works on: rows row0 .. of rank r, and for each lane its sub-row.
template <int HD, int ROWS>
struct Task {
    static constexpr int LANES = HD / 8, SUB = 32 / LANES;
    int row0, rows, r, sub, part, head;
    bool val, active, any;
    __device__ __forceinline__ Task(const KvSeqs& q, const KvPools& p) {
        const int lane = threadIdx.x & 31;
        const int subs = 2 * p.kv_heads, groups = (subs + SUB - 1) / SUB;
        const int per = p.t * groups;
        const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
        const int64_t set = quotient(warp, per);
        const int rest = static_cast<int>(warp - set * per);
        any = set * ROWS < q.n;
        row0 = static_cast<int>(set) * ROWS;
        rows = min(ROWS, q.n - row0);
        r = rest / groups;
        sub = (rest - r * groups) * SUB + lane / LANES;
        part = lane % LANES;
        active = sub < subs;
        head = active ? sub >> 1 : 0;
        val = sub & 1;
    }
};

template <int HD, int ROWS>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ KvAppendDesc d) {
    using B = KvBlock<HD>;
    pdl_wait();
    pdl_trigger();
    const Task<HD, ROWS> w(d.seqs, d.pools);
    if (!w.any) return;
    const int lane = threadIdx.x & 31;
    const int64_t ld = w.val ? d.ldv : d.ldk;
    const uint16_t* src = static_cast<const uint16_t*>(w.val ? d.v[w.r] : d.k[w.r]) + w.row0 * ld + w.head * HD + w.part * 8;
    uint4 raw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        raw[i] = w.active && i < w.rows ? __ldg(reinterpret_cast<const uint4*>(src + i * ld)) : make_uint4(0, 0, 0, 0);
    RowAt at{-1, 0};
    if (lane < w.rows) at = row_at<HD>(d.seqs, d.pools, w.row0 + lane);
    if (at.block == -2) raise_status(d.seqs.status, TP_ERR_INVALID_ARG);
    uint8_t* pool = d.pools.pool[w.r] + (static_cast<int64_t>(w.head) << d.pools.page_shift) * B::BYTES;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t block = __shfl_sync(0xffffffffu, at.block, i);
        const int slot = __shfl_sync(0xffffffffu, at.slot, i);
        if (block < 0) continue;                  // the same for the whole warp
        float lo, hi;
        row_range<Task<HD, ROWS>::LANES>(raw[i], lo, hi);
        // fp32 throughout; the base is a bf16 already (an element of the row), the step is rounded to bf16
        // once and the codes are taken with the rounded step, so that they are the nearest to it.
        lo = __fadd_rn(lo, 0.0f);                 // -0 becomes +0
        const float range = __fadd_rn(__fsub_rn(hi, lo), 0.0f);   // a step is never -0: attention compares its bits
        const bool finite = range <= 3.402823466e38f;             // false for NaN: one in the row, or inf - inf
        const uint16_t step16 = finite ? f32_to_bf16(__fmul_rn(range, 1.0f / 15.0f)) : 0;
        const float step = bf16_to_f32(step16);
        uint32_t code = 0;
        if (step > 0.0f) {
            const uint32_t word[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = __fsub_rn(__uint_as_float(word[j] << 16), lo);
                x[2 * j + 1] = __fsub_rn(__uint_as_float(word[j] & 0xffff0000u), lo);
            }
            // A quotient of at most 15.1 by the reciprocal is off by 15.1 2^-24 < 2^-20, and so is the definition's
            // rounded one: only within 2^-18 of a border between two codes (of 1 warp in 500), or with a step whose
            // rounding (below the normal numbers) or reciprocal is not that good, does the definition's division
            // decide.  Adding 1.5 2^23 leaves the nearest whole number, ties to even, in the low bits; its own bits
            // come off the packed word at the end.
            const float inv = __frcp_rn(step);
            bool near = !(step > 1e-30f);
            uint32_t fast = 0;
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const float t = fmaf(x[j], inv, 12582912.0f);
                near |= fabsf(fmaf(x[j], inv, -__fsub_rn(t, 12582912.0f))) > 0.5f - 0x1p-18f;
                fast = fast * 16 + __float_as_uint(t);
            }
            code = fast - (0x4b400000u + 0xb4000000u + 0x40000000u);
            if (near) {
                code = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    code |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(x[j], step)), 0.0f), 15.0f)) << (4 * j);
            }
        }
        if (!w.active) continue;
        uint8_t* rec = pool + block;
        *reinterpret_cast<uint32_t*>(rec + (w.val ? B::VALS : B::KEYS) + slot * B::ROW + w.part * 4) = code;
        if (w.part == 0) {
            const uint32_t base16 = finite ? __float_as_uint(lo) >> 16 : 0x7fc0u;
            *reinterpret_cast<uint32_t*>(rec + (w.val ? B::VPAIR : B::KPAIR) + slot * 4) = step16 | (base16 << 16);
        }
    }
}

template <int HD, int ROWS>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const __grid_constant__ KvLoadDesc d) {
    using B = KvBlock<HD>;
    pdl_wait();
    pdl_trigger();
    const Task<HD, ROWS> w(d.seqs, d.pools);
    if (!w.any) return;
    const int lane = threadIdx.x & 31;
    RowAt at{-1, 0};
    if (lane < w.rows) at = row_at<HD>(d.seqs, d.pools, w.row0 + lane);
    if (at.block == -2) raise_status(d.seqs.status, TP_ERR_INVALID_ARG);
    const bool wanted = w.active && (w.val ? d.with_v : d.with_k);
    const uint8_t* pool = d.pools.pool[w.r] + (static_cast<int64_t>(w.head) << d.pools.page_shift) * B::BYTES;
    uint32_t code[ROWS], pair[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t block = __shfl_sync(0xffffffffu, at.block, i);
        const int slot = __shfl_sync(0xffffffffu, at.slot, i);
        code[i] = pair[i] = 0;
        if (block >= 0 && wanted) {
            const uint8_t* rec = pool + block;
            code[i] = *reinterpret_cast<const uint32_t*>(rec + (w.val ? B::VALS : B::KEYS) + slot * B::ROW + w.part * 4);
            pair[i] = *reinterpret_cast<const uint32_t*>(rec + (w.val ? B::VPAIR : B::KPAIR) + slot * 4);
        }
    }
    if (!wanted) return;
    const int64_t ld = w.val ? d.ldv : d.ldk;
    const int64_t out0 = w.row0 * ld + w.head * HD + w.part * 8;
    void* out = w.val ? d.v[w.r] : d.k[w.r];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (i >= w.rows) break;
        const float step = __uint_as_float(pair[i] << 16), base = __uint_as_float(pair[i] & 0xffff0000u);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)          // 2^23 + u in the low bits: no conversion, of which there are few a cycle
            y[j] = fmaf(step, __uint_as_float(((code[i] >> (4 * j)) & 15u) | 0x4b000000u) - 8388608.0f, base);
        if (d.out_f32) {
            float* p = static_cast<float*>(out) + out0 + i * ld;
            if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {      // whole sectors
                store8(p, y);
            } else {
                reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + out0 + i * ld) =
                make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
    }
}

constexpr int kRows = 4;

// `rows` rows a warp.
template <typename Desc, typename Kern>
tp_status launch_rows(const Desc& d, Kern kern, int rows, int64_t per, cudaStream_t stream) {
    const int64_t warps = (d.seqs.n + rows - 1) / rows * per;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return TP_ERR_UNSUPPORTED;
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, d) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

// Warps that a group of rows takes: one for each 32 / (hd / 8) sub-rows of a rank.
int64_t warps_of_rows(int t, int kv_heads, int head_dim) {
    const int sub = 32 / (head_dim / 8);
    return static_cast<int64_t>(t) * ((2 * kv_heads + sub - 1) / sub);
}

// Four rows a warp where that leaves 32 warps for an SM, else one: with four and with one, 4 ranks of 2 heads of
// 128, 8192 rows take 18.0 and 25.4 us (108 warps), 2048 8.2 and 8.1 (27 warps), 256 4.9 and 3.7.
template <int HD>
tp_status append(const KvAppendDesc& d, cudaStream_t stream) {
    const int64_t per = warps_of_rows(d.pools.t, d.pools.kv_heads, HD);
    const int sms = device_sms();
    if (sms <= 0) return TP_ERR_CUDA;
    const bool few = (d.seqs.n + kRows - 1) / kRows * per < static_cast<int64_t>(sms) * 32;
    return few ? launch_rows(d, kv4_append_kernel<HD, 1>, 1, per, stream)
               : launch_rows(d, kv4_append_kernel<HD, kRows>, kRows, per, stream);
}

// Always four: 8192 rows take 10.8 us (20.5 with one a warp), 1024 3.9 (4.5), 256 and fewer the same 3.4.
template <int HD>
tp_status load(const KvLoadDesc& d, cudaStream_t stream) {
    return launch_rows(d, kv4_load_kernel<HD, kRows>, kRows, warps_of_rows(d.pools.t, d.pools.kv_heads, HD), stream);
}

}  // namespace

tp_status launch_kv4_append(const KvAppendDesc& d, cudaStream_t stream) {
    return d.head_dim == 128 ? append<128>(d, stream) : append<64>(d, stream);
}

tp_status launch_kv4_load(const KvLoadDesc& d, cudaStream_t stream) {
    return d.head_dim == 128 ? load<128>(d, stream) : load<64>(d, stream);
}

}  // namespace tpk

// Products of 8-bit rows and 8-bit weights on the 5th-generation tensor core:
//
//     y_ij = sum_g  s_x[g, i] * s_w[j / 128, g] * sum_{k in group g} x_ik w_jk
//
// with e4m3 codes x [n, K] and w [out, K], one fp32 scale for each row's group
// of 128 columns and each 128 x 128 block of the weight.  The codes' products
// are exact and the tensor core adds those of one group (one K block of 128)
// into a TMEM accumulator of its own; the epilogue warps read each block's
// accumulator, multiply it by the two scales' product and add it to fp32
// sums in their registers, so scales may be any fp32 numbers.
//
// Launches are programmatic (PDL): weights are loaded before the previous
// kernel's end only when that kernel belongs to the same call and writes none.
// Every wait is bounded (1 s) and reports TP_ERR_TIMEOUT.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "fp8.cuh"
#include "kernels.h"

namespace tpk {

struct Fp8GemmArgs {
    CUtensorMap mapX[TP_MAX_SHARDS];
    CUtensorMap mapW[TP_MAX_SHARDS];
    const float* xs[TP_MAX_SHARDS];
    const float* ws[TP_MAX_SHARDS];
    void* out[TP_MAX_SHARDS];
    float* os[TP_MAX_SHARDS];
    const uint16_t* bias[TP_MAX_SHARDS];
    int64_t ldxs, ldo, ldos;
    int M, N;             // tokens, output columns per group
    int k_blocks;         // K blocks of a segment (= the row pitch of a weight's scales)
    int segs, groups, x_per_group;
    int up_block;         // first block row of up in a gated weight's scales
    int m_tiles, n_tiles, total_tiles;
    int x_box_rows;       // rows of a token tile that a copy brings
    int out_kind;
    int split;            // CTAs (many rows: CTA pairs) of a cluster that share a tile's K blocks
    int band;             // many rows: row tiles of a raster band
    int weights_first;
    int* status;
};

// Instruction descriptor of tcgen05.mma kind::f8f6f4 with e4m3 A and B (format
// 0), f32 accumulator, both operands K-major.
__host__ __device__ constexpr uint32_t mma_idesc_e4m3(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Each thread of the warp reads 16 or 32 consecutive 32-bit columns of its own
// TMEM lane.  The values are there after tmem_wait on the same array, which
// the compiler sees as writing them, so that no use moves before it.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}
// An asm statement takes 30 operands: the arrays are named in four.
__device__ __forceinline__ void tmem_wait(float (&x)[32], float (&y)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
        asm volatile(""
                     : "+f"(x[i]), "+f"(x[i + 1]), "+f"(x[i + 2]), "+f"(x[i + 3]), "+f"(x[i + 4]), "+f"(x[i + 5]),
                       "+f"(x[i + 6]), "+f"(x[i + 7]), "+f"(x[i + 8]), "+f"(x[i + 9]), "+f"(x[i + 10]),
                       "+f"(x[i + 11]), "+f"(x[i + 12]), "+f"(x[i + 13]), "+f"(x[i + 14]), "+f"(x[i + 15]));
        asm volatile(""
                     : "+f"(y[i]), "+f"(y[i + 1]), "+f"(y[i + 2]), "+f"(y[i + 3]), "+f"(y[i + 4]), "+f"(y[i + 5]),
                       "+f"(y[i + 6]), "+f"(y[i + 7]), "+f"(y[i + 8]), "+f"(y[i + 9]), "+f"(y[i + 10]),
                       "+f"(y[i + 11]), "+f"(y[i + 12]), "+f"(y[i + 13]), "+f"(y[i + 14]), "+f"(y[i + 15]));
    }
}

// Asynchronous copies of one float to shared memory, in groups.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four neighbouring columns (lane * 4 of the warp's 128) of one row of a gated
// tile: act(gate) * up, stored, or brought to 8 bits with the row's group in
// the warp.
template <int ACT>
__device__ __forceinline__ void finish_gated(const Fp8GemmArgs& args, int g, int n, int64_t row, int lane,
                                             const float (&gate)[4], const float (&up)[4]) {
    const int col = n * 128 + lane * 4;
    const int nvalid = args.N - col;                     // this lane's columns inside the group
    const GateAct<ACT> act(args.out_kind == FP8_OUT_CODES);
    f32x2 v2[2] = {mul2(act(pack2(gate[0], gate[1])), pack2(up[0], up[1])), mul2(act(pack2(gate[2], gate[3])), pack2(up[2], up[3]))};
    if (args.out_kind == FP8_OUT_CODES) {
        float top = nvalid > 0 ? amax_pairs(v2) : 0.0f;  // N is a multiple of 16: all four or none
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float s = fp8_scale(top);
        uint32_t code[1];
        fp8_codes(v2, s, code);
        if (nvalid > 0)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(args.out[g]) + row * args.ldo + col) = code[0];
        if (lane == 0) args.os[g][static_cast<int64_t>(n) * args.ldos + row] = s;
    } else if (nvalid > 0) {
        float v[4];
        unpack2(v2[0], v[0], v[1]);
        unpack2(v2[1], v[2], v[3]);
        store_quad(args.out[g], args.ldo, args.out_kind == FP8_OUT_F32, row, col, min(4, nvalid), v);
    }
}

// ------------------------------------------------------- weights as the rows of the MMA
//
// Few tokens: the MMA's M = 128 rows are 128 output columns (a block row of
// the weight's scales) and its N columns are NT tokens, so that a K block's
// accumulator holds NT values a lane instead of 128 mostly unused rows.
// A cluster of `split` CTAs shares an output tile: CTA r runs K blocks
// [r KB / split, (r + 1) KB / split) and stages its sums in its shared memory,
// and the cluster's epilogue warps take one token each, add the CTAs' sums in
// rank order (over distributed shared memory) and store it; the 128 columns
// of a token's tile are one warp's, which for a gated tile is also the group
// of the 8-bit hidden row.
//
// Roles: warp 0 brings tiles (TMA), warp 1 multiplies, warp 2 brings scales,
// warps 3.. add up: of a gated tile four warps the gate's columns and four up's,
// of a plain one each warp all NT columns, or half of 128.
template <int NT, bool GLU>
struct FewCfg {
    static constexpr int W_BYTES = (GLU ? 2 : 1) * 128 * 128;
    static constexpr int X_BYTES = NT * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr bool ONE = NT > (GLU ? 32 : 64);          // CTAs per SM: one, else two
    static constexpr int BUDGET = (ONE ? 216 : 110) * 1024;    // of the ring
    static constexpr int STAGES = BUDGET / STAGE_BYTES;
    static constexpr int STAGING_BYTES = (GLU ? 2 : 1) * NT * 128 * 4;
    static constexpr int EPI_WARPS = (GLU || NT > 64) ? 8 : 4;
    static constexpr int NC = (!GLU && NT > 64) ? NT / 2 : NT; // columns of a warp
    static constexpr int ACC_COLS = NT * (GLU ? 2 : 1);        // TMEM columns of one K block
    static constexpr int TMEM_BUFS = (ONE ? 512 : 256) / ACC_COLS;
    // accumulators in turn; no more than stages, so that a block's start has one phase ahead of it at most
    static constexpr int BUFS = TMEM_BUFS >= 4 && STAGES >= 4 ? 4 : 2;
    static constexpr int TMEM_COLS = ACC_COLS * BUFS;
    static constexpr int THREADS = 96 + 32 * EPI_WARPS;
    static constexpr int NBARS = 2 * STAGES;
    static constexpr int AHEAD = 4;                            // K blocks ahead that scales are asked for
    static constexpr int SLOTS = AHEAD + STAGES + BUFS;
    // whether the scales' warp multiplies the tokens' scales with the weight blocks'; with 128 tokens of gate and up the warps
    // that use them do, for whose sums leave no registers for factors read ahead (100 tokens 102 us and 135)
    static constexpr bool FACTORED = !(GLU && NT == 128);
    static constexpr int FACTORS = (GLU && FACTORED ? 2 : 1) * NT;   // of a block: times gate's, and times up's
    static constexpr int SLOT_FLOATS = FACTORS + 4;            // ... and the weight blocks' scales
    static constexpr int SCALE_BYTES = SLOTS * SLOT_FLOATS * 4;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + SCALE_BYTES + NBARS * 8 + 16;
    static_assert(STAGES >= BUFS && TMEM_BUFS >= 2, "both pipelines need two slots");
    static_assert(STAGES * STAGE_BYTES >= STAGING_BYTES, "the sums are staged in the ring");
    static_assert(STAGE_BYTES % 1024 == 0 && W_BYTES % 1024 == 0, "swizzled tiles are 1024-byte aligned");
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS >= 32 && TMEM_COLS <= 512, "TMEM columns");
    static_assert(NT % 16 == 0 && NC % 16 == 0, "MMA N, and chunks of 16 columns");
    static_assert(SMEM_BYTES <= (ONE ? 227 : 113) * 1024, "shared memory");
};

template <int NT, int ACT>
__global__ void __launch_bounds__(FewCfg<NT, ACT != TP_ACT_NONE>::THREADS, FewCfg<NT, ACT != TP_ACT_NONE>::ONE ? 1 : 2)
    fp8_few_kernel(const __grid_constant__ Fp8GemmArgs args) {
    constexpr bool GLU = ACT != TP_ACT_NONE;
    using Cfg = FewCfg<NT, GLU>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    float* scales_ptr = reinterpret_cast<float*>(base_ptr + Cfg::STAGES * Cfg::STAGE_BYTES);
    constexpr int kBarOff = Cfg::STAGES * Cfg::STAGE_BYTES + Cfg::SCALE_BYTES;
    const uint32_t bar_base = base + kBarOff;
    // a stage's products may start: its tiles are there and the accumulator is free; they are done
    auto start_bar = [&](int s) { return bar_base + 8u * s; };
    auto done_bar = [&](int s) { return bar_base + 8u * (Cfg::STAGES + s); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + kBarOff + 8 * Cfg::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + kBarOff + 8 * Cfg::NBARS + 4);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // uniform to the compiler
    const int lane = threadIdx.x & 31;
    const int split = args.split;
    const int crank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    // tile: token tiles fastest, so that a weight's block is read by neighbours in time
    const int tile = static_cast<int>(blockIdx.x) / split;
    const int m = tile % args.m_tiles;
    const int n = (tile / args.m_tiles) % args.n_tiles;
    const int g = tile / (args.m_tiles * args.n_tiles);
    const int kb_all = args.k_blocks * args.segs;
    const int kb_lo = static_cast<int>(static_cast<int64_t>(crank) * kb_all / split);
    const int kb_hi = static_cast<int>(static_cast<int64_t>(crank + 1) * kb_all / split);
    const int token0 = m * NT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::STAGES; ++s) {
            mbar_init(start_bar(s), 1 + Cfg::EPI_WARPS);
            mbar_init(done_bar(s), 2);                   // the products, the scales
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<Cfg::TMEM_COLS>(smem_u32(tmem_slot));
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    bool aborted = false;

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        const uint32_t bytes = Cfg::W_BYTES + static_cast<uint32_t>(args.x_box_rows) * 128u;
        int seg = kb_lo / args.k_blocks, kb = kb_lo - seg * args.k_blocks;
        auto load_w = [&](int s, int seg, int kb) {
            const int wi = args.segs > 1 ? seg : g;
            const uint32_t sw = base + s * Cfg::STAGE_BYTES;
            mbar_arrive_expect_tx(start_bar(s), bytes);
            tma_load_2d(sw, &args.mapW[wi], start_bar(s), kb * 128, n * 128);
            if (GLU) tma_load_2d(sw + 128 * 128, &args.mapW[wi], start_bar(s), kb * 128, args.N + n * 128);
        };
        auto load_x = [&](int s, int seg, int kb) {
            const int xi = args.segs > 1 ? seg : (args.x_per_group ? g : 0);
            tma_load_2d(base + s * Cfg::STAGE_BYTES + Cfg::W_BYTES, &args.mapX[xi], start_bar(s), kb * 128, token0);
        };
        int pre = 0;
        if (args.weights_first) {              // the first ring of weights before the previous kernel's end
            int sg = seg, k = kb;
            pre = min(Cfg::STAGES, kb_hi - kb_lo);
            for (int s = 0; s < pre; ++s) {
                if (elect_one()) load_w(s, sg, k);
                __syncwarp();
                if (++k == args.k_blocks) {
                    k = 0;
                    ++sg;
                }
            }
        }
        // The next kernel may start from here on, not sooner: it may be one that loads weights before its own wait, and a
        // kernel before this one may be writing them still.
        pdl_wait();
        if (lane == 0) pdl_trigger();
        int s = 0;
        uint32_t phase = 0;
        for (int i = 0; i < kb_hi - kb_lo; ++i) {
            if (i >= pre && !mbar_wait_warp(done_bar(s), phase ^ 1u, abort_flag, args.status)) {
                aborted = true;
                break;
            }
            if (elect_one()) {
                if (i >= pre) load_w(s, seg, kb);
                load_x(s, seg, kb);
            }
            __syncwarp();
            if (++kb == args.k_blocks) {
                kb = 0;
                ++seg;
            }
            if (++s == Cfg::STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer (see the many-row kernel's)
        pdl_wait();                              // what the waits below wait for comes after it: their limit starts here
        constexpr uint32_t idesc = mma_idesc_e4m3(128, NT);
        int s = 0, b = 0;
        uint32_t phase = 0;
        for (int i = kb_lo; i < kb_hi; ++i) {
            const uint32_t d = tmem_base + static_cast<uint32_t>(b * Cfg::ACC_COLS);
            const uint32_t sw = base + s * Cfg::STAGE_BYTES;
            uint64_t wdesc = sw128_kmajor_desc(sw);
            uint64_t xdesc = sw128_kmajor_desc(sw + Cfg::W_BYTES);
            asm volatile("" : "+l"(xdesc), "+l"(wdesc));     // ready before the wait, not after it
            if (!mbar_wait_warp(start_bar(s), phase, abort_flag, args.status)) {
                aborted = true;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)      // 32 codes along K: 32 bytes inside the swizzle row
                    tc_mma_f8(d, wdesc + 2u * k, xdesc + 2u * k, idesc, k != 0 ? 1u : 0u);
                if (GLU) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f8(d + NT, wdesc + ((128 * 128) >> 4) + 2u * k, xdesc + 2u * k, idesc, k != 0 ? 1u : 0u);
                }
                tc_commit(done_bar(s));
            }
            __syncwarp();
            if (++s == Cfg::STAGES) {
                s = 0;
                phase ^= 1u;
            }
            b = (b + 1) & (Cfg::BUFS - 1);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------- scales
        // By asynchronous copies AHEAD blocks ahead (loaded one block ahead by the warps that use them, their latency
        // bounded the loop).  Block j's arrival waits for block j - STAGES's products, the barrier's phase before; by
        // then the sums have read block j - STAGES - BUFS's scales, whose slot may be asked for again.
        pdl_wait();
        const int blocks = kb_hi - kb_lo;
        const int tok = token0 + lane;
        const int wb = n + (lane == 1 ? args.up_block : 0);
        int seg = kb_lo / args.k_blocks, kb = kb_lo - seg * args.k_blocks, ask_slot = 0, asked = 0;
        const float *xs = nullptr, *ws = nullptr;
        auto segment = [&]() {
            xs = args.xs[args.segs > 1 ? seg : (args.x_per_group ? g : 0)] + static_cast<int64_t>(kb) * args.ldxs + tok;
            ws = args.ws[args.segs > 1 ? seg : g] + static_cast<int64_t>(wb) * args.k_blocks + kb;
        };
        segment();
        auto ask = [&](int i) {
            if (i < blocks) {
                const uint32_t at = smem_u32(scales_ptr + ask_slot * Cfg::SLOT_FLOATS + lane);
#pragma unroll
                for (int p = 0; p < NT; p += 32)
                    if (p + lane < NT && tok + p < args.M) cp_async4(at + p * 4, xs + p);
                if (lane < (GLU ? 2 : 1)) cp_async4(at + Cfg::FACTORS * 4, ws);
                xs += args.ldxs;
                ++ws;
                if (++kb == args.k_blocks && i + 1 < blocks) {
                    kb = 0;
                    ++seg;
                    segment();
                }
                ask_slot = ask_slot == Cfg::SLOTS - 1 ? 0 : ask_slot + 1;
            }
            cp_async_commit();
        };
        int s = 0, slot = 0;
        uint32_t phase = 0;
        for (int i = 0; i < blocks; ++i) {
            if (!mbar_wait_warp(done_bar(s), phase ^ 1u, abort_flag, args.status)) {
                aborted = true;
                break;
            }
            for (; asked <= i + Cfg::AHEAD; ++asked) ask(asked);
            cp_async_wait<Cfg::AHEAD>();
            __syncwarp();
            if (Cfg::FACTORED) {                 // the columns' factors, once for all warps that use them
                float* f = scales_ptr + slot * Cfg::SLOT_FLOATS;
                const float w = f[Cfg::FACTORS], up = f[Cfg::FACTORS + (GLU ? 1 : 0)];
#pragma unroll
                for (int p = 0; p < NT; p += 32) {
                    if (p + lane < NT) {
                        const float x = f[p + lane];
                        if (GLU) f[NT + p + lane] = x * up;
                        f[p + lane] = x * w;
                    }
                }
                __syncwarp();
            }
            slot = slot == Cfg::SLOTS - 1 ? 0 : slot + 1;
            if (elect_one()) mbar_arrive(done_bar(s));
            if (++s == Cfg::STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
        cp_async_wait<0>();
    } else {
        // ---------------------------------------------------- scaled sums
        const int e = warp - 3;
        const int q = warp & 3;                  // TMEM lane quarter this warp may access
        const int part = e >> 2;                 // gated: 0 gate, 1 up; plain: which half of the columns
        const int col0 = GLU ? 0 : part * Cfg::NC;
        const int blocks = kb_hi - kb_lo;
        // block i + BUFS may have block i's accumulator; the first ones' are free to begin with
        auto release = [&](int s) {
            if (elect_one()) mbar_arrive(start_bar(s));
        };
        for (int i = 0; i < Cfg::BUFS; ++i) release(i);
        f32x2 acc[Cfg::NC / 2];
#pragma unroll
        for (int j = 0; j < Cfg::NC / 2; ++j) acc[j] = 0;
        pdl_wait();                              // the previous kernel may read what this one writes
        int s = 0, b = 0, slot = 0;
        uint32_t phase = 0;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(GLU ? part * NT : col0);
        for (int i = 0; i < blocks; ++i) {
            if (!mbar_wait_warp(done_bar(s), phase, abort_flag, args.status)) {
                aborted = true;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = lane_base + static_cast<uint32_t>(b * Cfg::ACC_COLS);
            const float* f = scales_ptr + slot * Cfg::SLOT_FLOATS + (GLU && Cfg::FACTORED ? part * NT : col0);
            const float w = Cfg::FACTORED ? 1.0f : f[Cfg::FACTORS + part];
            const f32x2 w2 = pack2(w, w);
            constexpr bool kAhead = !Cfg::FACTORED;
            float dd[kAhead ? 2 : 1][16];
#pragma unroll
            for (int c = 0; c < Cfg::NC / 16; ++c) {
                float (&d)[16] = dd[kAhead ? c & 1 : 0];
                if (!kAhead || c == 0) tmem_ld(taddr + c * 16, d);
                f32x2 x[8];                      // the columns' factors
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(f + c * 16 + j);
                    x[j / 2] = Cfg::FACTORED ? pack2(v.x, v.y) : mul2(pack2(v.x, v.y), w2);
                    x[j / 2 + 1] = Cfg::FACTORED ? pack2(v.z, v.w) : mul2(pack2(v.z, v.w), w2);
                }
                tmem_wait(d);
                if (kAhead && c + 1 < Cfg::NC / 16) tmem_ld(taddr + (c + 1) * 16, dd[(c + 1) & 1]);
                if (c == Cfg::NC / 16 - 1) {     // all of this block is read: its columns are free again
                    tc_fence_before();
                    __syncwarp();
                    release(s + Cfg::BUFS < Cfg::STAGES ? s + Cfg::BUFS : s + Cfg::BUFS - Cfg::STAGES);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[c * 8 + j] = fma2(pack2(d[2 * j], d[2 * j + 1]), x[j], acc[c * 8 + j]);
            }
            slot = slot == Cfg::SLOTS - 1 ? 0 : slot + 1;
            b = (b + 1) & (Cfg::BUFS - 1);
            if (++s == Cfg::STAGES) {
                s = 0;
                phase ^= 1u;
            }
        }
        // Stage the sums [gate/up][token][128 columns] in the ring: the last block's products
        // have been waited for, so nothing reads or writes it any more.
        if (!aborted) {
            float* st = reinterpret_cast<float*>(base_ptr) + ((GLU ? part * NT : 0) + col0) * 128 + q * 32 + lane;
#pragma unroll
            for (int j = 0; j < Cfg::NC / 2; ++j) {
                float lo, hi;
                unpack2(acc[j], lo, hi);
                st[2 * j * 128] = lo;
                st[(2 * j + 1) * 128] = hi;
            }
        }
    }

    if (aborted) spin_ns(50000);        // let issued copies and products land
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) spin_ns(50000);
    // TMEM goes back before any peer is waited for: another kernel's CTAs that wait for some on this SM may be
    // what keeps a peer from having its own.
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc<Cfg::TMEM_COLS>(tmem_base);
    }
    if (split > 1) {
        __syncwarp();
        cluster_sync();
    }
    if (warp >= 3 && *abort_flag == 0) {
        const int e = warp - 3;
        const int tokens = min(NT, args.M - token0);
        const int col = n * 128 + lane * 4;
        const int nvalid = args.N - col;                     // this lane's columns inside the group
        auto sum = [&](int part, int j) {
            const uint32_t off = base + static_cast<uint32_t>(((part * NT + j) * 128 + lane * 4) * 4);
            if (split == 1) {
                float4 v;
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(off) : "memory");
                return v;
            }
            float4 x[8];
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < split) x[p] = ld_shared_cluster_f4(mapa_shared(off, static_cast<uint32_t>(p)));
            float4 v = x[0];
#pragma unroll
            for (int p = 1; p < 8; ++p) {
                if (p < split) {
                    v.x += x[p].x;
                    v.y += x[p].y;
                    v.z += x[p].z;
                    v.w += x[p].w;
                }
            }
            return v;
        };
        float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (!GLU && args.bias[g] != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < nvalid) bias[i] = bf16_to_f32(args.bias[g][col + i]);
        }
        for (int j = crank * Cfg::EPI_WARPS + e; j < tokens; j += split * Cfg::EPI_WARPS) {
            const float4 a = sum(0, j);
            float v[4] = {a.x, a.y, a.z, a.w};
            const int64_t row = token0 + j;
            if (GLU) {
                const float4 u = sum(1, j);
                const float up[4] = {u.x, u.y, u.z, u.w};
                finish_gated<ACT>(args, g, n, row, lane, v, up);
                continue;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += bias[i];
            }
            if (nvalid > 0)
                store_quad(args.out[g], args.ldo, args.out_kind == FP8_OUT_F32, row, col, min(4, nvalid), v);
        }
    }
    if (split > 1) {
        __syncwarp();
        cluster_sync_relaxed();                  // a peer may still read this CTA's sums
    }
}

// ------------------------------------------------------- many tokens: CTA pairs
//
// 256 x 256 tiles of a cluster of two CTAs on neighbouring SMs (cta_group::2),
// tokens as the MMA's rows: CTA r of a pair brings rows [128 r, 128 r + 128) of
// the tile's tokens and the r-th 128 rows of its weights (gated: CTA 0 gate's, CTA
// 1 the same rows of up).  With tokens as rows a thread needs one token's scale a
// block and one product with each weight block's; weights as rows would
// need one for every column.
//
// A K block's products (M = 256, N = 256) go to one of two TMEM accumulators,
// which eight warps a CTA read (a thread one token's 128 columns), scale and
// add to 128 fp32 sums a thread, while the MMAs fill the other.  From an
// accumulator's MMAs to the next ones that may overwrite it pass its MMAs (513
// cycles), their commit (330), the reading (310) and the release across the
// pair (265), with a trace's own cost; a K block takes about 610 cycles: 4096 rows
// of four shards' down projection 499 us with codes of zero (3.9 PFLOP/s), 718 with
// random ones, whose power lowers the clock; their gated products 1055 and 1397.
// What keeps each of these short was measured:
//  - one warp issues the MMAs, elected lanes in converged loops under a
//    warp-uniform branch (four MMAs, a wait and a commit: 380 cycles; one lane of a
//    diverged warp 690; two issuers' MMAs drain the tensor core between
//    them).  A wait and a commit cost it 50 to 100 cycles each, so one barrier a
//    stage says both that the tiles are there and that the accumulator is free,
//    and one that the products are done: the accumulator may be read and the
//    tiles overwritten.  Halves of N = 128 in twice the accumulators would need
//    eight MMAs a block, 900 cycles of issue.
//  - the scales come through shared memory, far ahead (loaded by the warps that
//    use them, their latency bounded the kernel).
//  - the last columns are read before the first half's multiply-adds are
//    all done: the registers hold 64 of the 128.
//
// split > 1: a cluster of `split` pairs shares a tile's K blocks in runs; the
// pairs' sums meet in shared memory (the ring, idle by then) and CTA p of
// each row half finishes its share of the rows, summing in the pairs' order.
constexpr int kManyStages = 6;
constexpr int kScaleAhead = 6;            // K blocks ahead that scales are asked for
constexpr int kScaleTurn = 5;             // stage of a turn of the ring at which the scales' warp waits for the last turn's reads
constexpr int kScaleSlots = 18;
// That wait, of a turn that begins with block T, says that the scales of blocks up to T - 2 have been read.  Until the next one, at
// blocks T + kScaleTurn to T + kScaleTurn + kManyStages - 1, scales of kScaleAhead blocks more are asked for, the last into
// the slot of block T + kScaleTurn + kManyStages - 1 + kScaleAhead - kScaleSlots.
static_assert(kScaleTurn + kManyStages - 1 + kScaleAhead - kScaleSlots <= -2 && kScaleTurn < kManyStages,
              "no slot is asked for before it is read");
constexpr int kManyThreads = 384;         // a warpgroup of producers, two of sums
constexpr int kManyFirst = 4;             // first warp of those
// Registers: 168 a thread at launch; the producers' warpgroup gives up 128 of them, each of the others takes 64.
constexpr int kManyProducerRegs = 40, kManySumRegs = 232;
static_assert(kManyProducerRegs + 2 * kManySumRegs <= 3 * 168, "a split takes no more than the launch has");

struct ManyCfg {
    static constexpr int STAGE_BYTES = 2 * 128 * 128;
    static constexpr int STG_PITCH = 80;                     // 64 bytes of a row and a pad: no bank conflicts
    static constexpr int STG_BYTES = 8 * 32 * STG_PITCH;
    static constexpr int AMAX_BYTES = 2 * 2 * 128 * 4;       // two halves' largest values, two tiles in turn
    static constexpr int NBARS = 2 * kManyStages + 5;
    static constexpr int RAW_FLOATS = 128 + 4;               // a block's scales: 128 rows', the two weight blocks'
    static constexpr int RAW_BYTES = kScaleSlots * RAW_FLOATS * 4;
    static constexpr int SUM_PITCH = 260;                    // floats of a staged row of sums
    static constexpr int SMEM_BYTES = 1024 + kManyStages * STAGE_BYTES + STG_BYTES + AMAX_BYTES + RAW_BYTES + NBARS * 8 + 16;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
    static_assert(128 * SUM_PITCH * 4 <= kManyStages * STAGE_BYTES, "a CTA's sums fit the ring");
};

__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tile index -> (group, row tile, column tile): bands of row tiles, the row
// tile fastest inside a band; with shared rows a band covers every group's columns.
__device__ __forceinline__ void many_coords(const Fp8GemmArgs& a, int tile, int& g, int& m, int& n) {
    const int cols = a.x_per_group ? a.n_tiles : a.groups * a.n_tiles;
    const int per_span = a.m_tiles * cols;
    const int outer = tile / per_span;
    const int l = tile - outer * per_span;
    const int band = l / (a.band * cols);
    const int first = band * a.band;
    const int gm = min(a.m_tiles - first, a.band);
    const int r = l - band * a.band * cols;
    m = first + r % gm;
    const int col = r / gm;
    g = a.x_per_group ? outer : col / a.n_tiles;
    n = a.x_per_group ? col : col - g * a.n_tiles;
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void st_global_32(void* to, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// A warp writes its rows' 64-byte pieces of an output (rows row0 .. row0 + live - 1, byte offset off of a row): each
// lane's piece is staged at lane * STG_PITCH.  Whole pieces of aligned rows go out as 16-byte stores of 8 rows at a
// time, others element by element.
template <int ES>
__device__ __forceinline__ void many_store(const uint8_t* st, uint8_t* out, int64_t row0, int live, int64_t pitch,
                                           int64_t off, int valid_bytes, int lane) {
    __syncwarp();
    if (valid_bytes >= 64 && ((reinterpret_cast<uintptr_t>(out) + off) & 15) == 0 && (pitch & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r < live)
                *reinterpret_cast<uint4*>(out + (row0 + r) * pitch + off + (lane & 3) * 16) =
                    *reinterpret_cast<const uint4*>(st + r * ManyCfg::STG_PITCH + (lane & 3) * 16);
        }
    } else {
        constexpr int PER = 64 / ES;
        for (int i = lane; i < live * PER; i += 32) {
            const int r = i / PER, b = (i % PER) * ES;
            if (b < valid_bytes) {
                uint8_t* dst = out + (row0 + r) * pitch + off + b;
                const uint8_t* src = st + r * ManyCfg::STG_PITCH + b;
                if constexpr (ES == 4)
                    *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
                else if constexpr (ES == 2)
                    *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
                else
                    *dst = *src;
            }
        }
    }
    __syncwarp();
}

// A warp's rows of 2 * PAIRS columns from col0 on, as fp32 or bf16.
template <int PAIRS>
__device__ __forceinline__ void store_sums(const Fp8GemmArgs& args, uint8_t* st, uint8_t* out, int64_t row0, int live,
                                           int col0, int valid, int lane, const f32x2 (&v)[PAIRS]) {
    uint8_t* st_lane = st + lane * ManyCfg::STG_PITCH;
    if (args.out_kind == FP8_OUT_F32) {
#pragma unroll
        for (int c = 0; c < PAIRS; c += 8) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float4 x;
                unpack2(v[c + j], x.x, x.y);
                unpack2(v[c + j + 1], x.z, x.w);
                *reinterpret_cast<float4*>(st_lane + j * 8) = x;
            }
            many_store<4>(st, out, row0, live, args.ldo * 4, (col0 + 2 * c) * 4LL, (valid - 2 * c) * 4, lane);
        }
    } else {
#pragma unroll
        for (int c = 0; c < PAIRS; c += 16) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    unpack2(v[c + j + i], lo, hi);
                    x[i] = pack_bf16x2(lo, hi);
                }
                *reinterpret_cast<uint4*>(st_lane + j * 4) = make_uint4(x[0], x[1], x[2], x[3]);
            }
            many_store<2>(st, out, row0, live, args.ldo * 2, (col0 + 2 * c) * 2LL, (valid - 2 * c) * 2, lane);
        }
    }
}

template <int ACT>
__global__ void __launch_bounds__(kManyThreads, 1) fp8_many_kernel(const __grid_constant__ Fp8GemmArgs args) {
    constexpr bool GLU = ACT != TP_ACT_NONE;
    using Cfg = ManyCfg;
    constexpr int STAGES = kManyStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    constexpr int kStgOff = STAGES * Cfg::STAGE_BYTES;
    constexpr int kAmaxOff = kStgOff + Cfg::STG_BYTES;
    constexpr int kRawOff = kAmaxOff + Cfg::AMAX_BYTES;
    constexpr int kBarOff = kRawOff + Cfg::RAW_BYTES;
    const uint32_t bar_base = base + kBarOff;
    // a stage's products may start: its tiles are there and the accumulator is free
    // ... and are done: the scales are there too, the accumulator may be read and the tiles overwritten
    auto start_bar = [&](int s) { return bar_base + 8u * s; };
    auto done_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
    auto half_bar = [&](int q) { return bar_base + 8u * (2 * STAGES + q); };   // the two warps of a lane quarter
    const uint32_t turn_bar = bar_base + 8u * (2 * STAGES + 4);   // this CTA's sums have read a turn's scales
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + kBarOff + 8 * Cfg::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + kBarOff + 8 * Cfg::NBARS + 4);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // uniform to the compiler
    const int lane = threadIdx.x & 31;
    const int split = args.split;
    const uint32_t crank = cluster_ctarank();
    const uint32_t rank = crank & 1;                     // 0: issues the pair's MMAs
    const uint32_t leader = crank & ~1u;
    const int part = static_cast<int>(crank >> 1);
    const uint16_t pair_mask = static_cast<uint16_t>(0x3u << leader);
    const int cluster = static_cast<int>(blockIdx.x) / (2 * split);
    const int nclusters = static_cast<int>(gridDim.x) / (2 * split);
    const int kb_all = args.k_blocks * args.segs;
    const int kb_lo = static_cast<int>(static_cast<int64_t>(part) * kb_all / split);
    const int kb_hi = static_cast<int>(static_cast<int64_t>(part + 1) * kb_all / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(start_bar(s), 1 + 16);             // the tiles, the eight warps of sums in either CTA
            mbar_init(done_bar(s), 2);                   // the products, the scales
        }
        for (int q = 0; q < 4; ++q) mbar_init(half_bar(q), 2);
        mbar_init(turn_bar, 8 * STAGES);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair<512>(smem_u32(tmem_slot));
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                      // the peer's barriers exist before any remote use
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // The end of either role: nothing of this CTA is in flight and every sum is staged when it returns.
    auto meet = [&](bool gave_up) {
        if (gave_up) spin_ns(50000);                     // let issued copies and products land
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        if (*abort_flag) spin_ns(50000);
        cluster_sync();                                  // no MMA or remote arrive still targets the peer
    };

    if (warp < kManyFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kManyProducerRegs));
        bool aborted = false;
        if (warp == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            pdl_wait();
            if (lane == 0) pdl_trigger();                // not sooner: see the few-row kernel's
            int s = 0;
            uint32_t phase = 0;
            for (int tile = cluster; tile < args.total_tiles && !aborted; tile += nclusters) {
                int g, m, n;
                many_coords(args, tile, g, m, n);
                const int x_row = m * 256 + static_cast<int>(rank) * 128;
                const int w_row = GLU ? (rank == 0 ? n * 128 : args.N + n * 128) : n * 256 + static_cast<int>(rank) * 128;
                int seg = kb_lo / args.k_blocks, kb = kb_lo - seg * args.k_blocks;
                for (int i = kb_lo; i < kb_hi; ++i) {
                    if (!mbar_wait_warp(done_bar(s), phase ^ 1u, abort_flag, args.status)) {
                        aborted = true;
                        break;
                    }
                    const int xi = args.segs > 1 ? seg : (args.x_per_group ? g : 0);
                    const int wi = args.segs > 1 ? seg : g;
                    const uint32_t full = mapa_shared(start_bar(s), leader);
                    const uint32_t sx = base + s * Cfg::STAGE_BYTES;
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(start_bar(s), 2u * Cfg::STAGE_BYTES);
                        tma_load_2d_pair(sx, &args.mapX[xi], full, kb * 128, x_row);
                        tma_load_2d_pair(sx + 128 * 128, &args.mapW[wi], full, kb * 128, w_row);
                    }
                    __syncwarp();
                    if (++kb == args.k_blocks) {
                        kb = 0;
                        ++seg;
                    }
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        if (warp == 3) {
            // ------------------------------------------------ scales (both CTAs)
            // Those of this CTA's 128 rows and the two weight blocks, by asynchronous copies kScaleAhead blocks ahead
            // (loaded two blocks ahead by the warps that use them, their latency bounded the kernel).  That a slot's scales
            // have been read says a barrier of its own, waited for once a turn of the ring: the accumulators' releases, by which
            // the products' barriers follow each other, order no reads of shared memory.  It costs 1 % (down projection of
            // 4096 rows 709 us without, 718 with it); one arrival a turn under a branch in place of one a block, 7 %.
            pdl_wait();
            float* raw = reinterpret_cast<float*>(base_ptr + kRawOff);
            int s = 0, ask_slot = 0;
            uint32_t phase = 0;
            for (int tile = cluster; tile < args.total_tiles && !aborted; tile += nclusters) {
                int g, m, n;
                many_coords(args, tile, g, m, n);
                const int64_t row0 = static_cast<int64_t>(m) * 256 + static_cast<int64_t>(rank) * 128 + lane;
                // the weight blocks of the tile's two halves; where the second does not exist its sums are never stored
                const int wb = lane == 0 ? (GLU ? n : n * 2)
                               : GLU     ? args.up_block + n
                                         : ((n * 2 + 1) * 128 < args.N ? n * 2 + 1 : n * 2);
                const int blocks = kb_hi - kb_lo;
                int seg = kb_lo / args.k_blocks, kb = kb_lo - seg * args.k_blocks;     // of the next block asked for
                const float *xs = nullptr, *ws = nullptr;
                auto segment = [&]() {
                    xs = args.xs[args.segs > 1 ? seg : (args.x_per_group ? g : 0)] + static_cast<int64_t>(kb) * args.ldxs + row0;
                    ws = args.ws[args.segs > 1 ? seg : g] + static_cast<int64_t>(wb) * args.k_blocks + kb;
                };
                segment();
                auto ask = [&](int i) {
                    if (i < blocks) {
                        const uint32_t at = smem_u32(raw + ask_slot * Cfg::RAW_FLOATS) + lane * 4;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (row0 + r * 32 < args.M) cp_async4(at + r * 128, xs + r * 32);
                        if (lane < 2) cp_async4(at + 512, ws);
                        xs += args.ldxs;
                        ++ws;
                        if (++kb == args.k_blocks && i + 1 < blocks) {
                            kb = 0;
                            ++seg;
                            segment();
                        }
                        ask_slot = ask_slot == kScaleSlots - 1 ? 0 : ask_slot + 1;
                    }
                    cp_async_commit();
                };
                // the first ones of a tile are asked for as its blocks come up, each after its wait
                int asked = 0;
                for (int i = 0; i < blocks; ++i) {
                    if (!mbar_wait_warp(done_bar(s), phase ^ 1u, abort_flag, args.status)) {
                        aborted = true;
                        break;
                    }
                    if (s == kScaleTurn && !mbar_wait_warp(turn_bar, phase ^ 1u, abort_flag, args.status)) {
                        aborted = true;
                        break;
                    }
                    for (; asked <= i + kScaleAhead; ++asked) ask(asked);
                    cp_async_wait<kScaleAhead>();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(done_bar(s));
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            cp_async_wait<0>();
        }
        if (warp == 1 && rank == 0) {
            // ------------------------------------------------ MMA issuer (even CTA)
            pdl_wait();                                  // the limit of the waits below starts after it
            constexpr uint32_t idesc = mma_idesc_e4m3(256, 256);
            int s = 0, b = 0;
            uint32_t phase = 0;
            const int tiles = cluster < args.total_tiles ? (args.total_tiles - 1 - cluster) / nclusters + 1 : 0;
            for (int64_t i = static_cast<int64_t>(tiles) * (kb_hi - kb_lo); i > 0; --i) {   // K blocks of all of the cluster's tiles
                const uint32_t sx = base + s * Cfg::STAGE_BYTES;
                uint64_t xdesc = sw128_kmajor_desc(sx);
                uint64_t wdesc = sw128_kmajor_desc(sx + 128 * 128);
                asm volatile("" : "+l"(xdesc), "+l"(wdesc));     // ready before the wait, not after it
                if (!mbar_wait_warp(start_bar(s), phase, abort_flag, args.status)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t d = tmem_base + static_cast<uint32_t>(b * 256);
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_f8_pair(d, xdesc + 2u * k, wdesc + 2u * k, idesc, k != 0 ? 1u : 0u);
                    tc_commit_pair(done_bar(s), pair_mask);
                }
                __syncwarp();
                b ^= 1;
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        meet(aborted);
        if (split > 1) cluster_sync_relaxed();           // a peer may still read this CTA's sums
        if (warp == 1) {
            __syncwarp();
            tc_fence_after();
            tmem_dealloc_pair<512>(tmem_base);
        }
    } else {
        // ---------------------------------------------------- scaled sums and output (both CTAs)
        bool aborted = false;
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManySumRegs));
        const int q = warp & 3;
        const int half = (warp - kManyFirst) >> 2;                 // plain: columns [128 half, +128); gated: [64 half, +64) of gate and of up
        const int row_in_tile = static_cast<int>(rank) * 128 + q * 32 + lane;
        uint8_t* st = base_ptr + kStgOff + (warp - kManyFirst) * 32 * Cfg::STG_PITCH;
        uint8_t* st_lane = st + lane * Cfg::STG_PITCH;
        float* amax = reinterpret_cast<float*>(base_ptr + kAmaxOff) + q * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        const int col_a = half * 64, col_b = 128 + half * 64;            // the tile's columns of sums 0..63 and 64..127
        pdl_wait();                                       // the previous kernel may read what this one writes
        const float* raw = reinterpret_cast<const float*>(base_ptr + kRawOff);
        // the accumulators are free to begin with: the first two blocks' starts
        const uint32_t start0 = mapa_shared(start_bar(0), leader);
        auto release = [&](int s, bool read) {
            if (elect_one()) {
                mbar_arrive_cluster_relaxed(start0 + 8u * s);
                if (read) mbar_arrive(turn_bar);          // the scales of the blocks before
            }
        };
        release(0, false);
        release(1, false);
        int s = 0, b = 0, turn = 0, slot = 0;
        uint32_t phase = 0, hphase = 0;
        for (int tile = cluster; tile < args.total_tiles && !aborted; tile += nclusters) {
            int g, m, n;
            many_coords(args, tile, g, m, n);
            const int64_t row = static_cast<int64_t>(m) * 256 + row_in_tile;
            const bool row_ok = row < args.M;
            f32x2 sums[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) sums[j] = 0;
            for (int i = kb_lo; i < kb_hi; ++i) {
                if (!mbar_wait_warp(done_bar(s), phase, abort_flag, args.status)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = lane_base + static_cast<uint32_t>(b * 256 + half * 64);
                float d0[32], d1[32];
                tmem_ld(taddr, d0);
                tmem_ld(taddr + 32, d1);
                const float* scales = raw + slot * Cfg::RAW_FLOATS;
                const float sx = scales[q * 32 + lane];
                const float fa = sx * scales[128];
                const f32x2 sa = pack2(fa, fa);
                auto add = [&](int c, float (&d)[32], f32x2 s) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) sums[c * 16 + j] = fma2(pack2(d[2 * j], d[2 * j + 1]), s, sums[c * 16 + j]);
                };
                tmem_wait(d0, d1);
                add(0, d0, sa);
                tmem_ld(taddr + 128, d0);
                add(1, d1, sa);
                tmem_ld(taddr + 160, d1);
                tmem_wait(d0, d1);
                tc_fence_before();                        // the accumulator is read: block i + 2's products may have it
                __syncwarp();
                release(s + 2 < STAGES ? s + 2 : s + 2 - STAGES, true);
                // read here, and not before: what is left to add is then scheduled behind the release (4096 gated rows of
                // 14336 x 8192 in four shards 1564 us without)
                const float fb = sx * *reinterpret_cast<const volatile float*>(scales + 129);
                const f32x2 sb = pack2(fb, fb);
                add(2, d0, sb);
                add(3, d1, sb);
                b ^= 1;
                slot = slot == kScaleSlots - 1 ? 0 : slot + 1;
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (aborted) break;
            const int64_t row0 = static_cast<int64_t>(m) * 256 + static_cast<int64_t>(rank) * 128 + q * 32;
            const int live = static_cast<int>(min(static_cast<int64_t>(32), args.M - row0));   // rows of this warp
            if (split > 1) {
                // this CTA's sums to the ring, a row of 256 at SUM_PITCH; joined below
                float* to = reinterpret_cast<float*>(base_ptr) + (q * 32 + lane) * Cfg::SUM_PITCH;
#pragma unroll
                for (int j = 0; j < 128; j += 4) {
                    float4 v;
                    unpack2(sums[j / 2], v.x, v.y);
                    unpack2(sums[j / 2 + 1], v.z, v.w);
                    *reinterpret_cast<float4*>(to + (j < 64 ? col_a + j : col_b + j - 64)) = v;
                }
            } else if (GLU) {
                const GateAct<ACT> act(args.out_kind == FP8_OUT_CODES);
                uint8_t* out = static_cast<uint8_t*>(args.out[g]);
                const int col0 = n * 128 + half * 64;
                const int valid = args.N - col0;          // columns of this half inside the group
                f32x2 v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = mul2(act(sums[j]), sums[32 + j]);
                if (args.out_kind == FP8_OUT_CODES) {
                    if (valid < 64) {                     // N is a multiple of 16: pairs are in or out
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 2 * j < valid ? v[j] : 0;
                    }
                    const float top = amax_pairs(v);
                    float* mine = amax + turn * 256;
                    mine[half * 128] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half_bar(q));
                    if (!mbar_wait_warp(half_bar(q), hphase, abort_flag, args.status)) {
                        aborted = true;
                        break;
                    }
                    hphase ^= 1u;
                    const float s = fp8_scale(max_nan(mine[0], mine[128]));
                    turn ^= 1;
                    if (half == 0 && row_ok) args.os[g][static_cast<int64_t>(n) * args.ldos + row] = s;
                    if (live > 0 && valid > 0) {
                        uint32_t code[16];
                        fp8_codes(v, s, code);
                        if (valid >= 64 && ((reinterpret_cast<uintptr_t>(out) | args.ldo) & 31) == 0) {
                            uint8_t* to = out + (row0 + lane) * args.ldo + col0;       // this lane's 64 bytes, a sector each
                            if (lane < live) {
                                st_global_32(to, &code[0]);
                                st_global_32(to + 32, &code[8]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; j += 4)
                                *reinterpret_cast<uint4*>(st_lane + j * 4) = make_uint4(code[j], code[j + 1], code[j + 2], code[j + 3]);
                            many_store<1>(st, out, row0, live, args.ldo, col0, valid, lane);
                        }
                    }
                } else if (live > 0 && valid > 0) {
                    store_sums<32>(args, st, out, row0, live, col0, valid, lane, v);
                }
            } else {
                uint8_t* out = static_cast<uint8_t*>(args.out[g]);
                const uint16_t* bias = args.bias[g];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int col0 = n * 256 + p * 128 + half * 64;
                    const int valid = args.N - col0;
                    if (live <= 0 || valid <= 0) break;
                    f32x2 v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = sums[p * 32 + j];
                    if (bias != nullptr) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float lo, hi;
                            unpack2(v[j], lo, hi);
                            if (2 * j < valid) lo += bf16_to_f32(bias[col0 + 2 * j]);
                            if (2 * j + 1 < valid) hi += bf16_to_f32(bias[col0 + 2 * j + 1]);
                            v[j] = pack2(lo, hi);
                        }
                    }
                    store_sums<32>(args, st, out, row0, live, col0, valid, lane, v);
                }
            }
        }
        meet(aborted);
        if (split > 1) {
            // Rows [part * 128 / split, ...) of this CTA's 128: a warp a row, a lane columns [4 lane, +4) of both halves.
            if (*abort_flag == 0) {
                int g, m, n;
                many_coords(args, cluster, g, m, n);         // one tile a cluster
                const int per = 128 / split;
                for (int r = part * per + warp - kManyFirst; r < (part + 1) * per; r += 8) {
                    const int64_t row = static_cast<int64_t>(m) * 256 + static_cast<int64_t>(rank) * 128 + r;
                    if (row >= args.M) break;
                    float v[2][4];
    #pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t off = base + static_cast<uint32_t>((r * Cfg::SUM_PITCH + h * 128 + lane * 4) * 4);
                        float4 x[4];
    #pragma unroll
                        for (int p = 0; p < 4; ++p)
                            if (p < split) x[p] = ld_shared_cluster_f4(mapa_shared(off, static_cast<uint32_t>(2 * p) + rank));
                        float4 a = x[0];
    #pragma unroll
                        for (int p = 1; p < 4; ++p) {
                            if (p < split) {
                                a.x += x[p].x;
                                a.y += x[p].y;
                                a.z += x[p].z;
                                a.w += x[p].w;
                            }
                        }
                        v[h][0] = a.x;
                        v[h][1] = a.y;
                        v[h][2] = a.z;
                        v[h][3] = a.w;
                    }
                    if (GLU) {
                        finish_gated<ACT>(args, g, n, row, lane, v[0], v[1]);
                    } else {
    #pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int col = n * 256 + h * 128 + lane * 4;
                            const int nvalid = args.N - col;
                            if (nvalid > 0) {
                                if (args.bias[g] != nullptr) {
    #pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        if (i < nvalid) v[h][i] += bf16_to_f32(args.bias[g][col + i]);
                                }
                                store_quad(args.out[g], args.ldo, args.out_kind == FP8_OUT_F32, row, col, min(4, nvalid), v[h]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            cluster_sync_relaxed();                      // a peer may still read this CTA's sums
        }
    }
}

// ------------------------------------------------------------------ host

// Costs in hundredths of a microsecond, fitted to the kernels' times over 70 shapes (the choice costs 1 % over the best of all
// variants there and over 250 others).  A wave of the few-row kernel takes so much a K block, by its tokens, plain and
// gated; 260 to 660 beside them, most of it the ends of tiles, which parts share; and parts that are joined 30 and 15 each
// (28).  A wave of the many-row kernel takes 34 a block, 380, and 400 where parts are joined.  Neither is less than the weights
// take, at 6.4 TB/s with 240 CTAs and a little less with fewer (the down projection of 32 tokens: 5.5 TB/s with 128, 6.2
// with 256).
constexpr int64_t few_block_cost(int nt, bool glu) {
    return nt <= 16 ? (glu ? 35 : 26) : nt <= 32 ? (glu ? 40 : 28) : nt <= 64 ? (glu ? 44 : 39) : glu ? 66 : 31;
}
constexpr int64_t few_wave_cost(int nt, bool glu, bool shared, int split) {
    return 260 + (nt > 64 ? (glu ? 400 : 70) : nt > 32 ? (glu ? 60 : shared ? 300 : 0) : 0) / split;
}
constexpr int64_t few_join_cost(int nt, int split) { return split > 1 ? 30 + (nt > 64 ? 28 : 15) * split : 0; }
constexpr int64_t kManyBlock = 34, kManyWave = 380, kManyJoin = 400;

static int64_t stream_cost(const Fp8GemmDesc& d, int64_t ctas) {
    const int64_t bytes = d.groups * d.segs * d.N * (d.glu ? 2 : 1) * d.K;
    return bytes / 64000 * 24000 / (20400 + 15 * std::min<int64_t>(ctas, 240));
}

// Clusters of `size` CTAs of a kernel that can be resident at once, looked up once per device (cache: the kernel's).  Its
// registers, shared memory and TMEM leave room for per_sm CTAs an SM.  The runtime's queries count one for every kernel that allocates TMEM
// (with 64 KB of shared memory as with 112; without the allocation 3 and 2), but two run at once, as their clocks on the SM show.
static int resident_clusters(const void* kern, int size, int threads, int smem, int per_sm, std::atomic<int>* cache) {
    int dev = 0;
    cudaGetDevice(&dev);
    std::atomic<int>* slot = dev >= 0 && dev < 64 ? cache + dev : nullptr;       // relaxed: racing first calls store the same value
    if (slot != nullptr && slot->load(std::memory_order_relaxed) != 0) return slot->load(std::memory_order_relaxed);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max(1, device_sms()) / size * size * 2), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int v = 0, counted = 0;
    if (cudaOccupancyMaxActiveClusters(&v, kern, &cfg) != cudaSuccess || v <= 0 ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&counted, kern, threads, static_cast<size_t>(smem)) != cudaSuccess || counted <= 0)
        v = -1;
    else if (counted < per_sm)
        v = v / counted * per_sm;
    if (slot != nullptr) slot->store(v, std::memory_order_relaxed);
    return v;
}

// The number of CTAs (1 to 8; of CTA pairs 1, 2 or 4) that share a tile, with two K blocks each at least (pairs four), and what that costs;
// resident(tile, parts) says how many such clusters run at once.  What the sizes of
// clusters that fit the GPU at once decide most: QKV of 8 shards (80 tiles), 16 tokens: 18.4, 17.9, 15.9, 20.0 us in 1, 2, 3, 4
// parts; the down projection of 32 tokens (64 tiles of 224 blocks) 65, 41, 40, 38, 46 us in 1 to 5; 8 tiles of 32 blocks
// 7.5, 5.4, 4.7, 4.1, 4.1, 4.2 us in 1 to 5 and 8.
template <typename Resident>
static Fp8Plan plan_tile(const Fp8GemmDesc& d, int tile, int sms, Resident&& resident) {
    Fp8Plan best;
    const bool pairs = tile == 256, glu = d.glu != 0;
    const int cols = pairs && !glu ? 256 : 128;
    const int64_t tiles = d.groups * ((d.M + tile - 1) / tile) * ((d.N + cols - 1) / cols), kb = fp8_groups(d.K) * d.segs;
    for (int parts = 1; parts <= (pairs ? 4 : 8); ++parts) {
        if (pairs && parts == 3) continue;
        if (d.force_parts > 0 ? parts != d.force_parts || kb < parts : parts > 1 && kb / parts < (pairs ? 4 : 2)) continue;
        const int mc = resident(tile, parts);
        if (mc <= 0) continue;
        const int64_t waves = (tiles + mc - 1) / mc, ctas = std::min<int64_t>(tiles, mc) * parts * (pairs ? 2 : 1);
        const int64_t stream = stream_cost(d, ctas), blocks = (kb + parts - 1) / parts;
        int64_t cost;
        if (pairs) {
            cost = std::max(waves * blocks * kManyBlock, stream) + waves * (kManyWave + (parts > 1 ? kManyJoin : 0));
        } else {
            const bool shared = ctas > sms;                              // two CTAs on an SM
            cost = std::max(waves * blocks * few_block_cost(tile, glu), stream) + waves * few_wave_cost(tile, glu, shared, parts) +
                   few_join_cost(tile, parts);
        }
        if (best.cost < 0 || cost < best.cost) {
            best.cost = cost;
            best.tile = tile;
            best.parts = parts;
            best.clusters = mc;
        }
    }
    return best;
}

// Up to 64 tokens one tile of them; more: whichever kernel and tile should take least.  100 tokens of four shards' down projection:
// 44 us in tiles of 128, 48 on CTA pairs; 300 in QKV of eight shards 47 and 50; gate_up of 100 tokens 102 and 86.
template <typename Resident>
static Fp8Plan plan_product(const Fp8GemmDesc& d, int sms, Resident&& resident) {
    if (d.force_tile > 0) return plan_tile(d, d.force_tile, sms, resident);
    if (d.M <= 64) return plan_tile(d, d.M <= 16 ? 16 : d.M <= 32 ? 32 : 64, sms, resident);
    Fp8Plan best;
    for (int tile : {256, 128, 64}) {
        const Fp8Plan p = plan_tile(d, tile, sms, resident);
        if (p.cost >= 0 && (best.cost < 0 || p.cost < best.cost)) best = p;
    }
    return best;
}

Fp8Plan plan_fp8_gemm(const Fp8GemmDesc& d, int sms, const int* resident) {
    return plan_product(d, sms, [&](int tile, int parts) {
        return resident[(tile == 16 ? 0 : tile == 32 ? 1 : tile == 64 ? 2 : tile == 128 ? 3 : 4) * 8 + parts - 1];
    });
}

// Clusters of `parts` CTAs (CTA pairs) that share a tile and can be resident at once; 0 or less: none.
template <int NT, int ACT>
static int resident_few(int parts) {
    using Cfg = FewCfg<NT, ACT != TP_ACT_NONE>;
    static std::atomic<int> resident[8][64];
    static std::atomic<uint64_t> smem_set{0};
    const void* kern = reinterpret_cast<const void*>(fp8_few_kernel<NT, ACT>);
    if (!smem_attribute_once(kern, Cfg::SMEM_BYTES, smem_set)) return 0;
    return resident_clusters(kern, parts, Cfg::THREADS, Cfg::SMEM_BYTES, Cfg::ONE ? 1 : 2, resident[parts - 1]);
}

template <int ACT>
static int resident_many(int parts) {
    static std::atomic<int> resident[3][64];
    static std::atomic<uint64_t> smem_set{0};
    const void* kern = reinterpret_cast<const void*>(fp8_many_kernel<ACT>);
    if (!smem_attribute_once(kern, ManyCfg::SMEM_BYTES, smem_set)) return 0;
    return resident_clusters(kern, 2 * parts, kManyThreads, ManyCfg::SMEM_BYTES, 1, resident[parts >> 1]);
}

template <int NT, int ACT>
static tp_status launch_few(Fp8GemmArgs& a, const Fp8GemmDesc& d, const Fp8Plan& plan, cudaStream_t stream) {
    using Cfg = FewCfg<NT, ACT != TP_ACT_NONE>;
    a.m_tiles = static_cast<int>((d.M + NT - 1) / NT);
    a.n_tiles = static_cast<int>((d.N + 127) / 128);
    const int64_t tiles = static_cast<int64_t>(d.groups) * a.m_tiles * a.n_tiles;
    const int split = plan.parts;
    if (tiles * split > INT32_MAX) return TP_ERR_UNSUPPORTED;
    a.total_tiles = static_cast<int>(tiles);
    a.split = split;
    a.x_box_rows = static_cast<int>(std::min<int64_t>(NT, (d.M + 7) / 8 * 8));
    const int nX = d.segs > 1 ? d.segs : (d.x_per_group ? d.groups : 1);
    const int nW = d.segs > 1 ? d.segs : d.groups;
    for (int i = 0; i < nX; ++i)
        if (!make_byte_operand_map(&a.mapX[i], d.x[i], d.M, d.K, d.ldx, a.x_box_rows)) return TP_ERR_CUDA;
    for (int i = 0; i < nW; ++i)
        if (!make_byte_operand_map(&a.mapW[i], d.w[i], ACT != TP_ACT_NONE ? 2 * d.N : d.N, d.K, d.ldw, 128)) return TP_ERR_CUDA;
    auto kern = fp8_few_kernel<NT, ACT>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

// CTA pairs: 256 x 256 tiles, whose K blocks are split over 1, 2 or 4 pairs.
template <int ACT>
static tp_status launch_many(Fp8GemmArgs& a, const Fp8GemmDesc& d, const Fp8Plan& plan, cudaStream_t stream) {
    using Cfg = ManyCfg;
    const int out_cols = ACT != TP_ACT_NONE ? 128 : 256;
    a.m_tiles = static_cast<int>((d.M + 255) / 256);
    a.n_tiles = static_cast<int>((d.N + out_cols - 1) / out_cols);
    const int64_t tiles = static_cast<int64_t>(d.groups) * a.m_tiles * a.n_tiles;
    a.total_tiles = static_cast<int>(tiles);
    a.x_box_rows = 128;
    // a band's rows stay in L2 while its columns of weights stream past: about 48 MB of them
    a.band = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.m_tiles, (int64_t(48) << 20) / (256 * d.K * d.segs))));
    const int nX = d.segs > 1 ? d.segs : (d.x_per_group ? d.groups : 1);
    const int nW = d.segs > 1 ? d.segs : d.groups;
    for (int i = 0; i < nX; ++i)
        if (!make_byte_operand_map(&a.mapX[i], d.x[i], d.M, d.K, d.ldx, 128)) return TP_ERR_CUDA;
    for (int i = 0; i < nW; ++i)
        if (!make_byte_operand_map(&a.mapW[i], d.w[i], ACT != TP_ACT_NONE ? 2 * d.N : d.N, d.K, d.ldw, 128)) return TP_ERR_CUDA;
    if (tiles * plan.parts > INT32_MAX / 2) return TP_ERR_UNSUPPORTED;
    a.split = plan.parts;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(2 * plan.parts);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // one pair a tile: a persistent grid; parts: a cluster a tile
    const int64_t resident = d.max_clusters > 0 ? std::min(d.max_clusters, plan.clusters) : plan.clusters;
    const int64_t clusters = plan.parts == 1 ? std::min<int64_t>(tiles, resident) : tiles;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * plan.parts), 1, 1);
    cfg.blockDim = dim3(kManyThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_many_kernel<ACT>, a) == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

template <int ACT>
static tp_status launch_sized(Fp8GemmArgs& a, const Fp8GemmDesc& d, cudaStream_t stream) {
    const Fp8Plan plan = plan_product(d, std::max(1, device_sms()), [](int tile, int parts) {
        switch (tile) {
            case 16: return resident_few<16, ACT>(parts);
            case 32: return resident_few<32, ACT>(parts);
            case 64: return resident_few<64, ACT>(parts);
            case 128: return resident_few<128, ACT>(parts);
            default: return resident_many<ACT>(parts);
        }
    });
    if (plan.cost < 0) return d.force_parts > 0 ? TP_ERR_UNSUPPORTED : TP_ERR_CUDA;
    switch (plan.tile) {
        case 16: return launch_few<16, ACT>(a, d, plan, stream);
        case 32: return launch_few<32, ACT>(a, d, plan, stream);
        case 64: return launch_few<64, ACT>(a, d, plan, stream);
        case 128: return launch_few<128, ACT>(a, d, plan, stream);
        default: return launch_many<ACT>(a, d, plan, stream);
    }
}

tp_status launch_fp8_gemm(const Fp8GemmDesc& d, cudaStream_t stream) {
    if (d.M == 0 || d.N == 0) return TP_OK;
    Fp8GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    for (int i = 0; i < TP_MAX_SHARDS; ++i) {
        a.xs[i] = d.xs[i];
        a.ws[i] = d.ws[i];
        a.out[i] = d.out[i];
        a.os[i] = d.os[i];
        a.bias[i] = static_cast<const uint16_t*>(d.bias[i]);
    }
    a.ldxs = d.ldxs;
    a.ldo = d.ldo;
    a.ldos = d.ldos;
    a.M = static_cast<int>(d.M);
    a.N = static_cast<int>(d.N);
    a.k_blocks = static_cast<int>(fp8_groups(d.K));
    a.segs = d.segs;
    a.groups = d.groups;
    a.x_per_group = d.x_per_group;
    a.up_block = static_cast<int>(fp8_groups(d.N));
    a.out_kind = d.out_kind;
    a.status = d.status;
    a.weights_first = d.weights_first;
    if (static_cast<int64_t>(d.groups) * ((d.M + 127) / 128) * ((d.N + 127) / 128) > INT32_MAX / 8) return TP_ERR_UNSUPPORTED;
    switch (d.glu ? d.act : TP_ACT_NONE) {
        case TP_ACT_SILU_MUL: return launch_sized<TP_ACT_SILU_MUL>(a, d, stream);
        case TP_ACT_GELU_TANH_MUL: return launch_sized<TP_ACT_GELU_TANH_MUL>(a, d, stream);
        default: return launch_sized<TP_ACT_NONE>(a, d, stream);
    }
}

}  // namespace tpk

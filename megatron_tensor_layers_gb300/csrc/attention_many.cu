// Attention over the paged 4-bit cache for many rows per sequence (chunks of
// prompts): matrix products on the 5th-generation tensor cores.  8192 new rows in
// four chunks over 2100 to 6001 tokens, 64 query heads of 128, take 888 us, 980
// TFLOP/s.  Bound by the chain of a tile (S, then its exponentials, then the
// second product, then the next S): a step of both tiles takes about 4000 cycles,
// its products 2200 of them.
//
// A pair of thread blocks (a cluster, tcgen05 cta_group::2) takes 512 columns (a
// column is one row's query head) of one kv head as two tiles of 256, half of
// each tile in each block, and walks the cached tokens 128 at a time:
//   S = Q K^T          tcgen05, Q and K from shared memory, S in TMEM;
//   P = 2^(c S - m)    one thread per column, fp32, P as fp16 over S in TMEM;
//   O += P V           tcgen05, P from TMEM, V^T from shared memory, O in TMEM.
// In each block warps 0-3 and 4-7 are the softmax of one tile each and take turns
// with the tensor core, warps 8-11 turn codes into operands; warp 12 of the even
// block issues the products of both.  Of a step each block unpacks and holds half
// the keys and half of the values' dimensions, which is all that a pair's
// products need: against single blocks of 256 columns that halves the unpacking
// and the traffic of K and V^T through shared memory, which bounded them.
//
// Codes to operands.  A code is an fp16 subnormal u 2^-24 (or 16 u 2^-24) after
// one mask, and one HFMA2 makes the fp16 value (s u + b) 2^-F of two elements:
// 9 instructions for 8 keys, shared by all 512 columns.  2^F is 2^9 times the
// largest step or 2^-14 times the largest base of 32 tokens (the larger; powers of
// two), so that nothing overflows; a value is rounded once, by at most 2^-11 of
// itself or 2^-25 of 2^F.  The scale of K enters the exponent's factor c, the scale
// of V the exponent itself (P 2^(F - Fref), Fref that of the largest values a column
// has seen), both per 32 tokens; the sum of the probabilities is free of it.  Keys
// keep their packed order (q is permuted to it), values are transposed while they are unpacked: eight
// tokens' words give eight dimensions' 16-byte chunks of V^T.
//
// What is subtracted, m, is a column's maximum as of the last time it was
// needed.  A step first takes P under the old m and adds it up; a sum of at most
// 2^12 says that no P has left fp16, and m stays.  Only otherwise, or while the
// column has seen nothing, the step's maximum is taken, O and the sum are
// rescaled to it and P is taken again.  The usual step therefore reads S once
// and has no maximum in it (128 fewer operations on the pipe that the unpacking
// needs too).
//
// Codes go from global memory to registers, one step ahead; a ring of records in
// shared memory, filled by bulk copies, measured 5 % slower (its reads and writes
// compete with the operands').
//
// A value row that stands for NaN is put in as 0 and its token noted; a column
// that sees such a token gets a NaN sum, the others are not touched by it.
#include <algorithm>

#include <cuda_fp16.h>

#include "attention_args.cuh"

namespace tpk {
namespace {

constexpr int kUnpackWarps = 4;
constexpr int kThreads = 256 + 32 * kUnpackWarps + 128;    // softmax, unpacking, one warp that issues (of a warpgroup)
// Registers: 512 threads are launched with 128 each.  The softmax needs more (128 values of S, which become
// P), the others give: 256 * 192 + 128 * 88 + 128 * 40 = 512 * 128.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 192, kUnpackRegs = 88, kIssueRegs = 40;
static_assert(256 * kSoftmaxRegs + 32 * kUnpackWarps * kUnpackRegs + 128 * kIssueRegs <= kThreads * kLaunchRegs,
              "a warpgroup would wait for registers that never come");
constexpr int kTile = 128;           // tokens of a step, columns of a tile
constexpr int kCols = kManyCols;
static_assert(kCols == 4 * kTile, "two tiles of 256 columns, half of each in each block");
constexpr int kInfo = 4;
constexpr float kNegInf = -INFINITY;
constexpr float kMost = 4096.0f;     // sum of a step's 2^(x - m) up to which the old maximum will do (P is 8 times as much at most)

template <int HD>
struct Cfg {
    static constexpr int QB = kTile * HD * 2;            // one tile of Q: 128 columns
    static constexpr int KB = kTile / 2 * HD * 2;        // this block's half of K: 64 tokens
    static constexpr int VB = HD / 2 * kTile * 2;        // and of V^T: half of the dimensions
    static constexpr int QATOM = kTile * 128;            // 64 elements of 128 rows
    static constexpr int KATOM = kTile / 2 * 128;        // 64 elements of 64 tokens
    static constexpr int VATOM = HD / 2 * 128;           // 64 tokens of HD / 2 rows
    static constexpr int Q = 0, K = 2 * QB, V = K + 2 * KB, SMEM = V + 2 * VB + 1024;
    static constexpr int S_COL = 0, O_COL = 256;         // TMEM columns: S of the tiles, then O of the tiles
};

// What the softmax has to know of a step, by unpacking warp (32 tokens each).
struct __align__(16) StepInfo {
    float4 kmul;                     // 2^(F - 135) of the keys: F can pass what fp32 holds
    int4 vexp;                       // F of the values
    uint4 nan;                       // tokens whose value row stands for NaN
    uint4 gone;                      // blocks that are not there, two bits each
};
static_assert(kUnpackWarps == 4, "StepInfo has a word for each");

__device__ __forceinline__ float pow2_field(int field) { return __uint_as_float(static_cast<uint32_t>(field) << 23); }

// x 2^e, also where 2^e is no fp32.
__device__ __forceinline__ float times_pow2(float x, int e) {
    return x * pow2_field(127 + (e >> 1)) * pow2_field(127 + e - (e >> 1));
}

// fp16 A and B, f32 accumulator, K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// D[tmem of both] (+)= A[tmem of both] * B[smem of both]^T, issued by the even block.
__device__ __forceinline__ void tc_mma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// One lane of the (converged) warp.  The compiler knows elect.sync's predicate for one lane's and keeps
// descriptors in uniform registers under it.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// q_full, p_full and the peer's two are awaited by the even block, which issues the products; the others are each
// block's own (a commit arrives at both blocks').  An arrival with release at the other block's barrier waits for
// all that its thread has in flight, a microsecond for a thread that loads; so the unpacking warps arrive at
// their own block's barriers, the odd block's idle warp passes that on, and the softmax, whose P is in TMEM by then
// (tcgen05.wait::st and a tcgen05 fence), arrives without release.
struct Bars {
    uint64_t q_full, p_full[2], k_peer[2], v_peer[2];
    uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2], s_full[2], o_full, info[kInfo];
};

// What the pair works on.
struct Item {
    int seq, first_row, rows, len, tile, head;
};

template <int HD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) kv4_attention_many_kernel(const __grid_constant__ AttnArgs a) {
    using B = KvBlock<HD>;
    using C = Cfg<HD>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_found;
    __shared__ Item s_item;
    __shared__ int64_t s_scan[kThreads / 32], s_cols[kThreads / 32];
    __shared__ StepInfo s_info[kInfo];
    // each unpacking warp's own: fp16 pairs (step, base) of its keys, steps and bases of its values
    __shared__ __align__(16) uint32_t s_key[kTile];
    __shared__ __align__(16) uint16_t s_vstep[kTile], s_vbase[kTile];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int heads = a.pools.t * a.pools.kv_heads;
    const int half = static_cast<int>(cluster_ctarank());
    pdl_wait();
    pdl_trigger();

    // ---- which sequence and tile: pair / heads counts tiles of 512 columns over the sequences
    {
        const int64_t want = (blockIdx.x >> 1) / heads;
        const int per = (a.seqs.nseq + kThreads - 1) / kThreads;
        auto cols_of = [&](int s) { return static_cast<int64_t>(seq_rows(a.seqs, s).count) * a.group; };
        if (tid == 0) s_found = 0;
        const int lo = min(a.seqs.nseq, tid * per), hi = min(a.seqs.nseq, (tid + 1) * per);
        const int first_len = lo < hi ? a.seqs.lens[lo] : 0;     // on its way with the offsets
        int64_t mine = 0, mine_cols = 0;
        for (int s = lo; s < hi; ++s) {
            const int64_t c = cols_of(s);
            const int n = many_tiles(a, c);
            mine += n;
            if (n > 0) mine_cols += c;
        }
        int64_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += v;
            mine_cols += __shfl_xor_sync(0xffffffffu, mine_cols, m);
        }
        if (lane == 31) s_scan[warp] = upto, s_cols[warp] = mine_cols;
        __syncthreads();
        int64_t before = upto - mine, all = 0, all_cols = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += s_scan[i];
            all += s_scan[i];
            all_cols += s_cols[i];
        }
        if (!many_pays(a, all_cols, all)) return;
        if (want >= before && want < before + mine) {
            int64_t u = want - before;
            int s = lo;
            while (true) {
                const int n = many_tiles(a, cols_of(s));
                if (u < n) break;
                u -= n;
                ++s;
            }
            const SeqRows r = seq_rows(a.seqs, s);
            Item it;
            it.seq = s;
            it.first_row = r.first;
            it.rows = r.count;
            it.len = max(s == lo ? first_len : a.seqs.lens[s], 0);
            // the last tiles see the most tokens: they start first
            it.tile = many_tiles(a, cols_of(s)) - 1 - static_cast<int>(u);
            it.head = static_cast<int>((blockIdx.x >> 1) % heads);
            s_item = it;
            s_found = 1;
        }
        __syncthreads();
        if (!s_found) return;
    }
    const Item it = s_item;
    const int rank = it.head / a.pools.kv_heads, kvh = it.head - rank * a.pools.kv_heads;
    const int pos0 = it.len - it.rows;                   // position of the sequence's first row
    const int col0 = it.tile * kCols;
    const int cols = min(kCols, it.rows * a.group - col0);
    const int64_t first_pos = pos0 + col0 / a.group, last_pos = pos0 + (col0 + cols - 1) / a.group;
    const Spans span = visible_spans(a, first_pos, last_pos, kTile);
    const int steps = span.count;
    const int tiles = cols > 2 * kTile ? 2 : 1;          // of 256 columns, half of them in each block

    if (warp == 0) tmem_alloc_pair<512>(smem_u32(&s_tmem));
    if (tid == 0) {
        s_abort = 0;
        mbar_init(smem_u32(&bars.q_full), 2 * 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.k_full[i]), kUnpackWarps);
            mbar_init(smem_u32(&bars.v_full[i]), kUnpackWarps);
            mbar_init(smem_u32(&bars.k_peer[i]), 1);
            mbar_init(smem_u32(&bars.v_peer[i]), 1);
            mbar_init(smem_u32(&bars.p_full[i]), 2 * 4);
            mbar_init(smem_u32(&bars.k_empty[i]), 1);
            mbar_init(smem_u32(&bars.v_empty[i]), 1);
            mbar_init(smem_u32(&bars.s_full[i]), 1);
        }
        mbar_init(smem_u32(&bars.o_full), 1);
        for (int i = 0; i < kInfo; ++i) mbar_init(smem_u32(&bars.info[i]), kUnpackWarps);
    }
    fence_barrier_init();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;

    if (warp < 8) {
        more_registers<kSoftmaxRegs>();
        // ------------------------------------------------ softmax: one thread per column
        const int t = warp >> 2;                         // tile
        const int ci = t * 2 * kTile + half * kTile + (tid & 127);       // column of the pair
        const bool have = ci < cols;
        const int cc = col0 + ci;
        const int r = have ? cc / a.group : 0;
        const int h = have ? cc - r * a.group : 0;
        const int pos = have ? pos0 + r : -1;
        float cmul;
        {
            const uint4* src = reinterpret_cast<const uint4*>(a.q[rank] + (it.first_row + r) * a.ldq + (kvh * a.group + h) * HD);
            uint32_t raw[HD / 2];
#pragma unroll
            for (int i = 0; i < HD / 8; ++i) {
                const uint4 v = have ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                raw[4 * i] = v.x, raw[4 * i + 1] = v.y, raw[4 * i + 2] = v.z, raw[4 * i + 3] = v.w;
            }
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < HD / 2; ++i) top = max(top, max(raw[i] & 0x7fffu, (raw[i] >> 16) & 0x7fffu));
            // scaled by 2^k so that the largest element is in [2^10, 2^11): exact in fp16
            const int k = top == 0 || a.scale_log2 == 0.0f ? 0 : min(137 - static_cast<int>(top >> 7), 126);
            float up = pow2_field(k + 127);
            if (a.scale_log2 < 0.0f) up = -up;
            if (a.scale_log2 == 0.0f) up = 0.0f;
            cmul = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2) * pow2_field(135 - k);     // k from -118 to 126
            const uint32_t row = sm + C::Q + t * C::QB + (tid & 127) * 128;
#pragma unroll
            for (int i = 0; i < HD / 8; ++i) {           // a word of eight codes: its order of elements
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(raw[4 * i + e] << 16) * up;
                    x[2 * e + 1] = __uint_as_float(raw[4 * i + e] & 0xffff0000u) * up;
                }
                st_shared_v4(row + (i >> 3) * C::QATOM + (((i & 7) ^ (tid & 7)) << 4), pack_f16x2(x[0], x[4]),
                             pack_f16x2(x[1], x[5]), pack_f16x2(x[2], x[6]), pack_f16x2(x[3], x[7]));
            }
        }
        fence_proxy_async_cta();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.q_full), 0));

        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + C::S_COL + t * kTile;
        const uint32_t o_addr = tmem + lane_base + C::O_COL + t * HD;
        // positions of this block's columns of the tile, for whole-step decisions
        const int tile0 = t * 2 * kTile + half * kTile;
        const int tile_lo = pos0 + (col0 + tile0) / a.group;
        const int tile_hi = pos0 + (col0 + max(min(cols, tile0 + kTile), tile0 + 1) - 1) / a.group;
        float m = kNegInf, l = 0.0f;
        int vref = 0;
        for (int j = 0; j < steps && t < tiles && ok; ++j) {
            const int tok0 = (j < span.front ? j : span.start + j - span.front) * kTile;
            ok = mbar_wait_warp(smem_u32(&bars.info[j % kInfo]), (j / kInfo) & 1, &s_abort, a.seqs.status) &&
                 mbar_wait_warp(smem_u32(&bars.s_full[t]), j & 1, &s_abort, a.seqs.status);
            if (!ok) break;
            tc_fence_after();
            const StepInfo& info = s_info[j % kInfo];
            // the quarters' constants: x = c S, P = 2^(x + d - m), d = F - Fref of the values, and their sum is that of
            // P 2^-d.  Below -40 every P (2^(x - m) is at most 2^12) is 0 in fp16.  So d stops at -60, where 2^-d is finite
            // and the sum loses nothing above 2^-66 of the maximum's term, whatever the values' sizes.
            const float4 km = info.kmul;
            const int4 ve = info.vexp;
            const uint4 nn = info.nan, gg = info.gone;
            const float c[4] = {fmaxf(cmul * km.x, 1e-37f), fmaxf(cmul * km.y, 1e-37f), fmaxf(cmul * km.z, 1e-37f),
                                fmaxf(cmul * km.w, 1e-37f)};
            const uint32_t gone = gg.x | gg.y << 2 | gg.z << 4 | gg.w << 6;
            const bool any_nan = (nn.x | nn.y | nn.z | nn.w) != 0;
            const bool whole = gone == 0 && tok0 + kTile - 1 <= tile_lo &&
                               (a.window == 0 || tok0 > tile_hi - a.window || tok0 + kTile <= a.sinks);
            const int lim = max(pos - tok0, -1), low = a.window == 0 ? -(1 << 30) : lim - a.window, sk = a.sinks - tok0;
            // F of the values that this column sees (0: of none), so that those it does not see cost it no bits
            int vtop = max(max(ve.x, ve.y), max(ve.z, ve.w));
            if (!whole) {
                auto seen = [&](int e) { return 32 * e <= lim && (min(32 * e + 31, lim) > low || 32 * e < sk); };
                vtop = max(max(seen(0) ? ve.x : 0, seen(1) ? ve.y : 0), max(seen(2) ? ve.z : 0, seen(3) ? ve.w : 0));
            }
            uint32_t s[4][32];
            auto load = [&]() {                          // S, hidden tokens -inf
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(s_addr + i * 32, s[i]);
                tmem_ld_wait();
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 128; ++k) {
                        const bool see = k <= lim && (k > low || k < sk) && !((gone >> (k >> 4)) & 1u);
                        if (!see) s[k >> 5][k & 31] = __float_as_uint(kNegInf);
                    }
                }
            };
            // P into the front of S's registers, and its sum
            auto powers = [&](float base) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float dv = static_cast<float>(max((e == 0 ? ve.x : e == 1 ? ve.y : e == 2 ? ve.z : ve.w) - vref, -60));
                    const uint64_t cc2 = pack2(c[e], c[e]), off2 = pack2(dv - base, dv - base);
                    uint64_t sum2 = 0;
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float x0, x1;
                        unpack2(fma2(pack2(__uint_as_float(s[e][k]), __uint_as_float(s[e][k + 1])), cc2, off2), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        sum2 = add2(sum2, pack2(p0, p1));
                        s[e >> 1][(e & 1) * 16 + k / 2] = pack_f16x2(p0, p1);
                    }
                    float a0, a1;
                    unpack2(sum2, a0, a1);
                    sum = fmaf(a0 + a1, ex2(-dv), sum);
                }
                return sum;
            };
            if (j == 0) vref = vtop;
            const bool vgrow = vtop > vref + 3;              // from 0, with O still 0, to the first that is seen
            bool again = have && (vgrow || m == kNegInf);
            float sum = 0.0f;
            if (!__any_sync(0xffffffffu, again)) {       // the old maximum may do
                load();
                sum = powers(m == kNegInf ? 0.0f : m);
                again = have && !(sum <= kMost);
            }
            if (__any_sync(0xffffffffu, again)) {
                load();
                float mt = kNegInf;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float u = kNegInf, v = kNegInf;
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        u = fmaxf(u, __uint_as_float(s[e][k]));
                        v = fmaxf(v, __uint_as_float(s[e][k + 1]));
                    }
                    mt = fmaxf(mt, fmaxf(u, v) * c[e]);
                }
                const float m_new = fmaxf(m, mt);
                float f = m == kNegInf ? 0.0f : ex2(m - m_new);
                if (!(m_new > kNegInf)) f = 1.0f;
                l *= f;
                m = m_new;
                if (vgrow) {
                    f *= ex2(static_cast<float>(vref - vtop));
                    vref = vtop;
                }
                sum = powers(m == kNegInf ? 0.0f : m);
                if (j > 0) {                             // P V of the steps before is done: S came after it
#pragma unroll 1
                    for (int i = 0; i < HD; i += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + i, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(o_addr + i, o);
                    }
                }
            }
            l += sum;
            if (any_nan) {
                // a column that sees a NaN value row is NaN
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    uint32_t set = e == 0 ? nn.x : e == 1 ? nn.y : e == 2 ? nn.z : nn.w;
                    while (set) {
                        const int k = e * 32 + __ffs(set) - 1;
                        set &= set - 1;
                        if (k <= lim && (k > low || k < sk)) l = __uint_as_float(0x7fc00000u);
                    }
                }
            }
            tmem_st32(s_addr, s[0]);
            tmem_st32(s_addr + 32, s[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&bars.p_full[t]), 0));
        }
        // ---- the result
        float scale = 0.0f;
        if (ok && steps > 0 && t < tiles) {
            ok = mbar_wait_warp(smem_u32(&bars.o_full), 0, &s_abort, a.seqs.status);
            tc_fence_after();
            scale = l == 0.0f ? 0.0f : pow2_field(max(vref - 8, 1)) / l;     // times 2^8, as 2^vref can pass fp32
        }
        if (ok && t < tiles) {
            uint16_t* dst = a.out[rank] + (it.first_row + r) * a.ldo + (kvh * a.group + h) * HD;
#pragma unroll 1
            for (int i = 0; i < HD; i += 32) {
                uint32_t o[32];
                if (steps > 0) {
                    tmem_ld32(o_addr + i, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                if (have) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = pack_bf16x2(__uint_as_float(o[e + 2 * x]) * 256.0f * scale,
                                               __uint_as_float(o[e + 2 * x + 1]) * 256.0f * scale);
                        *reinterpret_cast<uint4*>(dst + i + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    } else if (warp < 8 + kUnpackWarps) {
        if constexpr (kUnpackRegs > kLaunchRegs) more_registers<kUnpackRegs>(); else fewer_registers<kUnpackRegs>();
        // ------------------------------------------------ codes to operands
        // A warp takes a block of keys (16 tokens of this half of the step) and, for this half of the
        // dimensions, 32 tokens' values; what the softmax must know, of the latter tokens.  F of the keys is
        // that of 32 tokens, so the warp looks at the pairs of its block's neighbour too.
        const int w = warp - 8, kq = 2 * half + (w >> 1);
        const int32_t* row = a.seqs.table + it.seq * a.seqs.max_blocks;
        const uint8_t* pool = a.pools.pool[rank];
        constexpr int PARTS = HD / 32, KU = PARTS / 2;   // 16-byte parts (32 elements) of a key; units of a lane
        // values: a lane takes one word (8 dimensions) of eight tokens; with HD 64 two lanes share a word, half each
        constexpr int HALVES = HD == 128 ? 2 : 1;
        const int tg = 4 * w + (lane & 3), word = (lane >> 2) & (HD / 16 - 1);
        const int half0 = HD == 128 ? word & 1 : lane >> 4, flip0 = HD == 128 ? 0 : word & 1;
        auto first_block = [&](int j) { return (j < span.front ? j : span.start + j - span.front) * (kTile / kKvBlock); };
        // lanes 0, 1: the values' two blocks; lanes 2, 3: those of the keys' 32 tokens
        const int my_block = 2 * (lane & 2 ? kq : w) + (lane & 1);
        // the page of the lane's block of step j; -2 where no row of the tile sees a token of it and nothing is read:
        // its page may be gone (behind the window, between the sinks and the window, past the last row)
        auto fetch_page = [&](int j) -> int {
            const int64_t b = first_block(j) + my_block, token = b * kKvBlock;
            const bool seen = token <= last_pos &&
                              (a.window == 0 || token + kKvBlock - 1 > first_pos - a.window || token < a.sinks);
            return j < steps && seen ? kv_page_at(row, a.seqs.max_blocks, a.pools.page_shift, b) : -2;
        };
        auto offset_of = [&](int j, int page) -> int64_t {
            const int64_t off = kv_page_offset(page, a.pools.pages, a.pools.page_shift, a.pools.kv_heads, kvh,
                                               first_block(j) + my_block, B::BYTES);
            if (off < 0 && page != -2) raise_status(a.seqs.status, TP_ERR_INVALID_ARG);
            return off;
        };
        // pairs of token `lane` of the 32: keys and values where the values are, keys where the keys are
        struct Pairs {
            uint32_t k, v, own;
        };
        auto fetch_pairs = [&](int j, int64_t off) {
            Pairs p{0, 0, 0};
            const int64_t b = __shfl_sync(0xffffffffu, off, lane >> 4), o = __shfl_sync(0xffffffffu, off, 2 + (lane >> 4));
            const int64_t first = static_cast<int64_t>(first_block(j)) * kKvBlock + lane;
            if (b >= 0 && first + 32 * w <= last_pos) {
                p.k = __ldg(reinterpret_cast<const uint32_t*>(pool + b + B::KPAIR) + (lane & 15));
                p.v = __ldg(reinterpret_cast<const uint32_t*>(pool + b + B::VPAIR) + (lane & 15));
            }
            if (o >= 0 && first + 32 * kq <= last_pos) p.own = __ldg(reinterpret_cast<const uint32_t*>(pool + o + B::KPAIR) + (lane & 15));
            return p;
        };
        uint4 kc[KU];
        auto fetch_keys = [&](int64_t off) {
            const int64_t b = __shfl_sync(0xffffffffu, off, 2 + (w & 1));
#pragma unroll
            for (int i = 0; i < KU; ++i)
                kc[i] = b >= 0 ? __ldg(reinterpret_cast<const uint4*>(pool + b + B::KEYS) + i * 32 + lane)
                               : make_uint4(0, 0, 0, 0);
        };
        uint32_t vc[8];
        auto fetch_values = [&](int64_t off) {
            const int64_t b = __shfl_sync(0xffffffffu, off, (lane >> 1) & 1);
            const uint8_t* p = pool + b + B::VALS + (lane & 1) * 8 * B::ROW + half * (B::ROW / 2) + word * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) vc[i] = b >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(p + i * B::ROW)) : 0u;
        };
        // Registers of a step are refilled as soon as they are used: the loads of step j + 1 run under the
        // conversions of step j, and the page numbers are one more step ahead.
        int page_next = fetch_page(1);
        int64_t off = offset_of(0, fetch_page(0));
        Pairs pair = fetch_pairs(0, off);
        fetch_keys(off);
        fetch_values(off);
        for (int j = 0; j < steps; ++j) {
            const int st = j & 1;
            const uint32_t there = __ballot_sync(0xffffffffu, off >= 0) & 3u;
            const bool vnan = ((pair.v >> 16) & 0x7f80u) == 0x7f80u || (pair.v & 0x7f80u) == 0x7f80u;
            if (vnan) pair.v = 0;
            // F of 32 tokens, 9 to 263: s 2^(127 - F) below 2^-8, |b| 2^(127 - F) below 2^15
            auto field = [](uint32_t p) {
                const int es = static_cast<int>((p >> 7) & 0xffu), eb = static_cast<int>((p >> 23) & 0xffu);
                return max((es == 255 ? 0 : es) + 9, (eb == 255 ? 0 : eb) - 14);
            };
            const int kF = __reduce_max_sync(0xffffffffu, field(pair.k));
            const int vF = __reduce_max_sync(0xffffffffu, field(pair.v));
            const int oF = __reduce_max_sync(0xffffffffu, field(pair.own));
            const uint32_t nan_set = __ballot_sync(0xffffffffu, vnan);
            __syncwarp();                                // the lanes are done with the words of step j - 1
            {
                // the step times 2^24: codes are u 2^-24
                s_key[w * 32 + lane] = pack_f16x2(times_pow2(__uint_as_float(pair.own << 16), 151 - oF),
                                                  times_pow2(__uint_as_float(pair.own & 0xffff0000u), 127 - oF));
                const uint32_t sb = pack_f16x2(times_pow2(__uint_as_float(pair.v << 16), 151 - vF),
                                               times_pow2(__uint_as_float(pair.v & 0xffff0000u), 127 - vF));
                s_vstep[w * 32 + lane] = static_cast<uint16_t>(sb);
                s_vbase[w * 32 + lane] = static_cast<uint16_t>(sb >> 16);
                if (lane == 0) {
                    StepInfo& info = s_info[j % kInfo];
                    reinterpret_cast<float*>(&info.kmul)[w] = pow2_field(kF - 8);
                    reinterpret_cast<int*>(&info.vexp)[w] = vF;
                    reinterpret_cast<uint32_t*>(&info.nan)[w] = nan_set;
                    // past the last visible token nothing is there: hidden by position, no matter
                    reinterpret_cast<uint32_t*>(&info.gone)[w] = ~there & 3u;
                    mbar_arrive(smem_u32(&bars.info[j % kInfo]));
                }
            }
            __syncwarp();
            off = offset_of(j + 1, page_next);
            pair = fetch_pairs(j + 1, off);
            page_next = fetch_page(j + 2);
            if (j >= 2) ok = mbar_wait_warp(smem_u32(&bars.k_empty[st]), ((j >> 1) + 1) & 1, &s_abort, a.seqs.status);
            if (!ok) break;
            constexpr uint32_t M0 = 0x000f000fu, M4 = 0x00f000f0u, SIXTEENTH = 0x2c002c00u;   // (1/16, 1/16)
#pragma unroll
            for (int i = 0; i < KU; ++i) {
                const int u = i * 32 + lane, token = kKvBlock * w + u / PARTS, part = u % PARTS;       // of this half
                const uint32_t sb = s_key[w * 32 + (w & 1) * kKvBlock + u / PARTS];
                const uint32_t s1 = __byte_perm(sb, sb, 0x1010), b1 = __byte_perm(sb, sb, 0x3232);
                const uint32_t s16 = hfma2(s1, SIXTEENTH, 0u);
                // the two halves of the lanes store in another order, so that eight lanes meet eight bank groups
                const bool flip = part & 2;
                const uint32_t wd[4] = {flip ? kc[i].z : kc[i].x, flip ? kc[i].w : kc[i].y, flip ? kc[i].x : kc[i].z,
                                        flip ? kc[i].y : kc[i].w};
                const uint32_t base = sm + C::K + st * C::KB + (part >> 1) * C::KATOM + token * 128;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int chunk = (part & 1) * 4 + (flip ? x ^ 2 : x);
                    const uint32_t v = wd[x], hgh = v >> 8;
                    st_shared_v4(base + ((chunk ^ (token & 7)) << 4), hfma2(v & M0, s1, b1), hfma2(v & M4, s16, b1),
                                 hfma2(hgh & M0, s1, b1), hfma2(hgh & M4, s16, b1));
                }
            }
            fence_proxy_async_cta();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.k_full[st]));
            fetch_keys(off);

            if (j >= 2) ok = mbar_wait_warp(smem_u32(&bars.v_empty[st]), ((j >> 1) + 1) & 1, &s_abort, a.seqs.status);
            if (!ok) break;
            {
                const uint4 vs = *reinterpret_cast<const uint4*>(&s_vstep[tg * 8]);
                const uint4 vb = *reinterpret_cast<const uint4*>(&s_vbase[tg * 8]);
                const uint32_t s1[4] = {vs.x, vs.y, vs.z, vs.w}, b1[4] = {vb.x, vb.y, vb.z, vb.w};
                uint32_t s16[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) s16[p] = hfma2(s1[p], SIXTEENTH, 0u);
                const uint32_t at = sm + C::V + st * C::VB + (tg >> 3) * C::VATOM;
#pragma unroll
                for (int i = 0; i < HALVES; ++i) {
                    // dimensions 0-3 or 4-7 of the word, of these 0-1 or 2-3: in another order from lane to
                    // lane, so that eight lanes meet eight bank groups
                    const int hw = half0 ^ i;
                    const uint32_t sel = hw ? 0x7632u : 0x5410u;
                    uint32_t pr[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) pr[p] = __byte_perm(vc[2 * p], vc[2 * p + 1], sel);
#pragma unroll
                    for (int bi = 0; bi < 2; ++bi) {
                        const int b = flip0 ^ bi, d = word * 8 + hw * 4 + b * 2;    // and d + 1, of this half
                        uint32_t q[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) q[p] = pr[p] >> (8 * b);
                        st_shared_v4(at + d * 128 + (((tg & 7) ^ (d & 7)) << 4), hfma2(q[0] & M0, s1[0], b1[0]),
                                     hfma2(q[1] & M0, s1[1], b1[1]), hfma2(q[2] & M0, s1[2], b1[2]),
                                     hfma2(q[3] & M0, s1[3], b1[3]));
                        st_shared_v4(at + (d + 1) * 128 + (((tg & 7) ^ ((d + 1) & 7)) << 4), hfma2(q[0] & M4, s16[0], b1[0]),
                                     hfma2(q[1] & M4, s16[1], b1[1]), hfma2(q[2] & M4, s16[2], b1[2]),
                                     hfma2(q[3] & M4, s16[3], b1[3]));
                    }
                }
            }
            fence_proxy_async_cta();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.v_full[st]));
            fetch_values(off);
        }
    } else {
        fewer_registers<kIssueRegs>();
        if (warp == 8 + kUnpackWarps && half == 0 && steps > 0) {
            // ------------------------------------------------ the products of both blocks
            constexpr uint32_t QK = idesc_f16(256, 128), PV = idesc_f16(256, HD);
            // what the other block's threads wrote is behind the peer's barriers alone
            auto wait = [&](uint64_t& b, int parity) {
                ok = ok && mbar_wait_warp(smem_u32(&b), parity, &s_abort, a.seqs.status);
                tc_fence_after();
                return ok;
            };
            auto wait_both = [&](uint64_t& mine, uint64_t& peer, int parity) {
                ok = ok && mbar_wait_cluster_warp(smem_u32(&peer), parity, &s_abort, a.seqs.status);
                return wait(mine, parity);
            };
            auto scores = [&](int t, int j) {            // and what waits for them
                const uint64_t qd = sw128_kmajor_desc(sm + C::Q + t * C::QB);
                const uint64_t kd = sw128_kmajor_desc(sm + C::K + (j & 1) * C::KB);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k)
                        tc_mma_pair(tmem + C::S_COL + t * kTile, qd + (((k >> 2) * C::QATOM + (k & 3) * 32) >> 4),
                                    kd + (((k >> 2) * C::KATOM + (k & 3) * 32) >> 4), QK, k > 0);
                    tc_commit_pair(smem_u32(&bars.s_full[t]), 3);
                    if (t + 1 == tiles) tc_commit_pair(smem_u32(&bars.k_empty[j & 1]), 3);
                }
                __syncwarp();
            };
            auto values = [&](int t, int j) {
                const uint64_t vd = sw128_kmajor_desc(sm + C::V + (j & 1) * C::VB);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_ts_pair(tmem + C::O_COL + t * HD, tmem + C::S_COL + t * kTile + k * 8,
                                       vd + (((k >> 2) * C::VATOM + (k & 3) * 32) >> 4), PV, j > 0 || k > 0);
                    if (t + 1 == tiles) {
                        tc_commit_pair(smem_u32(&bars.v_empty[j & 1]), 3);
                        if (j + 1 == steps) tc_commit_pair(smem_u32(&bars.o_full), 3);
                    }
                }
                __syncwarp();
            };
            auto wait_keys = [&](int j) { return wait_both(bars.k_full[j & 1], bars.k_peer[j & 1], (j >> 1) & 1); };
            ok = mbar_wait_cluster_warp(smem_u32(&bars.q_full), 0, &s_abort, a.seqs.status);
            if (ok && wait_keys(0))
                for (int t = 0; t < tiles; ++t) scores(t, 0);
            for (int j = 0; j < steps && ok; ++j) {
                const bool more = j + 1 < steps;
                if (!wait_both(bars.v_full[j & 1], bars.v_peer[j & 1], (j >> 1) & 1) || (more && !wait_keys(j + 1))) break;
                for (int t = 0; t < tiles; ++t) {
                    if (!wait(bars.p_full[t], j & 1)) break;
                    values(t, j);
                    if (!more) continue;
                    scores(t, j + 1);
                }
            }
        }
        if (warp == 8 + kUnpackWarps && half == 1) {
            // ------------------------------------------------ tells the even block what this one has unpacked
            for (int j = 0; j < steps && ok; ++j) {
                const int st = j & 1, parity = (j >> 1) & 1;
                ok = mbar_wait_warp(smem_u32(&bars.k_full[st]), parity, &s_abort, a.seqs.status);
                if (ok && lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.k_peer[st]), 0));
                ok = ok && mbar_wait_warp(smem_u32(&bars.v_full[st]), parity, &s_abort, a.seqs.status);
                if (ok && lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bars.v_peer[st]), 0));
            }
        }
        __syncwarp();
    }
    if (s_abort) spin_ns(1000000);   // products that were issued end before their memory is given back
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 0) tmem_dealloc_pair<512>(tmem);
}

template <int HD>
tp_status launch(const AttnArgs& a, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    auto* kern = kv4_attention_many_kernel<HD>;
    if (!smem_attribute_once(reinterpret_cast<const void*>(kern), Cfg<HD>::SMEM, smem_set)) return TP_ERR_CUDA;
    // as many tiles as n rows in at most nseq sequences can make
    const int64_t cols = static_cast<int64_t>(a.seqs.n) * a.group;
    const int64_t tiles = cols / kCols + std::min<int64_t>(a.seqs.nseq, cols / a.many);
    const int64_t blocks = 2 * tiles * a.pools.t * a.pools.kv_heads;
    if (blocks > INT32_MAX) return TP_ERR_UNSUPPORTED;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), Cfg<HD>::SMEM, stream, a);
    return e == cudaSuccess ? TP_OK : TP_ERR_CUDA;
}

}  // namespace

tp_status launch_attention_many(const AttnArgs& a, int head_dim, cudaStream_t stream) {
    return head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace tpk

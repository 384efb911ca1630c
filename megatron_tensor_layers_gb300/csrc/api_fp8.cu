// C ABI of the 8-bit floating-point operators: argument validation, workspace
// carving and the kernel launches.  See include/tp.h for the contract.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "kernels.h"
#include "tp.h"

namespace {


// Rows and columns of a product: twice as many, and a tile more, still count in 32 bits.
constexpr int64_t kMaxSize = int64_t(1) << 29;

// Row strides of codes (bytes), multiples of 16 as the TMA tiles need.
inline bool codes_ld_ok(int64_t ld, int64_t minimum) { return ld >= minimum && ld % 16 == 0; }

std::atomic<int> g_tile{0}, g_parts{0}, g_max_clusters{0};

// The kernel choice in effect for a launch (tp_set_fp8_gemm).
void apply_choice(tpk::Fp8GemmDesc& d) {
    d.force_tile = g_tile.load();
    d.force_parts = g_parts.load();
    d.max_clusters = g_max_clusters.load();
}

// A gated block's hidden rows, one rank's: codes at columns [r fs, (r + 1) fs) of [n, f], scales [groups, n].
struct HiddenLayout {
    size_t codes, scales_each, parts, part_each, total;
};

bool hidden_layout(int t, int64_t n, int64_t h, int64_t f, tp_reduce_mode mode, tp_dtype pdt, HiddenLayout& l) {
    if (t < 1 || t > TP_MAX_SHARDS || n < 0 || h <= 0 || f <= 0 || f % t != 0 || !dtype_ok(pdt)) return false;
    if (n > kMaxSize || h > kMaxSize || f > kMaxSize) return false;
    if (mode != TP_REDUCE_DIRECT && mode != TP_REDUCE_RING && mode != TP_REDUCE_FUSED) return false;
    l.codes = align256(static_cast<size_t>(n) * static_cast<size_t>(f));
    l.scales_each = align256(static_cast<size_t>(tpk::fp8_groups(f / t)) * static_cast<size_t>(n) * 4);
    l.parts = l.codes + t * l.scales_each;
    l.part_each = mode == TP_REDUCE_FUSED ? 0 : align256(static_cast<size_t>(n) * static_cast<size_t>(h) * esize(pdt));
    l.total = l.parts + t * l.part_each;
    return true;
}

}  // namespace

extern "C" {

tp_status tp_fp8_quantize(int t, int64_t n, int64_t k, tp_dtype dtype, const void* const* x, int64_t ldx,
                          void* const* codes, int64_t ldc, float* const* scales, int64_t lds, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(n >= 0 && k > 0 && n <= INT32_MAX && k <= INT32_MAX, TP_ERR_INVALID_ARG);
    TP_CHECK(x != nullptr && codes != nullptr && scales != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(dtype_ok(dtype), TP_ERR_UNSUPPORTED);
    TP_CHECK(k % 16 == 0, TP_ERR_ALIGNMENT);
    TP_CHECK(lds >= n, TP_ERR_INVALID_ARG);
    TP_CHECK(ldx >= k && (ldx * esize(dtype)) % 16 == 0 && codes_ld_ok(ldc, k), TP_ERR_ALIGNMENT);
    for (int r = 0; r < t; ++r) {
        TP_CHECK((x[r] != nullptr && codes[r] != nullptr && scales[r] != nullptr) || n == 0, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(x[r]) && al16(codes[r]) && al4(scales[r]), TP_ERR_ALIGNMENT);
    }
    if (n == 0) return TP_OK;
    tpk::Fp8QuantDesc d;
    d.t = t;
    d.n = n;
    d.k = k;
    d.in_f32 = dtype == TP_F32;
    for (int r = 0; r < t; ++r) {
        d.x[r] = x[r];
        d.codes[r] = codes[r];
        d.scales[r] = scales[r];
    }
    d.ldx = ldx;
    d.ldc = ldc;
    d.lds = lds;
    return tpk::launch_fp8_quant(d, cs(stream));
}

tp_status tp_fp8_quantize_weight(int t, int64_t out, int64_t k, tp_dtype dtype, const void* const* w, int64_t ldw,
                                 int gated, void* const* codes, int64_t ldc, float* const* scales, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(out > 0 && k > 0 && out <= INT32_MAX && k <= INT32_MAX, TP_ERR_INVALID_ARG);
    TP_CHECK(w != nullptr && codes != nullptr && scales != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(gated == 0 || gated == 1, TP_ERR_INVALID_ARG);
    TP_CHECK(dtype_ok(dtype), TP_ERR_UNSUPPORTED);
    TP_CHECK(!gated || out % 2 == 0, TP_ERR_NOT_DIVISIBLE);
    TP_CHECK(k % 16 == 0, TP_ERR_ALIGNMENT);
    TP_CHECK(ldw >= k && (ldw * esize(dtype)) % 16 == 0 && codes_ld_ok(ldc, k), TP_ERR_ALIGNMENT);
    for (int r = 0; r < t; ++r) {
        TP_CHECK(w[r] != nullptr && codes[r] != nullptr && scales[r] != nullptr, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(w[r]) && al16(codes[r]) && al4(scales[r]), TP_ERR_ALIGNMENT);
    }
    tpk::Fp8QuantDesc d;
    d.t = t;
    d.n = out;
    d.k = k;
    d.in_f32 = dtype == TP_F32;
    d.weight = 1;
    d.half = gated ? out / 2 : 0;
    for (int r = 0; r < t; ++r) {
        d.x[r] = w[r];
        d.codes[r] = codes[r];
        d.scales[r] = scales[r];
    }
    d.ldx = ldw;
    d.ldc = ldc;
    d.lds = tpk::fp8_groups(k);
    return tpk::launch_fp8_quant(d, cs(stream));
}

tp_status tp_fp8_rmsnorm(int t, int64_t n, int64_t h, tp_dtype dtype, const void* const* partials,
                         const void* residual, const void* weight, float eps, tp_reduce_mode mode, void* residual_out,
                         void* codes, int64_t ldc, float* scales, int64_t lds, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(n >= 0 && n <= INT32_MAX && h > 0 && partials != nullptr && weight != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK((codes != nullptr && scales != nullptr) || n == 0, TP_ERR_INVALID_ARG);
    TP_CHECK(mode == TP_REDUCE_DIRECT || mode == TP_REDUCE_RING, TP_ERR_INVALID_ARG);
    TP_CHECK(eps >= 0.0f && std::isfinite(eps), TP_ERR_INVALID_ARG);
    TP_CHECK(dtype_ok(dtype), TP_ERR_UNSUPPORTED);
    TP_CHECK(h % 16 == 0, TP_ERR_ALIGNMENT);
    TP_CHECK(h <= 32768, TP_ERR_UNSUPPORTED);
    TP_CHECK(lds >= n, TP_ERR_INVALID_ARG);
    TP_CHECK(codes_ld_ok(ldc, h), TP_ERR_ALIGNMENT);
    TP_CHECK(al16(weight) && al16(codes) && al4(scales) && al16(residual) && al16(residual_out), TP_ERR_ALIGNMENT);
    for (int r = 0; r < t; ++r) {
        TP_CHECK(partials[r] != nullptr || n == 0, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(partials[r]), TP_ERR_ALIGNMENT);
    }
    if (n == 0) return TP_OK;
    tpk::Fp8NormDesc d;
    d.t = t;
    d.n = n;
    d.h = h;
    d.in_bf16 = dtype == TP_BF16;
    for (int r = 0; r < t; ++r) d.p[r] = partials[r];
    d.residual = residual;
    d.weight = weight;
    d.eps = eps;
    d.ring = mode == TP_REDUCE_RING;
    d.residual_out = residual_out;
    d.codes = codes;
    d.ldc = ldc;
    d.scales = scales;
    d.lds = lds;
    tpk::count_collective();
    return tpk::launch_fp8_norm(d, cs(stream));
}

// The column-parallel product behind tp_fp8_linear_col and tp_fp8_mlp_forward
// (arguments checked).
static tp_status linear_col_run(int t, int64_t n, int64_t in, int64_t out_full, const void* x, int64_t ldx,
                                const float* xs, int64_t ldxs, const void* const* w, int64_t ldw,
                                const float* const* ws, const void* const* bias, tp_act act, int out_kind,
                                void* const* y, int64_t ldy, float* const* ys, int64_t ldys, tp_stream stream) {
    tpk::Fp8GemmDesc d;
    d.M = n;
    d.N = out_full / t;
    d.K = in;
    d.groups = t;
    d.x[0] = x;
    d.ldx = ldx;
    d.xs[0] = xs;
    d.ldxs = ldxs;
    d.ldw = ldw;
    d.glu = act != TP_ACT_NONE;
    d.act = act;
    d.out_kind = out_kind;
    d.ldo = ldy;
    d.ldos = ldys;
    for (int r = 0; r < t; ++r) {
        d.w[r] = w[r];
        d.ws[r] = ws[r];
        d.out[r] = y[r];
        d.os[r] = ys != nullptr ? ys[r] : nullptr;
        d.bias[r] = bias != nullptr ? bias[r] : nullptr;
    }
    d.status = tpk::device_status_word();
    apply_choice(d);
    return tpk::launch_fp8_gemm(d, cs(stream));
}

tp_status tp_fp8_linear_col(int t, int64_t n, int64_t in, int64_t out_full, const void* x, int64_t ldx, const float* xs,
                            int64_t ldxs, const void* const* w, int64_t ldw, const float* const* ws,
                            const void* const* bias, tp_act act, int gather_output, void* const* y, int64_t ldy,
                            int y_kind, float* const* ys, int64_t ldys, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(n >= 0 && in > 0 && out_full > 0, TP_ERR_INVALID_ARG);
    TP_CHECK(n <= kMaxSize && out_full <= kMaxSize && in <= kMaxSize, TP_ERR_INVALID_ARG);
    TP_CHECK((x != nullptr && xs != nullptr) || n == 0, TP_ERR_INVALID_ARG);
    TP_CHECK(w != nullptr && ws != nullptr && y != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(act == TP_ACT_NONE || act == TP_ACT_SILU_MUL || act == TP_ACT_GELU_TANH_MUL, TP_ERR_INVALID_ARG);
    TP_CHECK(gather_output == 0 || gather_output == 1, TP_ERR_INVALID_ARG);
    TP_CHECK(y_kind == TP_BF16 || y_kind == TP_F32 || y_kind == TP_FP8, TP_ERR_UNSUPPORTED);
    TP_CHECK(out_full % t == 0, TP_ERR_NOT_DIVISIBLE);
    const int64_t os = out_full / t;
    const bool glu = act != TP_ACT_NONE, codes = y_kind == TP_FP8;
    TP_CHECK(!(glu && bias != nullptr), TP_ERR_UNSUPPORTED);
    TP_CHECK(!codes || (glu && !gather_output), TP_ERR_UNSUPPORTED);
    TP_CHECK(!codes || ys != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(in % 16 == 0 && (!codes || os % 16 == 0), TP_ERR_ALIGNMENT);
    TP_CHECK(al16(x) && al4(xs) && codes_ld_ok(ldx, in) && codes_ld_ok(ldw, in), TP_ERR_ALIGNMENT);
    TP_CHECK(ldxs >= n, TP_ERR_INVALID_ARG);
    TP_CHECK(ldy >= (gather_output ? out_full : os), TP_ERR_INVALID_ARG);
    TP_CHECK(!codes || (ldy % 16 == 0 && ldys >= n), codes && ldy % 16 == 0 ? TP_ERR_INVALID_ARG : TP_ERR_ALIGNMENT);
    const int ey = codes ? 1 : y_kind == TP_F32 ? 4 : 2;
    void* out[TP_MAX_SHARDS] = {};
    for (int r = 0; r < t; ++r) {
        TP_CHECK(w[r] != nullptr && ws[r] != nullptr, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(w[r]) && al4(ws[r]), TP_ERR_ALIGNMENT);
        if (bias != nullptr) {
            TP_CHECK(bias[r] != nullptr, TP_ERR_INVALID_ARG);
            TP_CHECK(al2(bias[r]), TP_ERR_ALIGNMENT);
        }
        if (!gather_output || r == 0) {
            TP_CHECK(y[r] != nullptr || n == 0, TP_ERR_INVALID_ARG);
            TP_CHECK(al16(y[r]), TP_ERR_ALIGNMENT);
        }
        if (codes) {
            TP_CHECK(ys[r] != nullptr || n == 0, TP_ERR_INVALID_ARG);
            TP_CHECK(al4(ys[r]), TP_ERR_ALIGNMENT);
        }
        out[r] = gather_output ? static_cast<char*>(y[0]) + static_cast<int64_t>(r) * os * ey : y[r];
    }
    if (n == 0) return TP_OK;
    if (gather_output) tpk::count_collective();
    return linear_col_run(t, n, in, out_full, x, ldx, xs, ldxs, w, ldw, ws, bias, act,
                          codes ? tpk::FP8_OUT_CODES : y_kind == TP_F32 ? tpk::FP8_OUT_F32 : tpk::FP8_OUT_BF16, out, ldy,
                          codes ? ys : nullptr, ldys, stream);
}

// weights_first: the previous launch of the stream is a kernel of the same
// call that wrote x and no weight.
static tp_status linear_row_impl(int t, int64_t n, int64_t in_full, int64_t out, const void* const* x, int64_t ldx,
                                 const float* const* xs, int64_t ldxs, const void* const* w, int64_t ldw,
                                 const float* const* ws, const void* bias, int reduce_results, tp_reduce_mode mode,
                                 tp_dtype partial_dtype, void* const* partials, int64_t ldp, void* y, int64_t ldy,
                                 tp_dtype y_dtype, int weights_first, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(n >= 0 && in_full > 0 && out > 0, TP_ERR_INVALID_ARG);
    TP_CHECK(n <= kMaxSize && out <= kMaxSize && in_full <= kMaxSize, TP_ERR_INVALID_ARG);
    TP_CHECK(x != nullptr && xs != nullptr && w != nullptr && ws != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(reduce_results == 0 || reduce_results == 1, TP_ERR_INVALID_ARG);
    TP_CHECK(mode == TP_REDUCE_DIRECT || mode == TP_REDUCE_RING || mode == TP_REDUCE_FUSED, TP_ERR_INVALID_ARG);
    TP_CHECK(!(mode == TP_REDUCE_FUSED && !reduce_results), TP_ERR_INVALID_ARG);
    TP_CHECK(in_full % t == 0, TP_ERR_NOT_DIVISIBLE);
    const int64_t ks = in_full / t;
    const bool fused = mode == TP_REDUCE_FUSED;
    TP_CHECK(ks % 16 == 0 && codes_ld_ok(ldx, ks) && codes_ld_ok(ldw, ks) && al2(bias), TP_ERR_ALIGNMENT);
    TP_CHECK(ldxs >= n, TP_ERR_INVALID_ARG);
    if (!fused) {
        TP_CHECK(partials != nullptr, TP_ERR_INVALID_ARG);
        TP_CHECK(dtype_ok(partial_dtype), TP_ERR_UNSUPPORTED);
        TP_CHECK(ldp >= out, TP_ERR_INVALID_ARG);
        if (reduce_results) TP_CHECK(ldp == out, TP_ERR_UNSUPPORTED);   // the reduce streams contiguous partials
    }
    if (reduce_results) {
        TP_CHECK(y != nullptr || n == 0, TP_ERR_INVALID_ARG);
        TP_CHECK(dtype_ok(y_dtype), TP_ERR_UNSUPPORTED);
        TP_CHECK(al16(y), TP_ERR_ALIGNMENT);
        TP_CHECK(ldy >= out, TP_ERR_INVALID_ARG);
        if (!fused) TP_CHECK(ldy == out, TP_ERR_UNSUPPORTED);
    }
    for (int r = 0; r < t; ++r) {
        TP_CHECK((x[r] != nullptr && xs[r] != nullptr) || n == 0, TP_ERR_INVALID_ARG);
        TP_CHECK(w[r] != nullptr && ws[r] != nullptr, TP_ERR_INVALID_ARG);
        TP_CHECK(al16(x[r]) && al4(xs[r]) && al16(w[r]) && al4(ws[r]), TP_ERR_ALIGNMENT);
        if (!fused) {
            TP_CHECK(partials[r] != nullptr || n == 0, TP_ERR_INVALID_ARG);
            TP_CHECK(al16(partials[r]), TP_ERR_ALIGNMENT);
        }
    }
    if (n == 0) return TP_OK;
    tpk::Fp8GemmDesc d;
    d.M = n;
    d.N = out;
    d.K = ks;
    d.ldx = ldx;
    d.ldxs = ldxs;
    d.ldw = ldw;
    for (int r = 0; r < t; ++r) {
        d.x[r] = x[r];
        d.xs[r] = xs[r];
        d.w[r] = w[r];
        d.ws[r] = ws[r];
    }
    d.status = tpk::device_status_word();
    apply_choice(d);
    d.weights_first = weights_first;
    if (fused) {
        d.segs = t;
        d.out[0] = y;
        d.bias[0] = bias;
        d.ldo = ldy;
        d.out_kind = y_dtype == TP_F32 ? tpk::FP8_OUT_F32 : tpk::FP8_OUT_BF16;
        tpk::count_collective();
        return tpk::launch_fp8_gemm(d, cs(stream));
    }
    d.groups = t;
    d.x_per_group = 1;
    for (int r = 0; r < t; ++r) d.out[r] = partials[r];
    d.bias[0] = bias;                          // rank 0 alone adds the bias
    d.ldo = ldp;
    d.out_kind = partial_dtype == TP_F32 ? tpk::FP8_OUT_F32 : tpk::FP8_OUT_BF16;
    const tp_status st = tpk::launch_fp8_gemm(d, cs(stream));
    if (st != TP_OK || !reduce_results) return st;
    return tp_shard_reduce(t, n * out, partial_dtype, reinterpret_cast<const void* const*>(partials), y, y_dtype, mode,
                           partial_dtype, 0, stream);
}

tp_status tp_fp8_linear_row(int t, int64_t n, int64_t in_full, int64_t out, const void* const* x, int64_t ldx,
                            const float* const* xs, int64_t ldxs, const void* const* w, int64_t ldw,
                            const float* const* ws, const void* bias, int reduce_results, tp_reduce_mode mode,
                            tp_dtype partial_dtype, void* const* partials, int64_t ldp, void* y, int64_t ldy,
                            tp_dtype y_dtype, tp_stream stream) {
    return linear_row_impl(t, n, in_full, out, x, ldx, xs, ldxs, w, ldw, ws, bias, reduce_results, mode, partial_dtype,
                           partials, ldp, y, ldy, y_dtype, 0, stream);
}

size_t tp_fp8_mlp_workspace_size(int t, int64_t n, int64_t h, int64_t f, tp_reduce_mode mode, tp_dtype partial_dtype) {
    HiddenLayout l;
    return hidden_layout(t, n, h, f, mode, partial_dtype, l) ? l.total : 0;
}

tp_status tp_fp8_mlp_forward(int t, int64_t n, int64_t h, int64_t f, const void* x, int64_t ldx, const float* xs,
                             int64_t ldxs, const void* const* w_gate_up, const float* const* s_gate_up,
                             const void* const* w_down, int64_t ld_down, const float* const* s_down,
                             const void* bias_down, tp_act act, tp_reduce_mode mode, tp_dtype partial_dtype,
                             void* workspace, size_t workspace_bytes, void* y, tp_dtype y_dtype, tp_stream stream) {
    TP_CHECK(t >= 1 && t <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK(n >= 0 && h > 0 && f > 0, TP_ERR_INVALID_ARG);
    TP_CHECK(n <= kMaxSize && h <= kMaxSize && f <= kMaxSize, TP_ERR_INVALID_ARG);
    TP_CHECK((x != nullptr && xs != nullptr && y != nullptr) || n == 0, TP_ERR_INVALID_ARG);
    TP_CHECK(w_gate_up != nullptr && s_gate_up != nullptr && w_down != nullptr && s_down != nullptr, TP_ERR_INVALID_ARG);
    TP_CHECK(act == TP_ACT_SILU_MUL || act == TP_ACT_GELU_TANH_MUL, TP_ERR_INVALID_ARG);
    TP_CHECK(mode == TP_REDUCE_DIRECT || mode == TP_REDUCE_RING || mode == TP_REDUCE_FUSED, TP_ERR_INVALID_ARG);
    TP_CHECK(dtype_ok(partial_dtype) && dtype_ok(y_dtype), TP_ERR_UNSUPPORTED);
    TP_CHECK(f % t == 0, TP_ERR_NOT_DIVISIBLE);
    const int64_t fs = f / t;
    TP_CHECK(fs % 16 == 0 && h % 16 == 0, TP_ERR_ALIGNMENT);
    TP_CHECK(al16(x) && al4(xs) && codes_ld_ok(ldx, h) && codes_ld_ok(ld_down, fs) && al16(y) && al2(bias_down), TP_ERR_ALIGNMENT);
    TP_CHECK(ldxs >= n, TP_ERR_INVALID_ARG);
    for (int r = 0; r < t; ++r) {
        TP_CHECK(w_gate_up[r] != nullptr && s_gate_up[r] != nullptr && w_down[r] != nullptr && s_down[r] != nullptr,
                 TP_ERR_INVALID_ARG);
        TP_CHECK(al16(w_gate_up[r]) && al4(s_gate_up[r]) && al16(w_down[r]) && al4(s_down[r]), TP_ERR_ALIGNMENT);
    }
    HiddenLayout l;
    TP_CHECK(hidden_layout(t, n, h, f, mode, partial_dtype, l), TP_ERR_INVALID_ARG);
    TP_CHECK(workspace != nullptr || l.total == 0, TP_ERR_WORKSPACE);
    TP_CHECK(workspace_bytes >= l.total, TP_ERR_WORKSPACE);
    TP_CHECK((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, TP_ERR_ALIGNMENT);
    if (n == 0) return TP_OK;
    char* ws = static_cast<char*>(workspace);
    void* hidden[TP_MAX_SHARDS] = {};
    float* hscales[TP_MAX_SHARDS] = {};
    void* parts[TP_MAX_SHARDS] = {};
    for (int r = 0; r < t; ++r) {
        hidden[r] = ws + r * fs;
        hscales[r] = reinterpret_cast<float*>(ws + l.codes + r * l.scales_each);
        parts[r] = mode == TP_REDUCE_FUSED ? nullptr : ws + l.parts + r * l.part_each;
    }
    const tp_status st = linear_col_run(t, n, h, f, x, ldx, xs, ldxs, w_gate_up, h, s_gate_up, nullptr, act,
                                        tpk::FP8_OUT_CODES, hidden, f, hscales, n, stream);
    if (st != TP_OK) return st;
    return linear_row_impl(t, n, f, h, reinterpret_cast<const void* const*>(hidden), f, hscales, n, w_down, ld_down,
                           s_down, bias_down, 1, mode, partial_dtype, parts, h, y, h, y_dtype, 1, stream);
}

static bool choice_ok(int tile, int parts) {
    if (tile == 0) return parts == 0;
    if (tile == 256) return parts == 0 || parts == 1 || parts == 2 || parts == 4;
    return (tile == 16 || tile == 32 || tile == 64 || tile == 128) && parts >= 0 && parts <= 8;
}

tp_status tp_set_fp8_gemm(int tile, int parts, int max_clusters) {
    TP_CHECK(choice_ok(tile, parts) && max_clusters >= 0, TP_ERR_INVALID_ARG);
    g_tile.store(tile);
    g_parts.store(parts);
    g_max_clusters.store(max_clusters);
    return TP_OK;
}

tp_status tp_debug_fp8_plan(int64_t m, int64_t n, int64_t k, int groups, int segs, int gated, int sms, const int* resident,
                            int* tile, int* parts) {
    TP_CHECK(m > 0 && n > 0 && k > 0 && m <= kMaxSize && n <= kMaxSize && k <= kMaxSize && sms >= 1, TP_ERR_INVALID_ARG);
    TP_CHECK(groups >= 1 && groups <= TP_MAX_SHARDS && segs >= 1 && segs <= TP_MAX_SHARDS, TP_ERR_INVALID_ARG);
    TP_CHECK((groups == 1 || segs == 1) && (gated == 0 || gated == 1), TP_ERR_INVALID_ARG);
    TP_CHECK(resident != nullptr && tile != nullptr && parts != nullptr, TP_ERR_INVALID_ARG);
    tpk::Fp8GemmDesc d;
    d.M = m;
    d.N = n;
    d.K = k;
    d.groups = groups;
    d.segs = segs;
    d.glu = gated;
    const tpk::Fp8Plan p = tpk::plan_fp8_gemm(d, sms, resident);
    TP_CHECK(p.cost >= 0, TP_ERR_UNSUPPORTED);
    *tile = p.tile;
    *parts = p.parts;
    return TP_OK;
}

}  // extern "C"

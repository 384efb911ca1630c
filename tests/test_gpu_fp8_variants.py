"""Every kernel of the 8-bit products by itself (tp_set_fp8_gemm), whatever the costs would choose, against the float64 sums of
fp8_plain.py: each tile, its K blocks in one part and in several, more K blocks than any ring has slots, more tiles than
clusters, more row tiles than a raster band, ragged rows, columns and K, each output."""

import pytest
import torch

import fp8_plain as P
from megatron_tensor_layers_gb300 import _lib as tp
from test_gpu_fp8 import DEV, FP8, check, gen, quantised, same_codes, weights

pytestmark = pytest.mark.gpu

# tile, parts, clusters at once: tiles of few tokens, CTA pairs (with 1 and 3 clusters each of them walks several tiles)
FEW = [(16, 1, 0), (16, 3, 0), (32, 2, 0), (32, 8, 0), (64, 1, 0), (64, 4, 0), (128, 1, 0), (128, 5, 0), (128, 8, 0)]
PAIRS = [(256, 1, 0), (256, 1, 1), (256, 1, 3), (256, 2, 0), (256, 4, 0)]


@pytest.fixture
def choose():
    yield tp.tp_set_fp8_gemm
    tp.tp_set_fp8_gemm()


def dev(pairs):
    return [a.to(DEV) for a, _ in pairs], [s.to(DEV) for _, s in pairs]


def held(codes, scales, v, e):
    assert ((P.rows64(codes, scales) - v).abs() <= P.held(v, e, scales)).all()


def twice(f):
    """f's outputs, which a second call repeats bit for bit."""
    a, b = f(), f()
    flat = lambda v: [v] if isinstance(v, torch.Tensor) else [u for w in v for u in flat(w)]  # noqa: E731
    for u, v in zip(flat(a), flat(b)):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)) if u.dtype is FP8 else torch.equal(u, v)
    assert tp.tp_device_status() == 0
    return a


# 17 K blocks, the last of 16 columns; n: less than a tile, and tiles of which the last is ragged; out odd, ragged in every tile
@pytest.mark.parametrize("variant", FEW + PAIRS)
@pytest.mark.parametrize("n,out", [(5, 301), (300, 301), (600, 648)])
def test_col(choose, variant, n, out):
    t, k = 2, 2064
    x, xs = quantised(n, k, n)
    ws = [weights(out, k, 50 + r) for r in range(t)]
    bias = [torch.randn(out, generator=gen(60 + r)).to(torch.bfloat16) for r in range(t)]
    choose(*variant)
    w, s = dev(ws)
    y32, y16 = (twice(lambda: tp.tp_fp8_linear_col(x.to(DEV), xs.to(DEV), w, s, bias=[b.to(DEV) for b in bias], y_dtype=d))
                for d in (torch.float32, torch.bfloat16))
    x64 = P.rows64(x, xs)
    for r in range(t):
        ref, bound = P.product([x64], [P.weight64(*ws[r])], bias[r])
        check(y32[r], ref, bound)
        check(y16[r], ref, bound)


# os of 203 (fp32 and bf16 alone), of 208 (rows of 16-byte pieces) and of 288 (rows of whole sectors, a last tile of 32 columns)
@pytest.mark.parametrize("variant", FEW + PAIRS)
@pytest.mark.parametrize("n,os,act", [(7, 208, "silu"), (300, 208, "gelu_tanh"), (300, 203, "silu"), (600, 288, "silu")])
def test_gated(choose, variant, n, os, act):
    t, k = 2, 2064
    x, xs = quantised(n, k, n)
    ws = [weights(2 * os, k, 90 + r, True) for r in range(t)]
    choose(*variant)
    a = (x.to(DEV), xs.to(DEV), *dev(ws))
    y32 = twice(lambda: tp.tp_fp8_linear_col(*a, act=act, y_dtype=torch.float32))
    y16 = twice(lambda: tp.tp_fp8_linear_col(*a, act=act))
    codes, scales = twice(lambda: tp.tp_fp8_linear_col(*a, act=act, y_dtype=FP8)) if os % 16 == 0 else (None, None)
    x64 = P.rows64(x, xs)
    for r in range(t):
        v, e = P.gated(x64, *P.halves64(*ws[r]), act)
        check(y32[r], v, e)
        check(y16[r], v, e)
        if codes is not None:
            held(codes[r], scales[r], v, e)
            rc, rs = P.quantise_rows(y32[r].cpu())           # the same fp32 values: the same codes
            assert torch.equal(scales[r].cpu(), rs) and same_codes(codes[r], rc)


# three shards of four K blocks: parts that begin and end inside a shard
@pytest.mark.parametrize("variant", [(16, 5, 0), (64, 8, 0), (128, 3, 0)] + PAIRS)
@pytest.mark.parametrize("n", [6, 290])
def test_row(choose, variant, n):
    t, k, out = 3, 400, 520
    xs = [quantised(n, k, n + r) for r in range(t)]
    ws = [weights(out, k, 70 + r) for r in range(t)]
    bias = torch.randn(out, generator=gen(80)).to(torch.bfloat16)
    choose(*variant)
    a = (*dev(xs), *dev(ws))
    x64, w64 = [P.rows64(*x) for x in xs], [P.weight64(*w) for w in ws]
    ref, bound = P.product(x64, w64, bias)
    check(twice(lambda: tp.tp_fp8_linear_row(*a, bias=bias.to(DEV), mode="fused", y_dtype=torch.float32)), ref, bound)
    if variant[1] > 4:                                       # a shard alone has fewer blocks than parts
        with pytest.raises(tp.TPError, match="UNSUPPORTED"):
            tp.tp_fp8_linear_row(*a, mode="direct")
        return
    y = twice(lambda: tp.tp_fp8_linear_row(*a, bias=bias.to(DEV), mode="ring", partial_dtype=torch.float32, y_dtype=torch.float32))
    check(y, ref, bound * 1.1)                               # fp32 partials: one more rounding for each of the t sums


# a raster band of CTA pairs holds 48 MB of rows: 6 tiles of 28672 columns, so that 7 are two bands
@pytest.mark.parametrize("clusters", [0, 5])
def test_raster_bands(choose, clusters):
    t, n, k, out = 2, 1700, 28672, 264
    xs = [quantised(n, k, n + r) for r in range(t)]
    ws = [weights(out, k, 70 + r) for r in range(t)]
    choose(256, 1, clusters)
    x64, w64 = [P.rows64(*x) for x in xs], [P.weight64(*w) for w in ws]
    y = twice(lambda: tp.tp_fp8_linear_col(xs[0][0].to(DEV), xs[0][1].to(DEV), *dev(ws), y_dtype=torch.float32))
    parts = twice(lambda: tp.tp_fp8_linear_row(*dev(xs), *dev(ws), reduce_results=False, partial_dtype=torch.float32))
    for r in range(t):
        check(y[r], *P.product([x64[0]], [w64[r]]))
        check(parts[r], *P.product([x64[r]], [w64[r]]))


@pytest.mark.parametrize("variant", [(64, 2, 0), (128, 1, 0), (256, 1, 2), (256, 2, 0), (256, 4, 0)])
@pytest.mark.parametrize("mode", ["fused", "direct"])
def test_mlp(choose, variant, mode):
    t, n, h, f = 2, 333, 1040, 2 * 528
    fs = f // t
    x, xs = (v.to(DEV) for v in quantised(n, h, 1))
    a = dev([weights(2 * fs, h, 100 + r, True) for r in range(t)])
    b = [weights(h, fs, 120 + r) for r in range(t)]
    choose(*variant)
    kw = dict(mode=mode, y_dtype=torch.float32, partial_dtype=torch.float32)
    y = twice(lambda: tp.tp_fp8_mlp_forward(x, xs, *a, *dev(b), **kw))
    hc, hs = tp.tp_fp8_linear_col(x, xs, *a, act="silu", y_dtype=FP8)
    assert torch.equal(y, tp.tp_fp8_linear_row(hc, hs, *dev(b), **kw))
    ref, bound = P.product([P.rows64(c, s) for c, s in zip(hc, hs)], [P.weight64(*w) for w in b])
    check(y, ref, bound * 1.1)


@pytest.mark.parametrize("variant", [(64, 3, 0), (128, 1, 0), (256, 1, 1), (256, 2, 0)])
def test_a_row_depends_on_itself_alone(choose, variant):
    """Rows with NaN codes and scales leave the others' codes and values as they were."""
    n, k, os = 300, 2064, 288
    x, xs = quantised(n, k, 8)
    w, s = (v.to(DEV) for v in weights(2 * os, k, 9, True))
    choose(*variant)
    xd, sd = x.to(DEV), xs.to(DEV)
    run = lambda: (tp.tp_fp8_linear_col(xd, sd, [w], [s], act="silu", y_dtype=FP8),  # noqa: E731
                   tp.tp_fp8_linear_col(xd, sd, [w], [s], act="silu", y_dtype=torch.float32)[0])
    (c0, s0), y0 = run()
    sd[1, 1] = float("nan")
    xd.view(torch.uint8)[257, 17] = 0x7F
    (c1, s1), y1 = run()
    keep = [i for i in range(n) if i not in (1, 257)]
    assert bool(y1[[1, 257]].isnan().all()) and bool(s1[0][:, [1, 257]].isnan().all())
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(s0[0][:, keep], s1[0][:, keep])
    assert torch.equal(c0[0].view(torch.uint8)[keep], c1[0].view(torch.uint8)[keep])


def test_untouched_bytes(choose):
    """Rows, columns and scales around the outputs stay as they were, in every kernel."""
    n, k, os = 300, 1040, 208
    x, xs = quantised(n, k, 2)
    w, s = (v.to(DEV) for v in weights(2 * os, k, 3, True))
    pw, ps = (v.to(DEV) for v in weights(301, k, 4))
    a = (x.to(DEV), xs.to(DEV))
    for variant in FEW + PAIRS:
        choose(*variant)
        buf = torch.full((n + 2, os + 32), 9, dtype=torch.uint8, device=DEV)
        sc = torch.full((3, n + 4), -1.0, device=DEV)
        tp.tp_fp8_linear_col(*a, [w], [s], act="silu", y=[buf.view(FP8)[1:n + 1, 16:16 + os]], y_scales=[sc[:2, 2:n + 2]])
        buf[1:n + 1, 16:16 + os] = 9
        sc[:2, 2:n + 2] = -1.0
        assert (buf == 9).all() and (sc == -1.0).all(), variant
        for dt in (torch.float32, torch.bfloat16):
            y = torch.full((n + 2, 301 + 19), 5.0, dtype=dt, device=DEV)
            tp.tp_fp8_linear_col(*a, [pw], [ps], y=[y[1:n + 1, 8:309]])
            y[1:n + 1, 8:309] = 5.0
            assert (y == 5.0).all(), variant


@pytest.mark.parametrize("variant", [(16, 2, 0), (64, 1, 0), (256, 1, 0), (256, 2, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gathered_columns_of_an_odd_width(choose, variant, dtype):
    """The second and third shards' columns begin at no 16-byte boundary."""
    t, n, k, out = 3, 270, 528, 301
    x, xs = quantised(n, k, 5)
    ws = [weights(out, k, 30 + r) for r in range(t)]
    choose(*variant)
    y = torch.full((n, t * out + 13), 5.0, dtype=dtype, device=DEV)
    tp.tp_fp8_linear_col(x.to(DEV), xs.to(DEV), *dev(ws), gather_output=True, y=y[:, :t * out])
    for r in range(t):
        check(y[:, r * out:(r + 1) * out], *P.product([P.rows64(x, xs)], [P.weight64(*ws[r])]))
    assert (y[:, t * out:] == 5.0).all()

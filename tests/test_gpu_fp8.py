"""The 8-bit operators against their plain forms (fp8_plain.py has the formulas and the bounds)."""

import pytest
import torch

import fp8_plain as P
from megatron_tensor_layers_gb300 import _lib as tp

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP8 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rows(n, k, seed, dtype=torch.bfloat16):
    g = gen(seed)
    return (torch.randn((n, k), generator=g) * torch.exp(0.6 * torch.randn(k, generator=g))).to(dtype)


def same_codes(a, b):
    """Bit for bit, NaN codes of either sign alike."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    an, bn = a.float().isnan(), b.float().isnan()
    return torch.equal(an, bn) and torch.equal(a.view(torch.uint8)[~an], b.view(torch.uint8)[~an])


def same_scales(a, b):
    return torch.equal(torch.nan_to_num(a.cpu(), nan=-1.0), torch.nan_to_num(b.cpu(), nan=-1.0))


def strided(x, pad=16, rows=0):
    """x as a view of a wider (and taller) buffer."""
    buf = torch.zeros((x.shape[0] + rows, x.shape[1] + pad), dtype=torch.uint8 if x.dtype is FP8 else x.dtype, device=DEV)
    buf = buf.view(x.dtype)
    buf[:x.shape[0], :x.shape[1]] = x.to(DEV)
    return buf[:x.shape[0], :x.shape[1]]


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("t,n,k,dtype", [(1, 1, 16, torch.bfloat16), (8, 64, 1024, torch.bfloat16),
                                         (3, 37, 400, torch.float32), (2, 1000, 8192, torch.bfloat16),
                                         (1, 130, 2064, torch.float32)])
def test_quantize_bits(t, n, k, dtype):
    xs = [rows(n, k, 10 + r, dtype) for r in range(t)]
    codes, scales = tp.tp_fp8_quantize([x.to(DEV) for x in xs])
    for x, c, s in zip(xs, codes, scales):
        rc, rs = P.quantise_rows(x)
        assert same_scales(s, rs) and same_codes(c, rc)


def test_quantize_extremes():
    x = rows(12, 300, 3)
    x[0] = 0
    x[1] = -0.0
    x[2, 128:256] = 2.0 ** -120              # a group of values below the floor of the scale
    x[3] *= 2.0 ** 100
    x[4, 5] = float("nan")
    x[5, 130] = float("inf")
    x[6, 299] = float("-inf")
    x[7] = torch.finfo(torch.bfloat16).max
    x[8, ::2] = 448.0
    x[9] = 2.0 ** -133                       # the smallest bf16
    x = torch.nn.functional.pad(x, (0, 4))   # 304 columns
    codes, scales = tp.tp_fp8_quantize([x.to(DEV)])
    rc, rs = P.quantise_rows(x)
    assert same_scales(scales[0], rs) and same_codes(codes[0], rc)
    v = codes[0].cpu().double() * scales[0].cpu().double().t().repeat_interleave(128, 1)[:, :304]
    assert v[4, :128].isnan().all() and v[5, 128:256].isnan().all() and v[6, 256:].isnan().all()
    assert v[4, 128:].isfinite().all() and v[5, :128].isfinite().all() and v[6, :256].isfinite().all()


def test_quantize_views_and_untouched_bytes():
    n, k = 33, 272
    x = rows(n, k, 5)
    codes = torch.full((n + 2, k + 32), 7, dtype=torch.uint8, device=DEV)
    scales = torch.full((P.groups(k) + 1, n + 5), -3.0, device=DEV)
    tp.tp_fp8_quantize([strided(x, 24)], codes=[codes.view(FP8)[1:n + 1, 16:k + 16]], scales=[scales[:-1, 2:n + 2]])
    rc, rs = P.quantise_rows(x)
    assert same_codes(codes.view(FP8)[1:n + 1, 16:k + 16], rc) and torch.equal(scales[:-1, 2:n + 2].cpu(), rs)
    codes[1:n + 1, 16:k + 16] = 7
    scales[:-1, 2:n + 2] = -3.0
    assert (codes == 7).all() and (scales == -3.0).all()


@pytest.mark.parametrize("out,k,gated,dtype", [(1, 16, False, torch.bfloat16), (128, 128, False, torch.bfloat16),
                                               (300, 400, False, torch.float32), (2, 64, True, torch.bfloat16),
                                               (600, 272, True, torch.bfloat16), (512, 1024, True, torch.float32)])
def test_quantize_weight_bits(out, k, gated, dtype):
    ws = [(torch.randn((out, k), generator=gen(7 + r)) * 0.02).to(dtype) for r in range(2)]
    if out > 2:
        ws[1][out // 2 + 1, 3] = float("nan")
    codes, scales = tp.tp_fp8_quantize_weight([strided(w, 8) for w in ws], gated=gated)
    for w, c, s in zip(ws, codes, scales):
        rc, rs = P.quantise_weight(w, gated)
        assert same_scales(s, rs) and same_codes(c, rc)


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("t,n,h,dtype,residual,mode", [
    (1, 1, 16, torch.bfloat16, False, "direct"), (4, 1, 8192, torch.bfloat16, True, "direct"),
    (2, 37, 1024, torch.float32, True, "ring"), (8, 300, 4112, torch.bfloat16, True, "ring"),
    (3, 5, 32768, torch.float32, False, "direct"), (5, 9, 2064, torch.bfloat16, True, "direct"),
    (2, 3, 16400, torch.bfloat16, True, "direct"), (1, 64, 640, torch.float32, True, "direct"),
    (8, 2, 32768, torch.bfloat16, True, "ring")])
def test_norm(t, n, h, dtype, residual, mode):
    ps = [(rows(n, h, 20 + r, torch.float32) * 0.4).to(dtype) for r in range(t)]
    res = rows(n, h, 40) if residual else None
    w = (1.0 + 0.2 * torch.randn(h, generator=gen(41))).to(torch.bfloat16)
    out = torch.zeros((n, h), dtype=torch.bfloat16, device=DEV)
    got, codes, scales = tp.tp_fp8_rmsnorm([p.to(DEV) for p in ps], w.to(DEV), residual=None if res is None else res.to(DEV),
                                           mode=mode, residual_out=out)
    assert got is out
    per = -(-n // t)
    fold = torch.zeros((n, h))
    for i in range(n):                                     # the fold order is the owner rank's
        start = (i // per + 1) % t if mode == "ring" else 0
        acc = ps[start][i].float()
        for j in range(1, t):
            acc = acc + ps[(start + j) % t][i].float()
        fold[i] = res[i].float() + acc if residual else acc
    assert torch.equal(out.cpu(), fold.to(torch.bfloat16))
    r = fold.double()
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * w.double()
    # the sum of squares: h roundings of a positive sum at most, halved by the root; rsqrt and two products
    e = ((h / 2 ** 5 + 64) / 2 + 8) * 2.0 ** -24 * y.abs()
    v = P.rows64(codes, scales)
    assert ((v - y).abs() <= P.held(y, e, scales)).all()
    rs = torch.nn.functional.pad(y.abs(), (0, -h % 128)).reshape(n, -1, 128).amax(-1).clamp(min=2.0 ** -100) / 448
    assert ((scales.cpu().double().t() - rs).abs() <= rs * (e / y.abs().clamp(min=1e-300)).max() + rs * 2.0 ** -23).all()


def test_norm_in_place_zero_rows_and_nan():
    n, h = 6, 1040
    p, res = rows(n, h, 1), rows(n, h, 2)
    p[0] = 0
    res[0] = 0
    p[3, 700] = float("nan")
    w = torch.ones(h, dtype=torch.bfloat16)
    buf = res.to(DEV)
    _, codes, scales = tp.tp_fp8_rmsnorm([p.to(DEV)], w.to(DEV), residual=buf, residual_out=buf)
    assert torch.equal(torch.nan_to_num(buf.cpu().float()), torch.nan_to_num((res.float() + p.float()).to(torch.bfloat16).float()))
    v = P.rows64(codes, scales)
    assert (v[0] == 0).all() and v[3].isnan().all()
    assert v[[1, 2, 4, 5]].isfinite().all()


# ------------------------------------------------------------------ products

def quantised(n, k, seed):
    return P.quantise_rows(rows(n, k, seed))


def weights(out, k, seed, gated=False):
    return P.quantise_weight(torch.randn((out, k), generator=gen(seed)) * 0.05, gated)


def check(y, ref, bound):
    half = 2.0 ** -8 * ref.abs() if y.dtype is torch.bfloat16 else 2.0 ** -24 * ref.abs()
    err = (y.cpu().double() - ref).abs()
    assert (err <= bound + half * 1.01).all(), (err - bound - half).max().item()


NS = [1, 7, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 600]


@pytest.mark.parametrize("n", NS)
@pytest.mark.parametrize("t,k,out,dtype", [(1, 16, 8, torch.float32), (2, 400, 300, torch.float32), (3, 1024, 640, torch.bfloat16)])
def test_col(n, t, k, out, dtype):
    x, xs = quantised(n, k, n)
    ws = [weights(out, k, 50 + r) for r in range(t)]
    bias = [torch.randn(out, generator=gen(60 + r)).to(torch.bfloat16) for r in range(t)]
    y = tp.tp_fp8_linear_col(x.to(DEV), xs.to(DEV), [w.to(DEV) for w, _ in ws], [s.to(DEV) for _, s in ws],
                             bias=[b.to(DEV) for b in bias], y_dtype=dtype)
    x64 = P.rows64(x, xs)
    for r in range(t):
        check(y[r], *P.product([x64], [P.weight64(*ws[r])], bias[r]))


@pytest.mark.parametrize("n", [1, 20, 100, 130, 256, 300])
@pytest.mark.parametrize("t,k,out", [(1, 4096, 128), (4, 2064, 520), (8, 1040, 1024)])
def test_long_sums_in_parts(n, t, k, out):
    """Few output tiles and long sums: the K blocks are cut over a cluster."""
    xs = [quantised(n, k, n + r) for r in range(t)]
    ws = [weights(out, k, 200 + r) for r in range(t)]
    y = tp.tp_fp8_linear_row([x.to(DEV) for x, _ in xs], [s.to(DEV) for _, s in xs], [w.to(DEV) for w, _ in ws],
                             [s.to(DEV) for _, s in ws], mode="fused", y_dtype=torch.float32)
    check(y, *P.product([P.rows64(*x) for x in xs], [P.weight64(*w) for w in ws]))
    x, s = xs[0]
    gw, gs = weights(2 * 272, k, 300, True)
    c, cs = tp.tp_fp8_linear_col(x.to(DEV), s.to(DEV), [gw.to(DEV)], [gs.to(DEV)], act="silu", y_dtype=FP8)
    v, e = P.gated(P.rows64(x, s), *P.halves64(gw, gs), "silu")
    assert ((P.rows64(c[0], cs[0]) - v).abs() <= P.held(v, e, cs[0])).all()


@pytest.mark.parametrize("n", NS)
@pytest.mark.parametrize("t,k,out", [(1, 48, 200), (4, 272, 1000), (8, 128, 64)])
def test_row_modes(n, t, k, out):
    xs = [quantised(n, k, n + r) for r in range(t)]
    ws = [weights(out, k, 70 + r) for r in range(t)]
    bias = torch.randn(out, generator=gen(80)).to(torch.bfloat16)
    a = ([x.to(DEV) for x, _ in xs], [s.to(DEV) for _, s in xs], [w.to(DEV) for w, _ in ws], [s.to(DEV) for _, s in ws])
    x64, w64 = [P.rows64(*x) for x in xs], [P.weight64(*w) for w in ws]
    ref, bound = P.product(x64, w64, bias)
    y = tp.tp_fp8_linear_row(*a, bias=bias.to(DEV), mode="fused", y_dtype=torch.float32)
    check(y, ref, bound)
    for mode in ("direct", "ring"):                      # fp32 partials: one more rounding for each of the t sums
        y = tp.tp_fp8_linear_row(*a, bias=bias.to(DEV), mode=mode, partial_dtype=torch.float32, y_dtype=torch.float32)
        check(y, ref, bound * 1.1)
    parts = tp.tp_fp8_linear_row(*a, bias=bias.to(DEV), reduce_results=False, partial_dtype=torch.bfloat16)
    for r in range(t):
        check(parts[r], *P.product([x64[r]], [w64[r]], bias if r == 0 else None))


@pytest.mark.parametrize("n", NS)
@pytest.mark.parametrize("t,k,os,act", [(1, 128, 16, "silu"), (2, 400, 208, "gelu_tanh"), (2, 1024, 384, "silu")])
def test_gated(n, t, k, os, act):
    x, xs = quantised(n, k, n)
    ws = [weights(2 * os, k, 90 + r, True) for r in range(t)]
    a = (x.to(DEV), xs.to(DEV), [w.to(DEV) for w, _ in ws], [s.to(DEV) for _, s in ws])
    codes, scales = tp.tp_fp8_linear_col(*a, act=act, y_dtype=FP8)
    y32 = tp.tp_fp8_linear_col(*a, act=act, y_dtype=torch.float32)
    y16 = tp.tp_fp8_linear_col(*a, act=act)
    x64 = P.rows64(x, xs)
    for r in range(t):
        v, e = P.gated(x64, *P.halves64(*ws[r]), act)
        check(y32[r], v, e)
        check(y16[r], v, e)
        assert ((P.rows64(codes[r], scales[r]) - v).abs() <= P.held(v, e, scales[r])).all()
        rc, rs = P.quantise_rows(y32[r].cpu())           # the same fp32 values: the same codes
        assert torch.equal(scales[r].cpu(), rs) and same_codes(codes[r], rc)


@pytest.mark.parametrize("t,n,h,f", [(2, 8, 1024, 4096), (1, 1, 256, 128), (4, 40, 528, 64 * 13), (8, 130, 512, 2048),
                                     (2, 300, 640, 1056), (1, 513, 2048, 1024)])
@pytest.mark.parametrize("mode", ["fused", "direct"])
def test_mlp_equals_its_two_calls(t, n, h, f, mode):
    x, xs = (v.to(DEV) for v in quantised(n, h, 1))
    fs = f // t
    a = [weights(2 * fs, h, 100 + r, True) for r in range(t)]
    b = [weights(h, fs, 120 + r) for r in range(t)]
    aw, as_ = [w.to(DEV) for w, _ in a], [s.to(DEV) for _, s in a]
    bw, bs = [w.to(DEV) for w, _ in b], [s.to(DEV) for _, s in b]
    bias = torch.randn(h, generator=gen(5)).to(torch.bfloat16).to(DEV)
    y = tp.tp_fp8_mlp_forward(x, xs, aw, as_, bw, bs, mode=mode, bias_down=bias, y_dtype=torch.float32,
                              partial_dtype=torch.float32)
    hc, hs = tp.tp_fp8_linear_col(x, xs, aw, as_, act="silu", y_dtype=FP8)
    z = tp.tp_fp8_linear_row(hc, hs, bw, bs, mode=mode, bias=bias, y_dtype=torch.float32, partial_dtype=torch.float32)
    assert torch.equal(y, z)
    ref, bound = P.product([P.rows64(c, s) for c, s in zip(hc, hs)], [P.weight64(*w) for w in b], bias.cpu())
    check(y, ref, bound * 1.1)
    assert tp.tp_device_status() == 0


@pytest.mark.parametrize("n", [3, 70, 300])
def test_views_gather_and_untouched_bytes(n):
    t, k, out = 2, 336, 136
    x, xs = quantised(n, k, 2)
    ws = [weights(out, k, 130 + r) for r in range(t)]
    x_s = torch.full((P.groups(k), n + 3), float("nan"), device=DEV)
    x_s[:, 1:n + 1] = xs.to(DEV)
    y = torch.full((n + 2, t * out + 24), 5.0, device=DEV)
    view = y[1:n + 1, 8:8 + t * out]
    got = tp.tp_fp8_linear_col(strided(x, 48), x_s[:, 1:n + 1], [strided(w, 16) for w, _ in ws], [s.to(DEV) for _, s in ws],
                               gather_output=True, y=view)
    assert got is view
    for r in range(t):
        check(view[:, r * out:(r + 1) * out], *P.product([P.rows64(x, xs)], [P.weight64(*ws[r])]))
    view.fill_(5.0)
    assert (y == 5.0).all()


@pytest.mark.parametrize("n", [5, 100, 300])
def test_gated_codes_into_views(n):
    k, os = 256, 144
    x, xs = quantised(n, k, 2)
    w, s = weights(2 * os, k, 3, True)
    buf = torch.full((n + 2, os + 32), 9, dtype=torch.uint8, device=DEV)
    sc = torch.full((3, n + 4), -1.0, device=DEV)
    a = (x.to(DEV), xs.to(DEV), [w.to(DEV)], [s.to(DEV)])
    tp.tp_fp8_linear_col(*a, act="silu", y=[buf.view(FP8)[1:n + 1, 16:16 + os]], y_scales=[sc[:2, 2:n + 2]])
    c, cs = tp.tp_fp8_linear_col(*a, act="silu", y_dtype=FP8)
    assert same_codes(buf.view(FP8)[1:n + 1, 16:16 + os], c[0]) and torch.equal(sc[:2, 2:n + 2], cs[0])
    buf[1:n + 1, 16:16 + os] = 9
    sc[:2, 2:n + 2] = -1.0
    assert (buf == 9).all() and (sc == -1.0).all()


@pytest.mark.parametrize("n", [4, 90, 260])
def test_a_row_depends_on_itself_alone(n):
    """A NaN scale of row 1, a NaN code of row 2 and an infinite scale of row 3 leave the others' bits as they were."""
    k, out = 512, 256
    x, xs = quantised(n, k, 8)
    w, s = (v.to(DEV) for v in weights(out, k, 9))
    xd, sd = x.to(DEV), xs.to(DEV)
    y = tp.tp_fp8_linear_col(xd, sd, [w], [s], y_dtype=torch.float32)[0]
    sd[1, 1] = float("nan")
    xd.view(torch.uint8)[2, 17] = 0x7F
    sd[2, 3] = float("inf")
    z = tp.tp_fp8_linear_col(xd, sd, [w], [s], y_dtype=torch.float32)[0]
    nan, finite = z.isnan(), z.isfinite()
    assert bool(nan[1].all()) and bool(nan[2].all())
    assert not bool(finite[3].any())                     # its infinite scale times sums that are not 0
    keep = [i for i in range(n) if i not in (1, 2, 3)]
    assert torch.equal(y[keep], z[keep])
    assert tp.tp_device_status() == 0


def test_zero_tokens():
    w, s = (v.to(DEV) for v in weights(64, 128, 1))
    x = torch.empty((0, 128), dtype=torch.uint8, device=DEV).view(FP8)
    xs = torch.empty((1, 0), device=DEV)
    assert tp.tp_fp8_linear_col(x, xs, [w], [s])[0].shape == (0, 64)
    assert tp.tp_fp8_linear_row([x], [xs], [w], [s], mode="fused").shape == (0, 64)
    c, sc = tp.tp_fp8_quantize([torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)])
    assert c[0].shape == (0, 256) and sc[0].shape == (2, 0)
    r, c, sc = tp.tp_fp8_rmsnorm([torch.empty((0, 256), device=DEV)], torch.ones(256, dtype=torch.bfloat16, device=DEV))
    assert r.shape == c.shape == (0, 256) and sc.shape == (2, 0)


@pytest.mark.parametrize("n", [2, 48, 150, 320])
def test_streams_graphs_and_prepared_calls(n):
    """A layer's operators in a row: eager, on another stream, prepared, and replayed from a graph with new inputs."""
    t, h, f = 2, 512, 1024
    fs = f // t
    a = [weights(2 * fs, h, 100 + r, True) for r in range(t)]
    b = [weights(h, fs, 120 + r) for r in range(t)]
    aw, as_ = [w.to(DEV) for w, _ in a], [s.to(DEV) for _, s in a]
    bw, bs = [w.to(DEV) for w, _ in b], [s.to(DEV) for _, s in b]
    wn = torch.ones(h, dtype=torch.bfloat16, device=DEV)
    parts = [rows(n, h, 30 + r).to(DEV) for r in range(t)]
    res = rows(n, h, 33).to(DEV)

    def layer():
        r, c, s = tp.tp_fp8_rmsnorm(parts, wn, residual=res)
        y = tp.tp_fp8_mlp_forward(c, s, aw, as_, bw, bs, mode="fused")
        r2, c2, s2 = tp.tp_fp8_rmsnorm([y], wn, residual=r)
        (c3,), (s3,) = tp.tp_fp8_quantize([r2])
        return r2, tp.tp_fp8_linear_row([c3], [s3], [aw[0]], [as_[0]], mode="fused", y_dtype=torch.float32)

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    new = [rows(n, h, 60 + r).to(DEV) for r in range(t)]
    for p, q in zip(parts, new):
        p.copy_(q)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    again = layer()
    assert all(torch.equal(u, v) for u, v in zip(again, out)) and not torch.equal(again[0], want[0])
    c, s = tp.tp_fp8_quantize([res])
    call = tp.prepare(tp.tp_fp8_mlp_forward, c[0], s[0], aw, as_, bw, bs, mode="direct")
    assert torch.equal(call(), tp.tp_fp8_mlp_forward(c[0], s[0], aw, as_, bw, bs, mode="direct"))
    assert tp.tp_device_status() == 0


@pytest.mark.parametrize("n", [1, 24, 200])
def test_weights_written_just_before(n):
    """A weight that the call before brings to 8 bits is what the MLP multiplies by, with nothing waited for between."""
    t, h, f = 2, 2048, 4096
    fs = f // t
    x, xs = (v.to(DEV) for v in quantised(n, h, 1))
    wa = [[(torch.randn((2 * fs, h), generator=gen(i * 10 + r)) * 0.05).to(torch.bfloat16).to(DEV) for r in range(t)] for i in range(2)]
    wb = [[(torch.randn((h, fs), generator=gen(i * 10 + 5 + r)) * 0.05).to(torch.bfloat16).to(DEV) for r in range(t)] for i in range(2)]
    want = []
    for i in range(2):
        a, b = tp.tp_fp8_quantize_weight(wa[i], gated=True), tp.tp_fp8_quantize_weight(wb[i])
        torch.cuda.synchronize()
        want.append(tp.tp_fp8_mlp_forward(x, xs, *a, *b, mode="fused"))
        torch.cuda.synchronize()
    ca, sa = tp.tp_fp8_quantize_weight(wa[0], gated=True)
    cb, sb = tp.tp_fp8_quantize_weight(wb[0])
    ys = []
    for i in range(40):                                  # the same buffers, other weights each time
        tp.tp_fp8_quantize_weight(wa[i % 2], gated=True, codes=ca, scales=sa)
        tp.tp_fp8_quantize_weight(wb[i % 2], codes=cb, scales=sb)
        ys.append(tp.tp_fp8_mlp_forward(x, xs, ca, sa, cb, sb, mode="fused"))
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(ys))


def test_two_streams_at_once():
    """Products of different kernels on two streams, each with its own buffers."""
    k, out = 4096, 1024
    w, s = (v.to(DEV) for v in weights(out, k, 3))
    g, gs = (v.to(DEV) for v in weights(2 * 512, k, 4, True))
    sizes = [1, 20, 60, 100, 300]
    xs = [tuple(v.to(DEV) for v in quantised(n, k, n)) for n in sizes]
    want = [(tp.tp_fp8_linear_row([x], [sc], [w], [s], mode="fused", y_dtype=torch.float32),
             tp.tp_fp8_linear_col(x, sc, [g], [gs], act="silu")[0]) for x, sc in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = {0: [], 1: []}
    for _ in range(10):
        for i in range(len(sizes)):
            for j, st in enumerate(streams):
                x, sc = xs[(i + 2 * j) % len(sizes)]
                with torch.cuda.stream(st):
                    got[j].append(((i + 2 * j) % len(sizes), tp.tp_fp8_linear_row([x], [sc], [w], [s], mode="fused", y_dtype=torch.float32),
                                   tp.tp_fp8_linear_col(x, sc, [g], [gs], act="silu")[0]))
    torch.cuda.synchronize()
    for i, y, z in got[0] + got[1]:
        assert torch.equal(y, want[i][0]) and torch.equal(z, want[i][1])
    assert tp.tp_device_status() == 0

"""Attention over the paged 4-bit cache for chunks that fill the device (the
many-rows kernel), against a float64 oracle.

Bound of an output element (`check`), with p the oracle's probabilities:
* keys are rounded once to fp16, by 2^-11 of themselves or 2^-25 of a scale of at
  most twice the largest step or base; a score is off by at most
  D = |scale| (2^-11 max_j sum|q k_j| + 2^-24 max(s, |b|) sum|q|) and by its fp32
  sum, (head_dim + 16) 2^-23 |scale| sum|q| max_j(15 s_j + |b_j|) (a sum's terms may
  be taken apart into steps and bases); a probability is then off by a factor
  within e^(+-2D), the output by (e^(2D) - 1) sum_j p_j |v_j - out|;
* values and probabilities are rounded to fp16 once each: 2 * 2^-11 max_j(15 s_j +
  |b_j|);
* fp32 sums, and what both roundings lose below the smallest fp16: (m + 16) 2^-23
  max_j(15 s_j + |b_j|) over m tokens;
* the store: half a bf16 step (2^-8 relative covers a value that crosses a binade).
"""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from test_gpu_kv4 import Cache, DEV, cu_of, f64

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


def rows_of(c, rows, heads, seed):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(rng.standard_normal((sum(rows), heads * c.hd)).astype(np.float32)).to(torch.bfloat16).to(DEV)
            for _ in range(c.t)]


def check(c, q, got, rows, heads, window=0, sinks=0, scale=None, hidden=None):
    """`hidden(s)`: tokens of sequence s that are not there."""
    sc = c.hd ** -0.5 if scale is None else scale
    group, n = heads // c.kv, sum(rows)
    for r in range(c.t):
        qr, y = f64(q[r]).reshape(n, heads, c.hd), f64(got[r]).reshape(n, heads, c.hd)
        at = 0
        for s, m in enumerate(rows):
            pos = (c.lens[s] - m + np.arange(m))[:, None]
            for h in range(heads):
                kk, ks, kb = c.tokens(c.kq, r, s, h // group)
                vv, vs, vb = c.tokens(c.vq, r, s, h // group)
                have, x = y[at:at + m, h], qr[at:at + m, h]
                if not m or not len(kk):
                    assert not have.any()
                    continue
                j = np.arange(len(kk))[None, :]
                see = j <= pos
                if window:
                    see &= (j > pos - window) | (j < sinks)
                if hidden is not None:
                    see &= ~hidden(s)[None, :]
                bad = np.isnan(kk).any(1) | np.isnan(vv).any(1)
                dead = (see & bad).any(1)
                see &= ~bad
                kz, vz = np.where(bad[:, None], 0, kk), np.where(bad[:, None], 0, vv)
                score = np.where(see, sc * (x @ kz.T), -np.inf)
                top = score.max(1, keepdims=True)
                p = np.exp(score - np.where(np.isfinite(top), top, 0))
                total = p.sum(1, keepdims=True)
                p = p / np.where(total > 0, total, 1)
                want = p @ vz
                kmost, vmost = np.nan_to_num(15 * ks + np.abs(kb)).max(), np.nan_to_num(15 * vs + np.abs(vb)).max()
                absq = np.abs(x).sum(1, keepdims=True)
                D = abs(sc) * (2.0 ** -11 * (np.abs(x) @ np.abs(kz).T).max(1, keepdims=True) + 2.0 ** -24 * kmost * absq +
                               (c.hd + 16) * 2.0 ** -23 * absq * kmost)
                spread = np.stack([p_ @ np.abs(vz - w_) for p_, w_ in zip(p, want)])
                tol = (2 * 2.0 ** -11 * vmost + (len(kk) + 16) * 2.0 ** -23 * vmost + np.expm1(2 * D) * spread +
                       2.0 ** -8 * np.abs(want))
                assert np.array_equal(np.isnan(have).all(1), dead) and not np.isnan(have[~dead]).any(), (r, s, h)
                err = np.abs(have - want)[~dead]
                assert (err <= tol[~dead]).all(), (r, s, h, float((err / tol[~dead]).max()))
            at += m


def run(c, rows, heads, seed, **kw):
    q = rows_of(c, rows, heads, seed)
    got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of(rows), **kw)
    assert tp.tp_device_status() == 0
    check(c, q, got, rows, heads, **kw)
    return q, got


# Heads and rows give 72 columns for each of 76 pairs of thread blocks and more.
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5), (1, 0), (200, 130)])
@pytest.mark.parametrize("t,kv,group,hd,ps", [(2, 4, 4, 128, 64), (1, 8, 5, 64, 16), (4, 8, 1, 128, 32), (4, 8, 2, 128, 32),
                                              (1, 3, 16, 64, 128)])
def test_ragged_chunks(t, kv, group, hd, ps, window, sinks):
    rows = [3, 0, 1, 70, 9, 160]
    lens = [3, 20, 77, 200, 9, 333]
    c = Cache(t, kv, hd, ps, lens, 31)
    run(c, rows, kv * group, 32, window=window, sinks=sinks)


@pytest.mark.parametrize("rows", [[73], [75], [76], [77], [64, 11, 1], [40, 37], [85], [86], [43, 43], [42, 43]])
def test_around_the_border_of_the_kernels(rows):
    """64 columns a row over all heads: 76 pairs of thread blocks ask for 72 columns each, so for 86 rows."""
    c = Cache(1, 8, 128, 64, [m + 150 for m in rows], 33)
    run(c, rows, 64, 34)


def test_more_heads_than_pairs():
    """Several waves of pairs, and a device full of tiles with a few columns each."""
    c = Cache(4, 16, 64, 16, [90, 40, 65], 35)
    run(c, [70, 33, 65], 64, 36)


def test_chunk_rows_before_the_first_token():
    c = Cache(1, 8, 128, 64, [90, 0, 40], 37)
    run(c, [100, 70, 41], 64, 38)


@pytest.mark.parametrize("hd", [64, 128])
def test_chunk_scales_and_extreme_rows(hd):
    c = Cache(1, 8, hd, 64, [300, 129], 39)
    c.vq[1][:, :, :, :, 3] = K.bf16(np.float32(1e-30))
    c.vq[1][:, :, :, :, 5] = 0
    c.kq[1][:, :, :, :, 6] = 0
    c.fill()
    rows = [60, 40]
    for mul in (1.0, 1e-20, 0.0, 4.0):
        q = [(x * mul).to(torch.bfloat16) for x in rows_of(c, rows, 64, 40)]
        for scale in (None, 0.0, -0.3):
            got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of(rows), scale=scale)
            check(c, q, got, rows, 64, scale=scale)
    c.vq[1][:] = 0
    c.fill()
    run(c, rows, 64, 41)


def test_chunk_nan_only_where_visible():
    lens = [200, 90]
    c = Cache(1, 8, 128, 64, lens, 42)
    page, off = c.table[0, 100 // 64], 100 % 64
    c.vq[1][0, page, :, off // 16, off % 16], c.vq[2][0, page, :, off // 16, off % 16] = 0, np.nan
    page, off = c.table[0, 150 // 64], 150 % 64
    c.kq[1][0, page, :, off // 16, off % 16], c.kq[2][0, page, :, off // 16, off % 16] = 0, np.nan
    for s, n in enumerate(lens):
        page, off = c.table[s, n // 64], n % 64
        for o in range(off, 64):
            for part in (c.kq, c.vq):
                part[1][0, page, :, o // 16, o % 16] = np.inf
                part[2][0, page, :, o // 16, o % 16] = np.nan
    c.fill()
    run(c, [120, 30], 64, 43)
    run(c, [120, 30], 64, 44, window=10, sinks=2)


def test_chunk_bad_pages_are_skipped_and_reported():
    lens, rows = [250, 100], [100, 64]
    c = Cache(1, 8, 128, 64, lens, 45)
    q = rows_of(c, rows, 64, 46)
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        c.dtable[0, 1] = bad
        got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of(rows))
        assert tp.tp_device_status() == 1
        assert tp.tp_device_status() == 0
        check(c, q, got, rows, 64, hidden=lambda s: (s == 0) & (np.arange(lens[s]) // 64 == 1))


def test_chunk_repeats_in_a_graph_and_on_a_stream():
    c = Cache(2, 4, 128, 32, [400, 700], 47)
    rows = [100, 90]
    q, plain = run(c, rows, 32, 48)
    ws = torch.full((tp.tp_kv4_attention_workspace_size(2, 190, 2, 32, 4, 128),), 255, dtype=torch.uint8, device=DEV)
    cu = cu_of(rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu, workspace=ws)
    for _ in range(2):
        for o in captured:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, e) for a, b, e in zip(plain, captured, again))


@pytest.mark.parametrize("hd,window,sinks", [(64, 0, 0), (128, 0, 0), (128, 40, 3)])
def test_many_sequences_of_few_rows(hd, window, sinks):
    """Enough columns for tiles of 16 of them, none of the sequences long enough for the many-rows kernel."""
    rng = np.random.default_rng(49)
    rows = rng.integers(2, 9, 20).tolist()
    lens = (np.array(rows) + rng.integers(0, 150, 20)).tolist()
    c = Cache(4, 8, hd, 32, lens, 50)
    run(c, rows, 32, 51, window=window, sinks=sinks)

"""Append, load and attention over the paged 4-bit cache against the float64
oracle: codes bit for bit, attention within a bound derived from its roundings.

Bound of an attention output (per element, `attention_bound`):
* the probabilities enter the products rounded to fp16, at most 2^-11 relative:
  2^-11 max_j(15 s_j) over the row's tokens;
* fp32 sums over m tokens and the exponent's approximation: (m + 16) 2^-24
  max_j(15 s_j + |b_j|);
* a score is a sum of head_dim products (fp32, at most head_dim + 8 roundings,
  each 2^-23 where the tensor core truncates) of magnitude A = scale sum|q|
  max_j(15 s_j + |b_j|) and a few fp32 roundings of it; an error d of every
  score changes the output by at most 2 d max|v|: d = (head_dim + 16) 2^-23 A;
* the store: half a bf16 step of the result (2^-8 relative covers a value that
  crosses a binade).
Chunks that fill the device round keys and values to fp16 as well; their bound is
in test_gpu_kv4_chunks.py, and those here stay within this one too.
"""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"


class Cache:
    """Pools with random contents everywhere, tables of shuffled pages, and the values per sequence."""

    def __init__(self, t, kv, hd, ps, lens, seed, extra=1):
        rng = np.random.default_rng(seed)
        self.t, self.kv, self.hd, self.ps, self.lens = t, kv, hd, ps, list(lens)
        used = [-(-n // ps) for n in lens]
        self.pages = sum(used) + 3
        self.cols = max(used + [0]) + extra
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.cols), -1, np.int32)
        at = 0
        for i, n in enumerate(used):
            self.table[i, :n] = order[at:at + n]
            at += n
        shape = (t, self.pages, kv, ps // 16, 16, hd)
        k = K.bf16(rng.standard_normal(shape).astype(np.float32) * (0.3 + 2 * rng.random(hd).astype(np.float32)) + 0.5)
        v = K.bf16(rng.standard_normal(shape).astype(np.float32))
        self.kq, self.vq = list(K.quantise(k)), list(K.quantise(v))
        self.fill()

    def fill(self):
        self.blocks = K.pack_blocks(*self.kq, *self.vq)
        self.pools = [torch.from_numpy(self.blocks[r].copy()).to(DEV) for r in range(self.t)]
        self.dtable = torch.from_numpy(self.table).to(DEV)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def tokens(self, part, r, s, h):
        """[tokens, hd] float64 of sequence s, and the (step, base) of each token."""
        pages = self.table[s, :-(-self.lens[s] // self.ps)]
        u, st, b = (a[r, pages, h].reshape(-1, a.shape[-1])[:max(self.lens[s], 0)] for a in part)
        return K.values(u, st, b), st[:, 0].astype(np.float64), b[:, 0].astype(np.float64)


def cu_of(rows):
    return torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)


def f64(x):
    return x.float().cpu().numpy().astype(np.float64)


def check_attention(c, rows, heads, seed, window=0, sinks=0, scale=None, cu=True, q=None, out=None, workspace=None):
    n = sum(rows)
    rng = np.random.default_rng(seed)
    group = heads // c.kv
    if q is None:
        q = [torch.from_numpy(rng.standard_normal((n, heads * c.hd)).astype(np.float32)).to(torch.bfloat16).to(DEV)
             for _ in range(c.t)]
    got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of(rows) if cu else None, window=window,
                              sinks=sinks, scale=scale, out=out, workspace=workspace)
    assert tp.tp_device_status() == 0
    sc = c.hd ** -0.5 if scale is None else scale
    worst = 0.0
    for r in range(c.t):
        qr, y = f64(q[r]).reshape(n, heads, c.hd), f64(got[r]).reshape(n, heads, c.hd)
        at = 0
        for s, m in enumerate(rows):
            pos = c.lens[s] - m + np.arange(m)
            for h in range(heads):
                kk, ks, kb = c.tokens(c.kq, r, s, h // group)
                vv, vs, vb = c.tokens(c.vq, r, s, h // group)
                with np.errstate(all="ignore"):
                    want = K.attention(qr[at:at + m, h], kk, vv, pos, sc, window, sinks)
                have = y[at:at + m, h]
                assert np.array_equal(np.isnan(want), np.isnan(have))
                if not len(kk) or not m:
                    assert not have.any()
                    continue
                fin = ~np.isnan(want)
                kb_, vb_ = np.nan_to_num(kb), np.nan_to_num(vb)
                vmax = np.max(15 * vs + np.abs(vb_))
                a = abs(sc) * np.abs(qr[at:at + m, h]).sum(-1, keepdims=True) * np.max(15 * ks + np.abs(kb_))
                tol = (2.0 ** -11 * np.max(15 * vs) + (len(kk) + 16) * 2.0 ** -24 * vmax +
                       2 * (c.hd + 16) * 2.0 ** -23 * a * vmax + 2.0 ** -8 * np.abs(want))
                err = np.where(fin, np.abs(have - np.where(fin, want, 0)), 0)
                assert (err <= np.where(fin, tol, 1)).all(), (r, s, h, float((err / tol).max()))
                worst = max(worst, float((err / tol).max()))
            at += m
    return got, worst


@pytest.mark.parametrize("t,kv,hd,ps", [(1, 1, 64, 16), (2, 2, 128, 64), (3, 1, 128, 32), (2, 5, 64, 128)])
def test_append_then_load(t, kv, hd, ps):
    """Rows of several lengths go to their places, bit for bit; everything else stays as it was."""
    lens, rows = [1, 40, 200, 17, 0, 129], [1, 23, 130, 0, 0, 129]
    c = Cache(t, kv, hd, ps, lens, 1)
    rng = np.random.default_rng(2)
    n = sum(rows)
    wide = [torch.from_numpy(rng.standard_normal((n, 3 * kv * hd)).astype(np.float32) * 5).to(torch.bfloat16).to(DEV)
            for _ in range(t)]
    k, v = [x[:, :kv * hd] for x in wide], [x[:, kv * hd:2 * kv * hd] for x in wide]
    for r in range(t):                                       # constant rows, signed zeros, large and tiny ranges
        k[r][0] = 3.0
        v[r][1] = -0.0
        k[r][2] *= 1e30
        v[r][3] *= 1e-36
        v[r][4, 0] = 0.0
    cu = cu_of(rows)
    tp.tp_kv4_append(k, v, c.pools, c.dtable, c.dlens, cu_rows=cu)
    want = c.blocks.copy()
    hk = [x.float().cpu().numpy().reshape(n, kv, hd) for x in k]
    hv = [x.float().cpu().numpy().reshape(n, kv, hd) for x in v]
    vals = np.zeros((2, t, n, kv, hd))
    at = 0
    for s, m in enumerate(rows):
        for i in range(m):
            pos = lens[s] - m + i
            page, blk, slot = c.table[s, pos // ps], pos % ps // 16, pos % 16
            for r in range(t):
                for which, x in ((0, hk[r][at]), (1, hv[r][at])):
                    u, st, b = K.quantise(x)
                    vals[which, r, at] = (u.astype(np.float32) * st + b).astype(np.float32)
                    rec = want[r, page, :, blk]
                    rec[:, which * 8 * hd + slot * hd // 2:][:, :hd // 2] = u[:, 0::2] | (u[:, 1::2] << 4)
                    bits = (np.concatenate([st, b], -1).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
                    rec[:, 16 * hd + which * 64 + slot * 4:][:, :4] = np.ascontiguousarray(bits).view(np.uint8)
            at += 1
    for r in range(t):
        assert np.array_equal(c.pools[r].cpu().numpy(), want[r])
    lk, lv = tp.tp_kv4_load(c.pools, c.dtable, c.dlens, n, cu_rows=cu, dtype=torch.float32)
    for r in range(t):
        assert np.array_equal(f64(lk[r]).reshape(n, kv, hd), vals[0, r]) and np.array_equal(f64(lv[r]).reshape(n, kv, hd), vals[1, r])
    lk, lv = tp.tp_kv4_load(c.pools, c.dtable, c.dlens, n, cu_rows=cu)
    for r in range(t):
        assert np.array_equal(f64(lk[r]).reshape(n, kv, hd), K.bf16(vals[0, r].astype(np.float32)))
    assert tp.tp_device_status() == 0


def test_append_one_row_each_and_not_finite():
    c = Cache(2, 2, 128, 32, [5, 64, 33], 3)
    rng = np.random.default_rng(4)
    k = [torch.from_numpy(rng.standard_normal((3, 256)).astype(np.float32)).to(torch.bfloat16).to(DEV) for _ in range(2)]
    v = [x.clone() for x in k]
    k[0][0, 7], k[0][1, 130], v[1][2, 0], v[1][2, 255] = float("nan"), float("inf"), 3.3e38, -3.3e38
    v[0][1, 0], v[0][1, 1] = 3.3e38, -3.3e38                  # a range past fp32
    tp.tp_kv4_append(k, v, c.pools, c.dtable, c.dlens)
    lk, lv = tp.tp_kv4_load(c.pools, c.dtable, c.dlens, 3, dtype=torch.float32)
    for x, y in ((k, lk), (v, lv)):
        for r in range(2):
            want = K.values(*K.quantise(x[r].float().cpu().numpy().reshape(3, 2, 128)))
            got = f64(y[r]).reshape(3, 2, 128)
            assert np.array_equal(np.isnan(want), np.isnan(got))
            ok = ~np.isnan(want)
            assert np.array_equal(got[ok], want[ok].astype(np.float32))
    assert tp.tp_device_status() == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 12])
def test_decode_lengths(hd, group):
    """One row per sequence, lengths from none to several pages, at and around block, stage and page edges."""
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1100]
    c = Cache(2, 2, hd, 64, lens, 5)
    check_attention(c, [1] * len(lens), 2 * group, 6, cu=False)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_decode_one_long_sequence(ps):
    """One sequence over all thread blocks: parts joined in order, the same result twice."""
    c = Cache(1, 1, 128, ps, [5003], 7)
    a, _ = check_attention(c, [1], 8, 8, cu=False)
    b, _ = check_attention(c, [1], 8, 8, cu=False)
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 16), (100, 40), (333, 0), (5000, 4), (2 ** 40, 2 ** 40)])
def test_window_and_sinks(window, sinks):
    lens = [1, 3, 70, 130, 700, 0, 1500]
    c = Cache(1, 2, 128, 32, lens, 9)
    check_attention(c, [1] * len(lens), 8, 10, cu=False, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5), (1, 0)])
@pytest.mark.parametrize("group,hd", [(1, 64), (4, 128), (8, 128), (16, 64)])
def test_ragged_rows(group, hd, window, sinks):
    """Chunks of prompts: several rows per sequence, some with none, some longer than a tile."""
    rows = [3, 0, 1, 70, 9, 160]
    lens = [3, 20, 77, 200, 9, 333]
    c = Cache(1, 2, hd, 64, lens, 11)
    check_attention(c, rows, 2 * group, 12, window=window, sinks=sinks)


def test_rows_before_the_first_token():
    """lens shorter than the rows: the rows at negative positions see nothing and give 0."""
    c = Cache(1, 1, 128, 64, [2, 40], 13)
    check_attention(c, [5, 3], 4, 14)


def test_many_short_sequences():
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 90, 300).tolist()
    c = Cache(2, 2, 64, 16, lens, 16)
    check_attention(c, [1] * 300, 6, 17, cu=False)


def test_scales_and_extreme_rows():
    """Scores of any size: a sharp and a flat softmax, zero scale, large and tiny q and steps, constant rows."""
    c = Cache(1, 1, 128, 64, [300, 129], 18)
    c.vq[1][:, :, :, :, 3] = K.bf16(np.float32(1e-30))        # tiny steps
    c.vq[1][:, :, :, :, 5] = 0                                # constant rows
    c.kq[1][:, :, :, :, 6] = 0
    c.fill()
    rng = np.random.default_rng(19)
    for mul in (1.0, 1e-20, 0.0, 30.0):
        q = [torch.from_numpy(rng.standard_normal((2, 4 * 128)).astype(np.float32) * mul).to(torch.bfloat16).to(DEV)]
        for scale in (None, 0.0, -0.3, 2.0):
            check_attention(c, [1, 1], 4, 20, cu=False, q=q, scale=scale)
    c.vq[1][:] = 0                                            # every value row constant
    c.fill()
    check_attention(c, [1, 1], 4, 21, cu=False)


def test_nan_only_where_visible():
    """NaN tokens: rows that see one give NaN, rows that do not are untouched by it; so for what lies past the end."""
    lens = [200, 90]
    c = Cache(1, 1, 128, 64, lens, 22)
    for part in (c.kq, c.vq):
        part[1][:], part[2][:] = np.where(np.isnan(part[2]), part[1], part[1]), part[2]
    page, off = c.table[0, 100 // 64], 100 % 64
    c.vq[1][0, page, 0, off // 16, off % 16], c.vq[2][0, page, 0, off // 16, off % 16] = 0, np.nan
    for s, n in enumerate(lens):                              # everything past the ends
        page, off = c.table[s, n // 64], n % 64
        for o in range(off, 64):
            for part in (c.kq, c.vq):
                part[1][0, page, 0, o // 16, o % 16] = np.inf
                part[2][0, page, 0, o // 16, o % 16] = np.nan
    c.fill()
    # rows at positions 80..199 of sequence 0: those from 100 on see the token without a window
    got, _ = check_attention(c, [120, 30], 8, 23)
    y = f64(got[0])
    assert np.isfinite(y[:20]).all() and np.isnan(y[20:120]).all() and np.isfinite(y[120:]).all()
    got, _ = check_attention(c, [120, 30], 8, 24, window=10, sinks=2)
    y = f64(got[0])
    assert np.isnan(y[20:30]).all() and np.isfinite(y[30:120]).all()


def test_strided_views_streams_and_workspace():
    """q as a part of the merged projection, out as a part of a wider buffer, on another stream, in a graph."""
    lens = [100, 257, 33]
    c = Cache(2, 2, 128, 64, lens, 25)
    rng = np.random.default_rng(26)
    wide = [torch.from_numpy(rng.standard_normal((3, 8 * 128 + 512)).astype(np.float32)).to(torch.bfloat16).to(DEV) for _ in range(2)]
    q = [x[:, :1024] for x in wide]
    buf = [torch.full((3, 1024 + 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = [b[:, 32:1056] for b in buf]
    need = tp.tp_kv4_attention_workspace_size(2, 3, 3, 8, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)     # contents do not matter
    check_attention(c, [1, 1, 1], 8, 27, cu=False, q=q, out=out, workspace=ws)
    assert all((b[:, :32] == 7).all() and (b[:, 1056:] == 7).all() for b in buf)
    plain = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, again))
    step = tp.prepare(tp.tp_kv4_attention, q, c.pools, c.dtable, c.dlens)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, workspace=ws)
    for o in captured:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, captured)) and all(torch.equal(a, b) for a, b in zip(plain, step.result))


def test_bad_pages_and_offsets_are_skipped_and_reported():
    """A page outside the pool hides its tokens and is reported; so are lengths past the table and bad row offsets."""
    lens = [150, 100]
    c = Cache(1, 1, 128, 64, lens, 28)
    good = c.table.copy()
    rng = np.random.default_rng(29)
    q = [torch.from_numpy(rng.standard_normal((2, 512)).astype(np.float32)).to(torch.bfloat16).to(DEV)]
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        c.dtable[0, 1] = bad
        got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens)
        assert tp.tp_device_status() == 1
        assert tp.tp_device_status() == 0
        keep = np.r_[0:64, 128:150]
        for h in range(4):
            kk, vv = c.tokens(c.kq, 0, 0, 0)[0][keep], c.tokens(c.vq, 0, 0, 0)[0][keep]
            want = K.attention(f64(q[0])[0:1, h * 128:(h + 1) * 128], kk, vv, [10 ** 6], 128 ** -0.5)
            assert np.abs(f64(got[0])[0, h * 128:(h + 1) * 128] - want[0]).max() < 0.02
    c.dtable.copy_(torch.from_numpy(good))
    c.dlens[1] = 10 ** 6                                             # past the table
    tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens)
    assert tp.tp_device_status() == 1
    k = [torch.ones((2, 128), dtype=torch.bfloat16, device=DEV)]
    before = c.pools[0].clone()
    c.dlens.copy_(torch.tensor([10 ** 6, 0], dtype=torch.int32))
    tp.tp_kv4_append(k, k, c.pools, c.dtable, c.dlens)
    assert tp.tp_device_status() == 1 and torch.equal(before, c.pools[0])
    lk, _ = tp.tp_kv4_load(c.pools, c.dtable, c.dlens, 2)
    assert tp.tp_device_status() == 1 and not lk[0].any()
    c.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
    for cu in ([0, 3, 2], [-1, 1, 2], [0, 1, 5], [1, 1, 1]):
        cu_t = torch.tensor(cu, dtype=torch.int32, device=DEV)
        tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_t)
        torch.cuda.synchronize()
        tp.tp_device_status()
        tp.tp_kv4_append(k, k, c.pools, c.dtable, c.dlens, cu_rows=cu_t)
        torch.cuda.synchronize()
        tp.tp_device_status()


def test_pool_past_two_gigabytes():
    """Block offsets past 32 bits."""
    pages = 2 ** 31 // (2 * 128 * 136) + 40                          # 2.15 GB and more at 34816 bytes a page
    pool = [tp.tp_kv4_pool(pages, 128, 2, 128)]
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([200], dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(30)
    k = [torch.from_numpy(rng.standard_normal((200, 256)).astype(np.float32)).to(torch.bfloat16).to(DEV)]
    cu = cu_of([200])
    tp.tp_kv4_append(k, k, pool, table, lens, cu_rows=cu)
    lk, lv = tp.tp_kv4_load(pool, table, lens, 200, cu_rows=cu, dtype=torch.float32)
    want = K.values(*K.quantise(k[0].float().cpu().numpy().reshape(200, 2, 128))).astype(np.float32)
    assert np.array_equal(lk[0].cpu().numpy().reshape(200, 2, 128), want) and torch.equal(lk[0], lv[0])
    q = [torch.from_numpy(rng.standard_normal((1, 1024)).astype(np.float32)).to(torch.bfloat16).to(DEV)]
    got = f64(tp.tp_kv4_attention(q, pool, table, lens)[0])
    for h in range(8):
        w = want[:, h // 4].astype(np.float64)
        ref = K.attention(f64(q[0])[:, h * 128:(h + 1) * 128], w, w, [199], 128 ** -0.5)
        assert np.abs(got[0, h * 128:(h + 1) * 128] - ref[0]).max() < 0.03
    assert tp.tp_device_status() == 0

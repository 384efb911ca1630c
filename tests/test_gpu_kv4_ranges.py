"""Attention over cached values of any size, for chunks that fill the device and
for single rows, against the float64 oracle of the other attention tests.

The bounds are those of test_gpu_kv4_chunks.py and test_gpu_kv4.py: every term is
relative to the values, so a factor on all of them changes nothing."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from test_gpu_kv4 import Cache, DEV, check_attention, cu_of
from test_gpu_kv4_chunks import check, rows_of, run

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


def scaled(c, factor):
    """Every value of the cache times `factor`."""
    c.vq[1], c.vq[2] = K.bf16(c.vq[1] * np.float32(factor)), K.bf16(c.vq[2] * np.float32(factor))
    c.fill()
    return c


@pytest.mark.parametrize("factor", [1e6, 1e20])
@pytest.mark.parametrize("hd,window,sinks", [(128, 0, 0), (64, 0, 0), (128, 50, 5)])
def test_chunks_of_large_values(hd, window, sinks, factor):
    """Lengths that leave the last step of 128 tokens partly empty, and rows whose first tokens see little of a step."""
    c = scaled(Cache(1, 8, hd, 64, [300, 129, 70], 61), factor)
    run(c, [60, 40, 70], 64, 62, window=window, sinks=sinks)


@pytest.mark.parametrize("factor", [1.0, 1e3, 1e10])
def test_chunks_over_tokens_of_zero_value(factor):
    """One token with values and 4185 of value 0, each with 2^-17 of its weight: together they are 3 % of the
    denominator, whatever the values' size."""
    c = Cache(1, 8, 128, 64, [4096 + 90], 63)
    page = c.table[0, 0]
    token = [c.vq[i][0, page, :, 0, 0].copy() for i in range(3)]
    for part, base in ((c.kq, -1.0), (c.vq, 0.0)):
        part[1][:], part[2][:] = 0, base                     # constant rows: a step of 0, the base is the value
    c.kq[2][0, page, :, 0, 0] = 0
    for i in range(3):
        c.vq[i][0, page, :, 0, 0] = token[i]
    scaled(c, factor)
    q = [torch.ones((90, 64 * 128), dtype=torch.bfloat16, device=DEV)]
    scale = 17 * np.log(2) / 128                             # q . k is -128 but for the first token
    got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of([90]), scale=scale)
    assert tp.tp_device_status() == 0
    check(c, q, got, [90], 64, scale=scale)


def check_some(c, q, got, m, heads, rows, window):
    """The bound of `check` for rows `rows` of one sequence's last m, with the largest value that each row sees in the
    place of the sequence's largest."""
    group, n = heads // c.kv, c.lens[0]
    for h in range(heads):
        kk, ks, kb = c.tokens(c.kq, 0, 0, h // group)
        vv, vs, vb = c.tokens(c.vq, 0, 0, h // group)
        x, y = (t[0].double().cpu().numpy().reshape(m, heads, c.hd)[rows, h] for t in (q, got))
        pos, j = (n - m + np.asarray(rows))[:, None], np.arange(n)[None, :]
        see = (j <= pos) & ((j > pos - window) if window else True)
        score = np.where(see, c.hd ** -0.5 * (x @ kk.T), -np.inf)
        p = np.exp(score - score.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want = p @ vv
        vmost = np.where(see, 15 * vs + np.abs(vb), 0).max(1, keepdims=True)
        kmost, absq = (15 * ks + np.abs(kb)).max(), np.abs(x).sum(1, keepdims=True)
        D = c.hd ** -0.5 * (2.0 ** -11 * (np.abs(x) @ np.abs(kk).T).max(1, keepdims=True) +
                            (2.0 ** -24 + (c.hd + 16) * 2.0 ** -23) * kmost * absq)
        spread = np.stack([a @ np.abs(vv - w) for a, w in zip(p, want)])
        tol = (2 * 2.0 ** -11 + (n + 16) * 2.0 ** -23) * vmost + np.expm1(2 * D) * spread + 2.0 ** -8 * np.abs(want)
        err = np.abs(y - want)
        assert (err <= tol).all(), (h, float((err / tol).max()))


@pytest.mark.parametrize("factor", [1e4, 1e9, 1e20])
@pytest.mark.parametrize("window", [0, 20])
def test_a_large_value_that_is_not_seen_costs_nothing(window, factor):
    """One token's values are `factor` times as large as the others'.  Rows that see none of its group of 32 tokens
    (before it, or with the window past the group) are as good as without it, beside rows that see it."""
    c = Cache(1, 8, 128, 64, [512], 64)
    page, off = c.table[0, 448 // 64], 448 % 64
    for i in (1, 2):
        c.vq[i][0, page, :, off // 16, off % 16] = K.bf16(c.vq[i][0, page, :, off // 16, off % 16] * np.float32(factor))
    c.fill()
    rng = np.random.default_rng(65)
    q = [torch.from_numpy(rng.standard_normal((100, 64 * 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)]
    got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of([100]), window=window)
    assert tp.tp_device_status() == 0
    rows = [i for i in range(100) if 412 + i < 448 or (window and 412 + i - window >= 479)]
    check_some(c, q, got, 100, 64, rows, window)


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("factor", [1e37, 1e-36])
def test_chunks_of_the_largest_and_smallest_values(hd, factor):
    c = scaled(Cache(1, 8, hd, 64, [300, 129, 70], 66), factor)
    run(c, [60, 40, 70], 64, 67)


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("factor", [1e37, 1e20, 1e-30])
def test_chunks_of_the_largest_and_smallest_keys(hd, factor):
    """q is as much smaller as the keys are larger."""
    c = Cache(1, 8, hd, 64, [300, 129, 70], 68)
    for i in (1, 2):
        c.kq[i] = K.bf16(c.kq[i] * np.float32(factor))
    c.fill()
    q = [(x.float() / factor).to(torch.bfloat16) for x in rows_of(c, [60, 40, 70], 64, 69)]
    got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of([60, 40, 70]))
    assert tp.tp_device_status() == 0
    check(c, q, got, [60, 40, 70], 64)


@pytest.mark.parametrize("hd,group", [(128, 8), (64, 3), (128, 16)])
@pytest.mark.parametrize("factor", [1e34, 1e35, 1e36, 1e37, 1e-33])
def test_rows_of_the_largest_and_smallest_values(hd, group, factor):
    """Single rows and a few: sequences that a warp holds, and one that is cut into parts."""
    c = scaled(Cache(1, 2, hd, 64, [300, 129, 70, 1, 2500], 73), factor)
    check_attention(c, [1] * 5, 2 * group, 74, cu=False)
    check_attention(c, [3, 2, 4, 1, 2], 2 * group, 75)


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("factor", [1e37, 1e20, 1e-30, 3e-35])
def test_rows_of_the_largest_and_smallest_keys(hd, factor):
    """q is as much smaller as the keys are larger."""
    lens = [300, 129, 70, 1, 2500]
    c = Cache(1, 2, hd, 64, lens, 76)
    for i in (1, 2):
        c.kq[i] = K.bf16(c.kq[i] * np.float32(factor))
    c.fill()
    for rows, seed in (([1] * 5, 77), ([3, 2, 4, 1, 2], 78)):
        q = [(x.float() / factor).to(torch.bfloat16) for x in rows_of(c, rows, 16, seed)]
        check_attention(c, rows, 16, seed, q=q)


@pytest.mark.parametrize("factor", [1e4, 1e9, 1e20])
@pytest.mark.parametrize("window", [0, 20])
def test_a_large_value_that_a_row_does_not_see_costs_it_nothing(window, factor):
    """The same for a few rows, which share their tokens' loads: the token among the last of a block, seen by the later
    rows alone, and with the window by the earlier ones alone."""
    c = Cache(1, 8, 128, 64, [512], 79)
    big = 507 if window == 0 else 488
    page, off = c.table[0, big // 64], big % 64
    for i in (1, 2):
        c.vq[i][0, page, :, off // 16, off % 16] = K.bf16(c.vq[i][0, page, :, off // 16, off % 16] * np.float32(factor))
    c.fill()
    rng = np.random.default_rng(80)
    q = [torch.from_numpy(rng.standard_normal((8, 16 * 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)]
    got = tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of([8]), window=window)
    assert tp.tp_device_status() == 0
    rows = [i for i in range(8) if 504 + i < big or (window and 504 + i - window >= big)]
    assert rows == ([0, 1, 2] if window == 0 else [4, 5, 6, 7])
    check_some(c, q, got, 8, 16, rows, window)

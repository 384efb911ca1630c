"""Fork, compaction and beam selection against the oracle: page numbers, counters
and tokens exactly, pool contents byte for byte."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=DEV)


def make_pools(t, layers, pages, kv, ps, hd, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randint(0, 256, (layers, pages, kv, ps // 16, 16 * (hd + 8)), dtype=torch.uint8, device=DEV, generator=g)
            for _ in range(t)]


def tables(rng, rows, cols, ps, pages, share):
    """Random tables; some pages stand in several rows."""
    lens = rng.integers(0, cols * ps + 1, rows)
    table = np.full((rows, cols), -1, np.int32)
    order = rng.permutation(pages)
    at = 0
    for i in range(rows):
        n = -(-int(lens[i]) // ps)
        for c in range(n):
            if i and rng.random() < share and table[i - 1, c] >= 0:
                table[i, c] = table[i - 1, c]
            else:
                table[i, c] = order[at % pages]
                at += 1
    return table, lens.astype(np.int32)


def check_fork(table, lens, parents, grow, ps, pages, held=None, pools=None):
    want = K.fork(table, lens, parents, grow, ps, pages, held)
    before = [p.clone() for p in pools] if pools else None
    g = dev(grow) if hasattr(grow, "__len__") else grow
    got = tp.tp_kv_fork(dev(table), dev(lens), dev(parents), pools, grow=g, page_size=ps, pages=pages,
                        held=None if held is None else dev(held, torch.uint8))
    for a, b in zip(got[:3], want[:3]):
        assert np.array_equal(a.cpu().numpy(), b)
    assert got[3].tolist() == want[3]
    if pools:
        for p, b in zip(pools, before):
            for src, dst in want[4]:
                b[:, dst] = b[:, src]
            assert torch.equal(p, b)
    return got


@pytest.mark.parametrize("seed", range(6))
def test_fork_random(seed):
    rng = np.random.default_rng(seed)
    ps = int(rng.choice([16, 32, 64, 128]))
    rows, cols = int(rng.integers(1, 40)), int(rng.integers(1, 9))
    pages = rows * cols * 2 + 4
    table, lens = tables(rng, rows, cols, ps, rows * cols, 0.5)
    m = int(rng.integers(1, 60))
    parents = rng.integers(-1, rows + 1, m)
    grow = rng.integers(-2 * ps, 2 * ps, m) if seed % 2 else 1
    held = (rng.random(pages) < 0.2).astype(np.uint8) if seed % 3 == 0 else None
    pools = make_pools(2, 2, pages, 1, ps, 64, seed) if seed < 4 else None
    check_fork(table, lens, parents, grow, ps, pages, held, pools)
    assert tp.tp_device_status() == 0


def test_fork_runs_out_of_pages_and_keeps_bad_entries():
    rng = np.random.default_rng(10)
    table, lens = tables(rng, 6, 4, 16, 24, 0.0)
    check_fork(table, lens, [0, 0, 1, 1, 2, 3, 4, 5, 5], 20, 16, 24)
    bad = table.copy()
    bad[0, 0], bad[2, 0], bad[3, 0] = -1, 24, 2 ** 31 - 1
    lens = np.full(6, 50, np.int32)
    full = np.where(table < 0, 5, bad)
    check_fork(full.astype(np.int32), lens, [0, 1, 2, 3, 3], 1, 16, 24, pools=make_pools(1, 1, 24, 1, 16, 64, 1))
    check_fork(full.astype(np.int32), [-5, 10 ** 9, 0, 1, 2, 3], [0, 1, 2], [2 ** 31 - 1, -2 ** 31, 0], 16, 24)


def test_fork_large_tables():
    """More rows and pages than threads."""
    rng = np.random.default_rng(11)
    rows, cols, ps = 700, 40, 16
    pages = rows * cols + 5000
    table, lens = tables(rng, rows, cols, ps, rows * cols, 0.3)
    check_fork(table, lens, rng.integers(0, rows, 900), 3, ps, pages)


def test_fork_empty():
    got = tp.tp_kv_fork(dev(np.zeros((2, 3))), dev([5, 5]), dev(np.zeros(0)), None, page_size=16, pages=9)
    assert got[0].shape == (0, 3) and got[2].tolist() == [0] * 9 and got[3].tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("seed", range(6))
def test_compact_random(seed):
    rng = np.random.default_rng(100 + seed)
    ps = int(rng.choice([16, 32, 64, 128]))
    rows, cols = int(rng.integers(1, 50)), int(rng.integers(1, 12))
    pages = rows * cols * int(rng.integers(1, 5)) + 3
    table, lens = tables(rng, rows, cols, ps, pages, 0.4)
    if seed == 5:
        table[0, 0], lens[0] = pages, cols * ps + 9
    held = (rng.random(pages) < 0.15).astype(np.uint8) if seed % 2 else None
    pools = make_pools(2, 2, pages, 1, ps, 64, seed)
    want = K.compact(table, lens, ps, pages, held)
    before = [p.clone() for p in pools]
    got = tp.tp_kv_compact(dev(table), dev(lens), pools, held=None if held is None else dev(held, torch.uint8))
    for a, b in zip(got[:2], want[:2]):
        assert np.array_equal(a.cpu().numpy(), b)
    assert got[2].tolist() == want[2]
    for p, b in zip(pools, before):
        for src, dst in want[3]:
            b[:, dst] = b[:, src]
        assert torch.equal(p, b)
    # compact again: nothing moves
    again = tp.tp_kv_compact(got[0], dev(lens), pools, held=None if held is None else dev(held, torch.uint8))
    assert again[2].tolist()[2] == 0 or held is not None
    assert tp.tp_device_status() == 0


# ---------------------------------------------------------------- beams

def split(x, t):
    """Vocab shards of [rows, vocab]: the ceil rule of the LM head."""
    per = -(-x.shape[1] // t)
    return [x[:, r * per:(r + 1) * per].contiguous() for r in range(t)]


def check_beams(x, scores, k, t=1, finished=None, eos=0, shards=None):
    """x [items, beams, vocab] of the dtype the kernel reads."""
    items, beams, vocab = x.shape
    sh = shards or split(x.reshape(items * beams, vocab), t)
    got = tp.tp_beam_select(sh, scores, k, finished=finished, eos=eos)
    want = K.beam_select(x.double().cpu().numpy(), scores.double().cpu().numpy(), k,
                         None if finished is None else finished.cpu().numpy(), eos)
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[2].cpu().numpy(), want[2])
    s, w = got[0].double().cpu().numpy(), want[0]
    fin = np.isfinite(w)
    assert np.array_equal(fin, np.isfinite(s))
    # fp64 until the store; the exponentials are fp32 (2 ulp: at most 2^-22 of the sum)
    s, w = s[fin], w[fin]
    assert (np.abs(s - w) <= 2.0 ** -24 * np.abs(w) + 2.0 ** -22).all()
    assert tp.tp_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("items,beams,k,vocab,t", [(1, 1, 1, 1, 1), (3, 4, 4, 1000, 2), (2, 5, 10, 4099, 3), (1, 8, 64, 20011, 4),
                                                    (7, 2, 4, 333, 8), (1, 64, 64, 130, 1), (2, 1, 7, 151936, 2)])
def test_beams(items, beams, k, vocab, t, dtype):
    g = torch.Generator(device=DEV).manual_seed(items * 1000 + vocab)
    x = (torch.randn((items, beams, vocab), device=DEV, generator=g) * 3).to(dtype)
    scores = -5 * torch.rand((items, beams), device=DEV, generator=g)
    check_beams(x, scores, k, t)
    fin = torch.rand((items, beams), device=DEV, generator=g) < 0.4
    check_beams(x, scores, k, t, finished=fin, eos=vocab - 1)


@pytest.mark.parametrize("vocab", [100, 9000, 60000])
def test_beams_ties(vocab):
    """Equal logits: the lowest (beam, token) first, also where more tie than are ranked at once."""
    x = torch.zeros((2, 3, vocab), device=DEV)
    check_beams(x, torch.zeros((2, 3), device=DEV), 9, 2)
    x[:, :, 1::2] = -0.0
    x[0, 1, vocab // 2:] = 1.0
    check_beams(x, torch.zeros((2, 3), device=DEV), 64, 2)
    x = torch.randint(0, 3, (2, 3, vocab), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).float()
    x[1, 2] = x[1, 0]
    check_beams(x.to(torch.bfloat16), torch.zeros((2, 3), device=DEV), 20, 1)


def test_beams_masked_and_not_finite():
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((6, 3, 5000), device=DEV, generator=g)
    scores = -torch.rand((6, 3), device=DEV, generator=g)
    x[0, :, 3:] = -float("inf")                              # fewer continuations than k
    x[1, 0], x[1, 1, 17] = -float("inf"), float("nan")       # rows that offer nothing
    x[2, 0, 5] = float("inf")
    scores[3, 0], scores[3, 1] = -float("inf"), float("nan")
    x[4] = -float("inf")
    x[5] = torch.finfo(torch.float32).min                    # a mask of the type's lowest value
    check_beams(x, scores, 12, 2)
    check_beams(x.to(torch.bfloat16), scores, 12, 4)


def test_beams_strided_and_gathered():
    """Rows at odd offsets and strides; one gathered matrix, and a shard of width 0."""
    g = torch.Generator(device=DEV).manual_seed(4)
    big = torch.randn((6, 3001), device=DEV, generator=g).to(torch.bfloat16)
    scores = -torch.rand((2, 3), device=DEV, generator=g)
    x = big[:, 5:2998]
    check_beams(x.reshape(2, 3, -1), scores, 8, shards=[x])
    check_beams(x.reshape(2, 3, -1), scores, 8, shards=[x[:, :1001], None, x[:, 1001:]])


def test_beam_step_through_fork():
    """A selection's rows are the fork's parents: -1 gives an empty row."""
    x = torch.full((1, 2, 3), -float("inf"), device=DEV)
    x[0, 0, 1] = 0.0
    s, rows, tokens = tp.tp_beam_select([x[0]], torch.tensor([[0.0, -float("inf")]], device=DEV), 2)
    assert rows.tolist() == [[0, -1]] and tokens.tolist() == [[1, -1]]
    t, n, _, info = tp.tp_kv_fork(dev([[4, 2], [1, 3]]), dev([17, 20]), rows.flatten(), None, page_size=16, pages=6)
    assert t.tolist() == [[4, 2], [-1, -1]] and n.tolist() == [18, 0] and info.tolist() == [2, 0, 0, 0]


def test_pages_and_beams_in_a_graph():
    g = torch.cuda.CUDAGraph()
    x = torch.randn((8, 2000), device=DEV)
    scores = torch.zeros((2, 4), device=DEV)
    table, lens = dev(np.arange(24).reshape(8, 3)), dev([40] * 8)
    pools = make_pools(1, 1, 40, 1, 16, 64, 5)
    run = lambda: tp.tp_kv_fork(table, lens, tp.tp_beam_select([x], scores, 4)[1].flatten(), pools)  # noqa: E731
    plain = [y.clone() for y in run()]
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = run()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(plain, got))


def test_compact_large_tables():
    """More pages than one block takes."""
    rng = np.random.default_rng(12)
    rows, cols, ps, pages = 700, 40, 16, 60000
    table, lens = tables(rng, rows, cols, ps, pages, 0.3)
    want = K.compact(table, lens, ps, pages)
    got = tp.tp_kv_compact(dev(table), dev(lens), None, page_size=ps, pages=pages)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
    assert got[2].tolist() == want[2]


@pytest.mark.parametrize("rows,cols,pages", [(2048, 31, 12288), (1, 65535, 12288), (2048, 32, 12289), (2049, 1, 100)])
def test_fork_at_the_limits_of_one_block(rows, cols, pages):
    rng = np.random.default_rng(13)
    table = rng.integers(0, pages, (rows, cols)).astype(np.int32)
    lens = rng.integers(0, min(cols, max(1, pages // rows)) * 16 + 1, rows).astype(np.int32)
    check_fork(table, lens, rng.integers(0, rows, rows), 1, 16, pages)


@pytest.mark.parametrize("rows,cols", [(2048, 16), (1, 32768), (2047, 17), (32, 1025)])
def test_fork_at_the_most_entries_of_one_block(rows, cols):
    rng = np.random.default_rng(14)
    pages = 12288
    table = rng.integers(0, pages, (rows, cols)).astype(np.int32)
    lens = rng.integers(0, min(cols, max(1, pages // rows)) * 16 + 1, rows).astype(np.int32)
    check_fork(table, lens, rng.integers(0, rows, rows), 1, 16, pages)


@pytest.mark.parametrize("rows,cols,pages", [(2048, 8, 12288), (1, 16384, 12288), (16, 1025, 12288), (2048, 8, 12289)])
def test_compact_at_the_limits_of_one_block(rows, cols, pages):
    rng = np.random.default_rng(15)
    table, lens = tables(rng, rows, cols, 16, pages, 0.3)
    want = K.compact(table, lens, 16, pages)
    got = tp.tp_kv_compact(dev(table), dev(lens), None, page_size=16, pages=pages)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
    assert got[2].tolist() == want[2]

"""Decode-loop operators on the CPU: refusals of the C ABI and of the binding
(before any CUDA call), the cache's addressing with bad pages, and the oracle
against hand-made examples."""

import ctypes

import numpy as np
import pytest
import torch

from megatron_tensor_layers_gb300 import _lib as tp
from megatron_tensor_layers_gb300.build import build
from oracle import kv_oracle as K

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build()
    return tp.load()


def arr(n, v=FAKE):
    a = (ctypes.c_void_p * n)()
    for i in range(n):
        a[i] = v
    return a


def test_append_and_load_reject_on_host(lib):
    two = arr(2)
    ok = dict(t=2, n=4, ns=4, kv=2, hd=128, ldk=256, ldv=256, pages=8, ps=64, mb=4, k=two, v=two, pool=two, table=FAKE,
              lens=FAKE, cu=None)

    def append(**kw):
        a = {**ok, **kw}
        return lib.tp_kv4_append(a["t"], a["n"], a["ns"], a["kv"], a["hd"], a["k"], a["ldk"], a["v"], a["ldv"], a["pool"],
                                 a["pages"], a["ps"], a["table"], a["mb"], a["lens"], a["cu"], None)

    def load(**kw):
        a = {**ok, "dt": 1, **kw}
        return lib.tp_kv4_load(a["t"], a["n"], a["ns"], a["kv"], a["hd"], a["pool"], a["pages"], a["ps"], a["table"],
                               a["mb"], a["lens"], a["cu"], a["k"], a["ldk"], a["v"], a["ldv"], a["dt"], None)

    for f in (append, load):
        assert f(t=0) == 1 and f(t=9) == 1 and f(n=-1) == 1 and f(kv=0) == 1 and f(pages=0) == 1 and f(mb=0) == 1
        assert f(hd=96) == 4 and f(ps=48) == 4 and f(ps=256) == 4
        assert f(n=5) == 1                               # one row per sequence without cu_rows
        assert f(pool=None) == 1 and f(table=None) == 1 and f(lens=None) == 1
        assert f(ldk=255) == 1 and f(ldv=128) == 1
        assert f(k=arr(2, FAKE + 2)) == 3 and f(pool=arr(2, FAKE + 8)) == 3
        assert f(mb=2 ** 30) == 4 and f(n=2 ** 31, cu=FAKE) == 4
    assert append(ldk=260) == 3 and load(ldk=258) == 3   # row stride not 16-byte aligned
    assert append(k=None) == 1
    assert load(k=None, v=None) == 1 and load(dt=5) == 4
    none = arr(2, None)
    assert append(n=0, ns=0, k=none, v=none) == 0 and load(n=0, ns=0, k=none, v=none) == 0


def test_attention_rejects_on_host(lib):
    two = arr(2)
    need = lib.tp_kv4_attention_workspace_size(2, 4, 4, 8, 2, 128)
    assert need > 0
    ok = dict(n=4, ns=4, heads=8, kv=2, hd=128, ldq=1024, ldo=1024, q=two, out=two, scale=0.1, window=0, sinks=0, ws=FAKE,
              bytes=need)

    def f(**kw):
        a = {**ok, **kw}
        return lib.tp_kv4_attention(2, a["n"], a["ns"], a["heads"], a["kv"], a["hd"], a["q"], a["ldq"], two, 8, 64, FAKE, 4,
                                    FAKE, None, a["scale"], a["window"], a["sinks"], a["ws"], a["bytes"], a["out"], a["ldo"],
                                    None)

    assert f(heads=7) == 2 and f(heads=0) == 1 and f(heads=2 * 129) == 4
    assert f(scale=float("nan")) == 1 and f(scale=float("inf")) == 1 and f(window=-1) == 1 and f(sinks=-1) == 1
    assert f(bytes=need - 1) == 7 and f(ws=None) == 7 and f(ws=FAKE + 128) == 3
    assert f(ldq=1023) == 1 and f(ldo=1028) == 3 and f(q=arr(2, FAKE + 4)) == 3 and f(out=None) == 1
    assert f(n=0, ns=0, q=arr(2, None), out=arr(2, None), ws=None, bytes=0) == 0
    for bad in (dict(t=0), dict(hd=80), dict(heads=9)):
        a = dict(t=2, hd=128, heads=8, **{}) | bad
        assert lib.tp_kv4_attention_workspace_size(a["t"], 4, 4, a["heads"], 2, a["hd"]) == 0


def test_pages_reject_on_host(lib):
    two = arr(2)
    ws = lib.tp_kv_pages_workspace_size(4, 8)
    assert ws > 0 and lib.tp_kv_pages_workspace_size(-1, 8) == 0 and lib.tp_kv_pages_workspace_size(4, 0) == 0
    ok = dict(t=2, ri=4, ro=4, mb=4, ps=16, pages=8, table=FAKE, lens=FAKE, parents=FAKE, pool=two, layers=1, pb=1024,
              to=FAKE * 2, lo=FAKE * 3, refs=FAKE * 4, info=FAKE * 5, ws=FAKE * 6, bytes=ws)

    def fork(**kw):
        a = {**ok, **kw}
        return lib.tp_kv_fork(a["t"], a["ri"], a["ro"], a["mb"], a["ps"], a["pages"], a["table"], a["lens"], a["parents"],
                              None, 1, None, a["pool"], a["layers"], a["pb"], a["to"], a["lo"], a["refs"], a["info"],
                              a["ws"], a["bytes"], None)

    def compact(**kw):
        a = {**ok, **kw}
        return lib.tp_kv_compact(a["t"], a["ri"], a["mb"], a["ps"], a["pages"], a["table"], a["lens"], None, a["pool"],
                                 a["layers"], a["pb"], a["to"], a["refs"], a["info"], a["ws"], a["bytes"], None)

    for f in (fork, compact):
        assert f(t=0) == 1 and f(mb=0) == 1 and f(pages=0) == 1 and f(ri=-1) == 1
        assert f(ps=24) == 4 and f(ri=2 ** 30, ro=2 ** 30) in (4, 7)
        assert f(refs=None) == 1 and f(info=None) == 1 and f(to=None) == 1 and f(table=None) == 1
        assert f(bytes=ws - 1) == 7 and f(ws=None) == 7
        assert f(pb=1000) == 3 and f(pb=0) == 1 and f(layers=0) == 1 and f(pool=arr(2, FAKE + 4)) == 3
        assert f(to=FAKE) == 1                           # in place
    assert fork(parents=None) == 1 and fork(lo=FAKE + 4) == 1


def test_beam_rejects_on_host(lib):
    two = arr(2)
    cols = (ctypes.c_int64 * 2)(5, 5)
    need = lib.tp_beam_workspace_size(2, 3, 3, 10)
    assert need > 0 and lib.tp_beam_workspace_size(2, 65, 3, 10) == 0 and lib.tp_beam_workspace_size(2, 3, 0, 10) == 0
    ok = dict(t=2, items=2, beams=3, k=3, cols=cols, logits=two, ldl=cols, dt=0, fin=None, eos=-1, ws=FAKE, bytes=need,
              so=FAKE)

    def f(**kw):
        a = {**ok, **kw}
        return lib.tp_beam_select(a["t"], a["items"], a["beams"], a["k"], a["cols"], a["logits"], a["ldl"], a["dt"], FAKE,
                                  a["fin"], a["eos"], a["so"], FAKE, FAKE, a["ws"], a["bytes"], None)

    assert f(t=0) == 1 and f(beams=0) == 1 and f(k=0) == 1 and f(beams=65) == 4 and f(k=65) == 4 and f(dt=3) == 4
    assert f(cols=(ctypes.c_int64 * 2)(0, 0)) == 1 and f(cols=(ctypes.c_int64 * 2)(5, -1)) == 1
    assert f(ldl=(ctypes.c_int64 * 2)(5, 4)) == 1 and f(logits=arr(2, FAKE + 1)) == 3 and f(logits=arr(2, None)) == 1
    assert f(fin=FAKE) == 1 and f(fin=FAKE, eos=10) == 1
    assert f(bytes=need - 1) == 7 and f(so=None) == 1
    assert f(items=0, ws=None, bytes=0) == 0


def test_binding_refuses_before_any_call(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    pool = lambda hd=128, kv=2, ps=32, pages=5, layers=None: tp.tp_kv4_pool(pages, ps, kv, hd, layers=layers, device="cpu")  # noqa: E731
    assert pool().shape == (5, 2, 2, 16 * 136) and pool(layers=3).shape == (3, 5, 2, 2, 16 * 136)
    with pytest.raises(ValueError):
        tp.tp_kv4_pool(4, 48, 2, 128, device="cpu")
    k, table, lens = [z(3, 256)], i32(3, 4), i32(3)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_kv4_append(k, k, [pool()], table, lens)
    with pytest.raises(ValueError, match="shape"):
        tp.tp_kv4_append([z(3, 128)], k, [pool()], table, lens)
    with pytest.raises(ValueError, match="one row"):
        tp.tp_kv4_append([z(4, 256)], [z(4, 256)], [pool()], table, lens)
    with pytest.raises(ValueError, match="dimensions"):
        tp.tp_kv4_append(k, k, [pool(layers=2)], table, lens)
    with pytest.raises(TypeError, match="dtype"):
        tp.tp_kv4_append(k, k, [pool()], table.long(), lens)
    with pytest.raises(ValueError, match="contiguous"):
        tp.tp_kv4_append(k, k, [pool()], i32(4, 3).t(), lens)
    with pytest.raises(ValueError, match="same number"):
        tp.tp_kv4_append(k, k, [pool(), pool()], table, lens)
    with pytest.raises(ValueError, match="columns"):
        tp.tp_kv4_attention([z(3, 384)], [pool()], table, lens)
    with pytest.raises(ValueError, match="negative"):
        tp.tp_kv4_attention([z(3, 512)], [pool()], table, lens, window=-1)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_kv4_attention([z(3, 512)], [pool()], table, lens, workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_kv4_load([pool()], table, lens, 3)
    with pytest.raises(ValueError, match="needed"):
        tp.tp_kv_fork(table, lens, i32(3), None)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_kv_fork(table, lens, i32(3), [pool(layers=1)])
    with pytest.raises(ValueError, match="shape"):
        tp.tp_kv_fork(table, i32(2), i32(3), [pool(layers=1)])
    with pytest.raises(ValueError, match="32 bits"):
        tp.tp_kv_fork(table, lens, i32(3), [pool(layers=1)], grow=2 ** 31)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_kv_compact(table, lens, [pool(layers=1)])
    f = torch.zeros((2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_beam_select([z(6, 10)], f, 3)
    with pytest.raises(ValueError, match="width"):
        tp.tp_beam_select([z(5, 10)], f, 3)
    with pytest.raises(ValueError, match="beams and k"):
        tp.tp_beam_select([z(6, 10)], f, 65)
    with pytest.raises(ValueError, match="eos"):
        tp.tp_beam_select([z(6, 10)], f, 3, finished=torch.zeros((2, 3), dtype=torch.bool))


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("hd", [64, 128])
def test_block_addresses(lib, page_size, hd):
    """The kernels' addressing, run on the host: every block of a sequence, its end, and bad pages."""
    pages, kv, rec = 7, 3, 16 * (hd + 8)
    row = np.array([4, 0, 6, 7, -1, 2 ** 31 - 1, -2 ** 31], dtype=np.int32)      # four of them bad
    at = lambda head, pos, p=pages: lib.tp_debug_kv4_block(row.ctypes.data, len(row), p, page_size, kv, hd, head, pos)  # noqa: E731
    for i in range(3):
        for head in range(kv):
            for off in range(0, page_size, 5):
                want = ((int(row[i]) * kv + head) * (page_size // 16) + off // 16) * rec
                assert at(head, i * page_size + off) == want
                assert want + rec <= pages * kv * page_size * (hd + 8)
    for i in range(3, len(row) + 2):
        assert at(0, i * page_size) == -1 and at(0, (i + 1) * page_size - 1) == -1
    assert at(0, -1) == -1 and at(kv, 0) == -1 and at(0, 2 ** 40) == -1
    # a pool past 2^31 bytes: offsets keep 64 bits
    big = np.array([2 ** 30], dtype=np.int32)
    got = lib.tp_debug_kv4_block(big.ctypes.data, 1, 2 ** 31 - 1, page_size, kv, hd, 2, page_size - 1)
    assert got == ((2 ** 30 * kv + 2) * (page_size // 16) + page_size // 16 - 1) * rec


def test_oracle_format():
    x = np.array([[0.0, 15.0, 7.4, -0.0], [2.0, 2.0, 2.0, 2.0]], np.float32)
    u, s, b = K.quantise(x)
    assert u[0].tolist() == [0, 15, 7, 0] and s[0, 0] == 1 and b[0, 0] == 0 and not np.signbit(b[0, 0])
    assert u[1].tolist() == [0] * 4 and s[1, 0] == 0 and K.values(u, s, b)[1].tolist() == [2.0] * 4
    for bad in ([np.nan, 1, 2, 3], [np.inf, 1, 2, 3], [-np.inf, 1, 2, 3], [3.38e38, -3.38e38, 0, 0]):
        u, s, b = K.quantise(np.array([bad], np.float32))
        assert np.isnan(K.values(u, s, b)).all() and s[0, 0] == 0
    # the nearest of 16 levels: off by at most half a step, and the top by the step's rounding
    rng = np.random.default_rng(0)
    x = K.bf16(rng.standard_normal((500, 64)).astype(np.float32) * 3)
    u, s, b = K.quantise(x)
    assert (np.abs(K.values(u, s, b) - x) <= s * (0.5 + 15 * 2.0 ** -8)).all()
    blocks = K.pack_blocks(*(np.zeros((2, 16, 64), np.uint8), np.ones((2, 16, 1), np.float32), -np.ones((2, 16, 1), np.float32)) * 2)
    assert blocks.shape == (2, 16 * 72) and blocks[0, 1024:1028].tolist() == [0x80, 0x3F, 0x80, 0xBF]


def test_oracle_pages():
    table = np.array([[3, 5, -1], [2, 7, -1]], np.int32)
    # both children of row 0 write inside page 5: the first keeps it, the second gets a copy in the lowest free page
    t, n, refs, info, copies = K.fork(table, [20, 30], [0, 0, 5], 1, 16, 8)
    assert t.tolist() == [[3, 5, -1], [3, 0, -1], [-1] * 3] and n.tolist() == [21, 21, 0] and copies == [(5, 0)]
    assert refs.tolist() == [1, 0, 0, 2, 0, 1, 0, 0] and info == [3, 0, 1, 0]
    # a page boundary: shared pages stay shared, each row gets a fresh page
    t, n, refs, info, copies = K.fork(table, [32, 30], [0, 0], 1, 16, 8)
    assert t.tolist() == [[3, 5, 0], [3, 5, 1]] and not copies and refs[5] == 2
    # one row only reads the page: the writer copies
    t, _, _, info, copies = K.fork(table, [20, 30], [0, 0], [0, 1], 16, 8)
    assert t.tolist() == [[3, 5, -1], [3, 0, -1]] and copies == [(5, 0)]
    # held pages are neither dealt nor written
    t, _, _, info, copies = K.fork(table, [20, 30], [0], 1, 16, 8, held=[1, 0, 0, 0, 0, 1, 0, 0])
    assert t.tolist() == [[3, 1, -1]] and copies == [(5, 1)] and info[0] == 4
    # pages run out
    t, _, _, info, _ = K.fork(table[:, :2], [32, 32], [0, 1, 0], [0, 0, -17], 16, 8)
    assert t.tolist() == [[3, 5], [2, 7], [3, -1]] and info[1] == 0
    t, _, _, info, copies = K.fork(np.array([[0, 1]], np.int32), [17], [0, 0], 1, 16, 2)
    assert t.tolist() == [[0, 1], [0, -1]] and info[1] == 1 and not copies
    t, refs, info, moves = K.compact(table, [20, 30], 16, 8)
    assert moves == [(5, 0), (7, 1)] and t.tolist() == [[3, 0, -1], [2, 1, -1]] and info == [4, 0, 2, 0]
    t, refs, info, moves = K.compact(table, [20, 30], 16, 8, held=[0, 0, 0, 0, 0, 0, 0, 1])
    assert moves == [(5, 0)] and t.tolist() == [[3, 0, -1], [2, 7, -1]]


def test_oracle_beams():
    x = np.log(np.array([[[0.5, 0.25, 0.25], [0.25, 0.5, 0.25]]]))
    s, r, t = K.beam_select(x, np.zeros((1, 2)), 3)
    assert r.tolist() == [[0, 1, 0]] and t.tolist() == [[0, 1, 1]] and np.allclose(np.exp(s), [[0.5, 0.5, 0.25]])
    s, r, t = K.beam_select(x, np.array([[0.0, -np.inf]]), 4)
    assert r.tolist() == [[0, 0, 0, -1]] and t.tolist() == [[0, 1, 2, -1]]
    s, r, t = K.beam_select(x, np.array([[0.0, -0.1]]), 2, finished=np.array([[0, 1]]), eos=2)
    assert r.tolist() == [[1, 0]] and t.tolist() == [[2, 0]] and np.isclose(s[0, 0], -0.1)

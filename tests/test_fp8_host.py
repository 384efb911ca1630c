"""Argument checks of the 8-bit operators: the C ABI's, without a GPU (a rejected call launches nothing, and zero rows
reach no CUDA call), and the binding's."""

import ctypes

import pytest
import torch

from megatron_tensor_layers_gb300 import _lib as tp
from megatron_tensor_layers_gb300.build import build

FP8 = torch.float8_e4m3fn
OK, INVALID, DIVIDE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def lib():
    build()
    return tp.load()


def arr(*p):
    return (ctypes.c_void_p * 8)(*p)


A = 0x10000          # 16-byte aligned addresses that nothing reads
B = 0x20000


def quantize(lib, t=1, n=0, k=128, dtype=0, x=A, ldx=128, c=B, ldc=128, s=A, lds=0, lists=True):
    return lib.tp_fp8_quantize(t, n, k, dtype, arr(x, x) if lists else None, ldx, arr(c, c), ldc, arr(s, s), lds, None)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(t=0), INVALID), (dict(t=9), INVALID), (dict(n=-1), INVALID), (dict(k=0), INVALID), (dict(lists=False), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(k=120), ALIGN), (dict(ldx=112), ALIGN), (dict(ldx=132), ALIGN), (dict(ldc=136), ALIGN),
    (dict(n=5, lds=4), INVALID), (dict(n=5, lds=5, x=None), INVALID), (dict(n=5, lds=5, x=A + 8), ALIGN),
    (dict(n=5, lds=5, c=B + 8), ALIGN), (dict(n=5, lds=5, s=A + 2), ALIGN), (dict(n=2 ** 31, lds=2 ** 31), INVALID),
])
def test_quantize(lib, kw, code):
    assert quantize(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(out=0), INVALID), (dict(k=24), ALIGN), (dict(gated=2), INVALID), (dict(out=7, gated=1), DIVIDE), (dict(dtype=5), UNSUPPORTED),
    (dict(ldw=64), ALIGN), (dict(w=None), INVALID), (dict(w=A + 4), ALIGN), (dict(s=A + 1), ALIGN),
])
def test_quantize_weight(lib, kw, code):
    a = dict(out=8, k=128, dtype=0, w=A, ldw=128, gated=0, c=B, ldc=128, s=A) | kw
    assert lib.tp_fp8_quantize_weight(1, a["out"], a["k"], a["dtype"], arr(a["w"]), a["ldw"], a["gated"], arr(a["c"]), a["ldc"],
                                      arr(a["s"]), None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(t=0), INVALID), (dict(h=24), ALIGN), (dict(h=32784, ldc=32784), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(mode=2), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(weight=None), INVALID), (dict(weight=A + 2), ALIGN), (dict(ldc=64), ALIGN), (dict(n=3, lds=2), INVALID),
    (dict(n=3, lds=3, codes=None), INVALID), (dict(n=3, lds=3, p=None), INVALID), (dict(n=3, lds=3, res=A + 8), ALIGN),
])
def test_norm(lib, kw, code):
    a = dict(t=1, n=0, h=128, dtype=0, p=A, res=None, weight=A, eps=1e-6, mode=0, out=None, codes=B, ldc=128, s=A, lds=0) | kw
    assert lib.tp_fp8_rmsnorm(a["t"], a["n"], a["h"], a["dtype"], arr(a["p"]), a["res"], a["weight"], a["eps"], a["mode"],
                              a["out"], a["codes"], a["ldc"], a["s"], a["lds"], None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(t=2, out=33), DIVIDE), (dict(k=136, ldx=144, ldw=144), ALIGN), (dict(ldx=120), ALIGN), (dict(ldw=136), ALIGN),
    (dict(kind=3), UNSUPPORTED), (dict(kind=2), UNSUPPORTED), (dict(kind=2, act=1, gather=1), UNSUPPORTED), (dict(act=3), INVALID),
    (dict(act=1, bias=A), UNSUPPORTED), (dict(kind=2, act=1, ys=None), INVALID), (dict(kind=2, act=1, out=24, ldy=32), ALIGN),
    (dict(kind=2, act=1, ldy=40), ALIGN), (dict(n=3, ldxs=2), INVALID), (dict(n=3, ldxs=3, kind=2, act=1, ldys=2), INVALID),
    (dict(ldy=16), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(w=A + 8), ALIGN), (dict(ws=A + 2), ALIGN),
    (dict(n=3, ldxs=3, x=None), INVALID), (dict(n=3, ldxs=3, xs=None), INVALID), (dict(n=3, ldxs=3, y=None), INVALID),
    (dict(n=3, ldxs=3, y=A + 8), ALIGN), (dict(gather=2), INVALID), (dict(n=2 ** 31, ldxs=2 ** 31), INVALID),
])
def test_col(lib, kw, code):
    a = dict(t=1, n=0, k=128, out=32, x=A, ldx=128, xs=A, ldxs=0, w=A, ldw=128, ws=A, bias=None, act=0, gather=0, y=B, ldy=32,
             kind=0, ys=A, ldys=0) | kw
    assert lib.tp_fp8_linear_col(a["t"], a["n"], a["k"], a["out"], a["x"], a["ldx"], a["xs"], a["ldxs"], arr(a["w"], a["w"]),
                                 a["ldw"], arr(a["ws"], a["ws"]), arr(a["bias"]) if a["bias"] else None, a["act"], a["gather"],
                                 arr(a["y"], a["y"]), a["ldy"], a["kind"], arr(a["ys"], a["ys"]) if a["ys"] else None, a["ldys"],
                                 None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(t=3), DIVIDE), (dict(k=40), ALIGN), (dict(mode=3), INVALID), (dict(mode=2, reduce=0), INVALID), (dict(ldp=16), INVALID),
    (dict(mode=2, parts=None), OK), (dict(parts=None), INVALID), (dict(ldp=40), UNSUPPORTED), (dict(pdt=2), UNSUPPORTED),
    (dict(ydt=2), UNSUPPORTED), (dict(ldy=40), UNSUPPORTED), (dict(mode=2, ldy=40), OK), (dict(n=2, ldxs=1), INVALID),
    (dict(n=2, ldxs=2, xs=None), INVALID), (dict(w=None), INVALID), (dict(ldw=72), ALIGN), (dict(n=2, ldxs=2, y=None), INVALID),
])
def test_row(lib, kw, code):
    a = dict(t=2, n=0, k=256, out=32, x=A, ldx=128, xs=A, ldxs=0, w=A, ldw=128, ws=A, reduce=1, mode=0, pdt=0, parts=A, ldp=32, y=B,
             ldy=32, ydt=0) | kw
    two = lambda p: arr(p, p, p)  # noqa: E731
    assert lib.tp_fp8_linear_row(a["t"], a["n"], a["k"], a["out"], two(a["x"]), a["ldx"], two(a["xs"]), a["ldxs"], two(a["w"]),
                                 a["ldw"], two(a["ws"]), None, a["reduce"], a["mode"], a["pdt"],
                                 two(a["parts"]) if a["parts"] else None, a["ldp"], a["y"], a["ldy"], a["ydt"], None) == code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(t=3), DIVIDE), (dict(f=48), ALIGN), (dict(h=40), ALIGN), (dict(act=0), INVALID), (dict(mode=3), INVALID),
    (dict(ldd=24), ALIGN), (dict(n=4, ldxs=4, bytes=100), WORKSPACE), (dict(n=4, ldxs=4, ws=None), WORKSPACE),
    (dict(n=4, ldxs=3), INVALID), (dict(n=4, ldxs=4, ws=A + 128), ALIGN), (dict(ydt=2), UNSUPPORTED), (dict(sd=None), INVALID),
])
def test_mlp(lib, kw, code):
    a = dict(t=2, n=0, h=128, f=64, x=A, xs=A, ldxs=0, w=A, sg=A, ldd=32, sd=A, act=1, mode=0, ws=A, bytes=1 << 20, y=B, ydt=0) | kw
    two = lambda p: arr(p, p)  # noqa: E731
    assert lib.tp_fp8_mlp_forward(a["t"], a["n"], a["h"], a["f"], a["x"], 128 if a["h"] == 128 else 48, a["xs"], a["ldxs"],
                                  two(a["w"]), two(a["sg"]), two(a["w"]), a["ldd"], two(a["sd"]), None, a["act"], a["mode"], 0,
                                  a["ws"], a["bytes"], a["y"], a["ydt"], None) == code


def test_mlp_workspace(lib):
    size = tp.tp_fp8_mlp_workspace_size
    assert size(2, 5, 256, 512, "fused") == 2560 + 2 * 256          # codes 5 x 512; 2 groups x 5 scales a rank
    assert size(2, 5, 256, 512, "direct") == 2560 + 2 * 256 + 2 * 2560
    assert size(2, 5, 256, 512, "ring", torch.float32) == 2560 + 2 * 256 + 2 * 5120
    assert size(3, 5, 256, 512) == 0 and size(2, -1, 256, 512) == 0 and size(0, 5, 256, 512) == 0


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(FP8)


def test_binding_refuses():
    """What the binding says before it asks for a GPU."""
    x, xs, w, ws = codes(4, 256), torch.zeros(2, 4), codes(64, 256), torch.zeros(1, 2)
    with pytest.raises(ValueError, match="x_scales"):
        tp.tp_fp8_linear_col(x, torch.zeros(4, 2), [w], [ws])
    with pytest.raises(ValueError, match="w_scales"):
        tp.tp_fp8_linear_col(x, xs, [w], [torch.zeros(2, 2)])
    with pytest.raises(ValueError, match="w_scales"):
        tp.tp_fp8_linear_col(x, xs, [w], [ws, ws])
    with pytest.raises(TypeError, match="dtype"):
        tp.tp_fp8_linear_col(x.float(), xs, [w], [ws])
    with pytest.raises(ValueError, match="gated"):
        tp.tp_fp8_linear_col(x, xs, [w], [ws], y_dtype=FP8)
    with pytest.raises(ValueError, match="y_scales"):
        tp.tp_fp8_linear_col(x, xs, [w], [ws], y_scales=[torch.zeros(1, 4)])
    with pytest.raises(TypeError, match="y has dtype"):
        tp.tp_fp8_linear_col(x, xs, [w], [ws], y_dtype=torch.float16)
    with pytest.raises(ValueError, match="act"):
        tp.tp_fp8_linear_col(x, xs, [w], [ws], act="relu")
    with pytest.raises(ValueError, match="same number"):
        tp.tp_fp8_linear_row([x], [xs, xs], [w], [ws])
    with pytest.raises(ValueError, match="mode"):
        tp.tp_fp8_linear_row([x], [xs], [w], [ws], mode="tree")
    with pytest.raises(ValueError, match="even"):
        tp.tp_fp8_quantize_weight([torch.zeros(3, 32)], gated=True)
    with pytest.raises(ValueError, match="row-major"):
        tp.tp_fp8_quantize([torch.zeros(32, 8).t()])
    with pytest.raises(ValueError, match="mode"):
        tp.tp_fp8_rmsnorm([torch.zeros(2, 32)], torch.ones(32, dtype=torch.bfloat16), mode="fused")
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_fp8_quantize([torch.zeros(2, 32)])
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_fp8_linear_col(x, xs, [w], [ws])

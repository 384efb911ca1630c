"""The gate of 8-bit products to the last bits, on sums that are exact.

Column 0 of x is 1 and its scale s_i has 12 significant bits, every other column 0; gate and up have one code in column 0, with
weight scales of 1.  A sum is then code * s_i: at most 4 + 12 bits, exact in fp32 with the products' one rounding gone, so
what is left of the error is the gate's:

    2^t with t = -log2(e) z: the argument's own rounding is carried, the hardware's 2^x is within 2 ulp (2^-22)
    1 + 2^t: half an ulp (2^-24), its reciprocal: 1 ulp (2^-23), the carried rounding's product: half an ulp
    times the gate, times up: half an ulp each

10 * 2^-24 of the value in all, to first order; terms of second order (the argument's rounding squared, below 2^-35, and
constants and squares kept to 2^-46) are within the half ulp that is added.  Below 2^-126 a reciprocal is a subnormal number, off by 2^-149 times
gate and up; past the largest float 2^t is an infinity and the gate 0.
"""

import pytest
import torch

import fp8_plain as P
from megatron_tensor_layers_gb300 import _lib as tp
from test_gpu_fp8 import DEV, FP8, gen, same_codes

pytestmark = pytest.mark.gpu

K = 16


def operands(n, os, gates, seed):
    """(x, xs, w, ws, gate, up): gates [os] of e4m3 values, up 1."""
    s = (1.0 + torch.randint(0, 2048, (n,), generator=gen(seed)).float() / 2048) * 0.5
    x = torch.zeros((n, K))
    x[:, 0] = 1.0
    w = torch.zeros((2 * os, K))
    w[:os, 0] = gates
    w[os:, 0] = 1.0
    blocks = 2 * P.groups(os)
    return x.to(FP8), s[None].contiguous(), w.to(FP8), torch.ones((blocks, 1)), s[:, None].double() * gates.double(), s[:, None].double()


def exact(g, act):
    """act(g) in float64 as g / (1 + exp(-z)), which loses nothing where act is small."""
    z = g if act == "silu" else 2.0 * 0.7978845608028654 * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(z)


def e4m3_between(lo, hi):
    v = torch.arange(256, dtype=torch.uint8).view(FP8).float()
    return v[(v >= lo) & (v <= hi)].unique()


# tile, parts: each kernel's own end of a tile, and the one that joins parts cannot be had with one K block
@pytest.mark.parametrize("tile", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("act,lo,hi", [("silu", -60, 20), ("silu", -120, 120), ("silu", -448, 448), ("gelu_tanh", -9, 9),
                                       ("gelu_tanh", -448, 448)])
def test_gate(tile, act, lo, hi):
    gates = e4m3_between(lo, hi)
    gates = torch.cat([gates, torch.zeros(-len(gates) % 16)])
    n, os = 512, len(gates)
    x, xs, w, ws, g, up = operands(n, os, gates, 1)
    a = (x.to(DEV), xs.to(DEV), [w.to(DEV)], [ws.to(DEV)])
    tp.tp_set_fp8_gemm(tile)
    try:
        (y,) = tp.tp_fp8_linear_col(*a, act=act, y_dtype=torch.float32)
        (codes,), (scales,) = tp.tp_fp8_linear_col(*a, act=act, y_dtype=FP8)
    finally:
        tp.tp_set_fp8_gemm()
    v = exact(g, act) * up
    # 2^t past the largest float: the gate is 0, which is off by the value itself, below 2^-126 of gate times up
    err = (y.cpu().double() - v).abs() - (g * up).abs() * 2.0 ** -126
    bound = 10.5 * 2.0 ** -24 * v.abs()
    assert (err <= bound).all(), ((err / v.abs().clamp(min=1e-300)).max().item() * 2 ** 24, "units of 2^-24")
    rc, rs = P.quantise_rows(y.cpu())                        # the same fp32 values: the same codes
    assert torch.equal(scales.cpu(), rs) and same_codes(codes, rc)


@pytest.mark.parametrize("tile", [16, 256])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gate_of_extremes(tile, act):
    """Sums over fp32's whole range, infinities and NaN: what g / (1 + exp(-z)) gives."""
    vals = [0.0, 1e-38, 1e-45, 3e-39, 1e10, 1e19, 2e19, 1e30, 1.15e38, 1.6e38, 3.4e38, float("nan")]
    n = len(vals)
    x = torch.zeros((n, 256))
    x[:, 0] = 1.0
    x[:, 128] = 1.0
    w = torch.zeros((32, 256))
    w[0:16:2, 0], w[1:16:2, 0] = 1.0, -1.0                   # gates of either sign
    w[16:, 128] = 1.0                                        # up is a column of its own group: 1 whatever the row's scale is
    xs = torch.stack([torch.tensor(vals), torch.ones(n)])
    ws = torch.tensor([[2.0, 1.0], [1.0, 1.0]])              # gate's scale doubles a row's, the last one's to an infinity
    a = (x.to(FP8).to(DEV), xs.to(DEV), [w.to(FP8).to(DEV)], [ws.to(DEV)])
    tp.tp_set_fp8_gemm(tile)
    try:
        y = tp.tp_fp8_linear_col(*a, act=act, y_dtype=torch.float32)[0].cpu()
    finally:
        tp.tp_set_fp8_gemm()
    for i, g in enumerate((2.0 * xs[0]).tolist()):
        for j, sign in ((0, 1.0), (1, -1.0)):
            got = y[i, j].double()
            if abs(g) < 1e-37:
                assert abs(got - 0.5 * sign * g) <= 2.0 ** -148, (g, sign, got)    # act(g) = g / 2 there
            elif g != g or (g == float("inf") and sign < 0):
                assert got.isnan(), (g, sign, got)
            else:
                assert got == (g if sign > 0 else 0.0), (g, sign, got)

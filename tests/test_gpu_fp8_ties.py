"""Codes of values next to the ties between codes, where a quotient's last bit decides, at scales over the whole range."""

import pytest
import torch

import fp8_plain as P
from megatron_tensor_layers_gb300 import _lib as tp
from test_gpu_fp8 import DEV, FP8, check, gen, same_codes, same_scales, weights

pytestmark = pytest.mark.gpu


def ulps(x, d):
    """fp32 x moved by d units of its last place, away from zero."""
    return (x.view(torch.int32) + d).view(torch.float32)


def near_ties(n, e, seed):
    """Rows of one group: the largest value first, then values within 2 ulp of scale times a tie of any binade of codes."""
    g = gen(seed)
    top = (1.0 + torch.rand((n, 1), generator=g)) * 2.0 ** e
    top[0] = 2.0 ** e
    top[1] = ulps(torch.full((1,), 2.0 ** (e + 1)), -1)
    s = P._scale(top)
    tie = torch.randint(16, 32, (n, 127), generator=g).float() * torch.exp2(torch.randint(-12, 4, (n, 127), generator=g).float())
    x = ulps((s * tie.clamp(max=447.0)), torch.randint(-2, 3, (n, 127), generator=g).int())
    x = torch.minimum(x, top)
    sign = torch.where(torch.rand((n, 127), generator=g) < 0.5, -1.0, 1.0)
    return torch.cat([top, x * sign], 1)


@pytest.mark.parametrize("e", [-99, -61, -52, -51, 0, 60, 126])
def test_rows_next_to_ties(e):
    x = torch.cat([near_ties(4096, e, 7), near_ties(4096, min(e + 9, 126), 8)], 1)   # groups either side of a threshold
    codes, scales = tp.tp_fp8_quantize([x.to(DEV)])
    rc, rs = P.quantise_rows(x)
    assert same_scales(scales[0], rs) and same_codes(codes[0], rc)


@pytest.mark.parametrize("e", [-99, -52, 0, 126])
def test_weights_next_to_ties(e):
    w = near_ties(128 * 128, e, 9).reshape(128, 128 * 128)       # 128 blocks
    w.reshape(128, 128, 128)[:, :, 0] = 0                        # their own largest values
    w[0, ::128] = near_ties(128, e, 10)[:, 0]
    codes, scales = tp.tp_fp8_quantize_weight([w.to(DEV)])
    rc, rs = P.quantise_weight(w)
    assert same_scales(scales[0], rs) and same_codes(codes[0], rc)


@pytest.mark.parametrize("n", [5, 40, 300])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_codes_of_mixed_sizes(n, act):
    """Every third row is 2^-35 of its size and its outputs 2^-70, so rows with scales below 2^-60 stand among ordinary ones."""
    k, out = 256, 144
    x, xs = P.quantise_rows(torch.randn((n, k), generator=gen(11)))
    xs[:, ::3] *= 2.0 ** -35
    w, ws = weights(2 * out, k, 12, True)
    a = (x.to(DEV), xs.to(DEV), [w.to(DEV)], [ws.to(DEV)])
    (codes,), (scales,) = tp.tp_fp8_linear_col(*a, act=act, y_dtype=FP8)
    (y,) = tp.tp_fp8_linear_col(*a, act=act, y_dtype=torch.float32)
    assert n < 4 or float(scales[:, ::3].max()) < 2.0 ** -60 < float(scales[:, 1::3].min())
    rc, rs = P.quantise_rows(y.cpu())
    assert torch.equal(scales.cpu(), rs) and same_codes(codes, rc)
    check(y, *P.gated(P.rows64(x, xs), *P.halves64(w, ws), act))

"""Attention over cached values of any size, for chunks that fill the device and
for single rows, against the float64 oracle of the other attention tests.

The bounds are those of test_gpu_kv4_chunks.py and test_gpu_kv4.py: every term is
relative to the values, so a factor on all of them changes nothing."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from test_gpu_kv4 import Cache, DEV, cu_of
from test_gpu_kv4_chunks import check, run

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

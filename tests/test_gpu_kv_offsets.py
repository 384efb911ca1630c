"""Row offsets and lengths that a call cannot use: reported, and nothing else touched."""

import pytest
import torch

from test_gpu_kv4 import Cache, DEV

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


def cache():
    c = Cache(1, 1, 128, 64, [150, 100], 81)
    q = [torch.randn((2, 512), device=DEV).to(torch.bfloat16)]
    k = [torch.ones((2, 128), dtype=torch.bfloat16, device=DEV)]
    return c, q, k


@pytest.mark.parametrize("cu,stored", [([0, 3, 2], 0), ([1, 1, 1], 0), ([0, 0, 0], 0), ([0, 0, 1], 1), ([1, 1, 2], 1),
                                       ([-1, 1, 2], 1), ([0, 1, 5], 1), ([-2 ** 31, 2 ** 31 - 1, 2], 0)])
def test_bad_offsets_are_reported(cu, stored):
    """Out of order, out of range, and offsets that leave rows without a sequence; `stored` of the two rows have one."""
    c, q, k = cache()
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    before = c.pools[0].clone()
    out = [torch.full((2, 512), 7.0, dtype=torch.bfloat16, device=DEV)]
    tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu, out=out)
    assert tp.tp_device_status() == 1 and torch.equal(before, c.pools[0])
    assert int((out[0] == 7.0).all(1).sum()) >= 2 - stored
    tp.tp_kv4_append(k, k, c.pools, c.dtable, c.dlens, cu_rows=cu)
    assert tp.tp_device_status() == 1
    # a row's key and value are 2 * 64 bytes of codes and 2 * 4 of pairs
    changed = (before != c.pools[0]).sum().item()
    assert changed <= 136 * stored and (changed > 0) == (stored > 0)
    k2, _ = tp.tp_kv4_load(c.pools, c.dtable, c.dlens, 2, cu_rows=cu)
    assert tp.tp_device_status() == 1 and int(k2[0].any(1).sum()) == stored


def test_the_least_length():
    """Lengths below 0 are lengths of 0, down to the least int32: the row is at a negative position and is not stored."""
    c, _, k = cache()
    before = c.pools[0].clone()
    c.dlens.copy_(torch.tensor([-2 ** 31, -1], dtype=torch.int32))
    tp.tp_kv4_append(k, k, c.pools, c.dtable, c.dlens)
    assert tp.tp_device_status() == 0 and torch.equal(before, c.pools[0])
    k2, v2 = tp.tp_kv4_load(c.pools, c.dtable, c.dlens, 2)
    assert tp.tp_device_status() == 0 and not k2[0].any() and not v2[0].any()

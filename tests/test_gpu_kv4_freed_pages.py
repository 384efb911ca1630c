"""Pages that no row sees may be gone: behind a window, and between the sinks and
the window.  Bounds as in the other attention tests."""

import pytest
import torch

from test_gpu_kv4 import Cache, cu_of
from test_gpu_kv4_chunks import check, rows_of

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [[100, 60], [3, 1]])
@pytest.mark.parametrize("hd,window,sinks", [(128, 200, 5), (64, 200, 0), (128, 17, 140), (128, 1, 16)])
def test_pages_behind_the_window_are_not_asked_for(hd, window, sinks, rows):
    """The same outputs as with every page in the table, and nothing reported."""
    c = Cache(1, 8, hd, 16, [1000, 333], 71)
    q = rows_of(c, rows, 64, 72)
    call = lambda: tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, cu_rows=cu_of(rows), window=window, sinks=sinks)  # noqa: E731
    whole = call()
    assert tp.tp_device_status() == 0
    check(c, q, whole, rows, 64, window=window, sinks=sinks)
    gone = 0
    for s, m in enumerate(rows):
        first = c.lens[s] - m
        for i in range(first // 16):
            if 16 * i + 15 <= first - window and 16 * i >= sinks:
                c.dtable[s, i] = -1
                gone += 1
    assert gone > 10
    got = call()
    assert tp.tp_device_status() == 0
    assert torch.equal(whole[0], got[0])

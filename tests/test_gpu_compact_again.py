"""A compaction that has been made leaves nothing for the next one, with held pages too."""

import numpy as np
import pytest
import torch

from test_gpu_kv_pages import dev, make_pools, tables

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages_of_row", [2, 40])
@pytest.mark.parametrize("seed", range(4))
def test_nothing_moves_the_second_time(seed, pages_of_row):
    """As many pages in use lie at or above their count as holes below it, held ones counted among the former."""
    rng = np.random.default_rng(200 + seed)
    rows, cols, ps = 20, 8, 16
    pages = rows * cols * pages_of_row
    table, lens = tables(rng, rows, cols, ps, pages, 0.4)
    held = dev(rng.random(pages) < 0.2, torch.uint8)
    pools = make_pools(1, 1, pages, 1, ps, 64, seed)
    first = tp.tp_kv_compact(dev(table), dev(lens), pools, held=held)
    assert first[2][2].item() > 0
    before = pools[0].clone()
    again = tp.tp_kv_compact(first[0], dev(lens), pools, held=held)
    assert again[2].tolist() == [first[2][0].item(), 0, 0, 0]
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1]) and torch.equal(pools[0], before)
    assert tp.tp_device_status() == 0

"""The flags by which attention's thread blocks hand over parts of a row's context,
run on the host in every order of their steps."""

import pytest

from megatron_tensor_layers_gb300 import _lib as tp
from megatron_tensor_layers_gb300.build import build

TOP = 1 << 63


@pytest.fixture(scope="module")
def lib():
    build()
    return tp.load()


@pytest.mark.parametrize("word", [0, 12345, TOP | 6, 2 ** 64 - 1])
def test_no_flag_outlives_a_join_that_gave_up(lib, word):
    """A graph's replay has its call's number again: a flag that stayed up would be taken for the replay's own."""
    tag = TOP | 7
    assert lib.tp_debug_part_flag(word, tag, 0) == tag       # left and awaited: up until the join takes it down
    for order in (1, 2, 3, 4):
        assert lib.tp_debug_part_flag(word, tag, order) == 0


@pytest.mark.parametrize("groups", [1, 4, 8])
def test_a_part_waits_for_its_own_and_lower_blocks(lib, groups):
    """Neighbouring parts lie in the same block or in one above, so a grid of which only the first blocks run gets on."""
    for blocks in (1, 7, 152):
        for workers in sorted({0, 1, blocks - 1, blocks, blocks * groups // 2 + 1, blocks * groups - 1, blocks * groups}):
            if not 0 <= workers <= blocks * groups:
                continue
            first = [lib.tp_debug_first_worker(b, blocks, groups, workers) for b in range(blocks + 1)]
            assert first[0] == 0 and first[-1] == workers
            assert all(0 <= b - a <= groups for a, b in zip(first, first[1:]))
    assert lib.tp_debug_first_worker(0, 152, groups, 152 * groups + 1) == -1

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

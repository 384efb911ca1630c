"""Which kernel an 8-bit product takes (host logic, no GPU), and the refusals of tp_set_fp8_gemm."""

import pytest

from megatron_tensor_layers_gb300 import _lib as tp
from megatron_tensor_layers_gb300.build import build

UNSUPPORTED = "UNSUPPORTED"


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return tp.load()


def residents(sms=152):
    """Clusters at once: two CTAs an SM for tiles of 16 and 32 tokens (and 64, plain), one for the others and for pairs."""
    few = [[sms * per // p for p in range(1, 9)] for per in (2, 2, 2, 1)]
    return few + [[sms // (2 * p) for p in range(1, 9)]]


def test_choices():
    r = residents()
    assert tp.tp_debug_fp8_plan(1, 1280, 8192, r, groups=8)[0] == 16
    assert tp.tp_debug_fp8_plan(17, 1280, 8192, r, groups=8)[0] == 32
    assert tp.tp_debug_fp8_plan(64, 1280, 8192, r, groups=8)[0] == 64
    assert tp.tp_debug_fp8_plan(4096, 7168, 8192, r, groups=4, gated=True) == (256, 1)
    assert tp.tp_debug_fp8_plan(4096, 8192, 7168, r, segs=4) == (256, 1)
    tile, parts = tp.tp_debug_fp8_plan(4, 256, 8192, r)          # two tiles of 64 blocks: shared by clusters
    assert tile == 16 and parts > 1
    assert tp.tp_debug_fp8_plan(4, 256, 128, r) == (16, 1)       # one block: nothing to share


@pytest.mark.parametrize("bad", [dict(m=0), dict(n=0), dict(k=0), dict(groups=9), dict(segs=0), dict(groups=2, segs=2), dict(sms=0),
                                 dict(m=2 ** 29 + 1)])
def test_plan_refuses(bad):
    a = dict(m=8, n=128, k=128) | bad
    with pytest.raises(tp.TPError, match="INVALID_ARG"):
        tp.tp_debug_fp8_plan(a.pop("m"), a.pop("n"), a.pop("k"), residents(), **a)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("left", [2, 3, 4])
def test_one_kernel_that_can_run_is_enough(left, gated):
    """More than 64 tokens: tiles of 64 or 128 tokens or CTA pairs, of which two cannot run."""
    r = [row if i == left else [0] * 8 for i, row in enumerate(residents())]
    for m, n, k in [(65, 128, 128), (500, 1280, 8192), (4096, 7168, 8192)]:
        tile, parts = tp.tp_debug_fp8_plan(m, n, k, r, gated=gated)
        assert tile == (64, 128, 256)[left - 2] and parts >= 1


def test_no_kernel_that_can_run():
    with pytest.raises(tp.TPError, match=UNSUPPORTED):
        tp.tp_debug_fp8_plan(8, 128, 128, [[0] * 8] * 5)


def test_choice_set_by_hand():
    try:
        for ok in [(16, 0, 0), (32, 8, 0), (64, 1, 0), (128, 7, 0), (256, 0, 3), (256, 4, 0), (0, 0, 0)]:
            tp.tp_set_fp8_gemm(*ok)
        for bad in [(8, 0, 0), (0, 1, 0), (16, 9, 0), (16, -1, 0), (256, 3, 0), (256, 8, 0), (0, 0, -1), (512, 0, 0)]:
            with pytest.raises(tp.TPError, match="INVALID_ARG"):
                tp.tp_set_fp8_gemm(*bad)
    finally:
        tp.tp_set_fp8_gemm()

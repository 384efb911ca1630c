"""A bias at an odd address, which no kernel could read, is refused on the host; one aligned to its elements is taken."""

import ctypes

import pytest

from megatron_tensor_layers_gb300 import _lib as tp
from megatron_tensor_layers_gb300.build import build

A = 0x10000          # an address that nothing reads: no row, no launch
OK, ALIGN = 0, 3


@pytest.fixture(scope="module")
def lib():
    build()
    return tp.load()


def one(p):
    return (ctypes.c_void_p * 1)(p)


CALLS = {
    "tp_linear_col": lambda f, b: f(1, 0, 128, 32, A, 128, one(A), 128, one(b), 0, 0, one(A), 32, 0, None),
    "tp_linear_row": lambda f, b: f(1, 0, 128, 32, one(A), 128, one(A), 128, b, 1, 2, 0, None, 32, A, 32, 0, None),
    "tp_mlp_forward": lambda f, b: f(1, 0, 128, 64, A, 128, one(A), one(A), 64, b, 1, 2, 0, None, 0, A, 0, None),
    "tp_mlp_forward_static": lambda f, b: f(1, 0, 128, 64, A, 128, one(A), one(A), 64, b, 1, 2, 0, A, 0, None),
    "tp_fp8_linear_col": lambda f, b: f(1, 0, 128, 32, A, 128, A, 0, one(A), 128, one(A), one(b), 0, 0, one(A), 32, 0, None, 0, None),
    "tp_fp8_linear_row": lambda f, b: f(1, 0, 128, 32, one(A), 128, one(A), 0, one(A), 128, one(A), b, 1, 2, 0, None, 32, A, 32, 0, None),
    "tp_fp8_mlp_forward": lambda f, b: f(1, 0, 128, 64, A, 128, A, 0, one(A), one(A), one(A), 64, one(A), b, 1, 2, 0, None, 0, A, 0, None),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_bias(lib, name):
    f = getattr(lib, name)
    assert CALLS[name](f, A) == OK and CALLS[name](f, A + 2) == OK
    assert CALLS[name](f, A + 1) == ALIGN

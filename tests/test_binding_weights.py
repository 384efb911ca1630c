"""Weights that are no matrices are called that, not blocks of an odd number of rows."""

import pytest
import torch

from megatron_tensor_layers_gb300 import _lib as tp


def f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(tp.FP8)


def b(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("call,name", [
    (lambda w: tp.tp_linear_col(b(4, 64), [w], act="silu"), "w"),
    (lambda w: tp.tp_mlp_forward(b(4, 64), [w], [b(64, 32)]), "w_gate_up"),
    (lambda w: tp.tp_fp8_linear_col(f8(4, 64), torch.zeros(1, 4), [w], [torch.zeros(2, 1)], act="silu"), "w"),
    (lambda w: tp.tp_fp8_mlp_forward(f8(4, 64), torch.zeros(1, 4), [w], [torch.zeros(2, 1)], [f8(64, 32)], [torch.zeros(1, 1)]), "w_gate_up"),
], ids=["linear_col", "mlp", "fp8_linear_col", "fp8_mlp"])
def test_a_weight_that_is_no_matrix(call, name):
    for w in (b(64), f8(2, 32, 64)):
        with pytest.raises(ValueError, match=rf"{name}\[0\] must be a row-major matrix"):
            call(w)
    with pytest.raises(TypeError, match=rf"{name}\[0\] must be a torch.Tensor"):
        call([[1.0]])

"""A CUDA error of one call is that call's: the next one, which runs, does not report it."""

import ctypes

import pytest
import torch

from megatron_tensor_layers_gb300 import _lib as tp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def failed_call():
    """A call that CUDA refuses on the host: a stream that is being captured is synchronised, which ends its capture."""
    cu = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(handle, 2) == 0        # relaxed: other streams are as they were
    code = tp.tp_device_status(s)
    cu.cuStreamEndCapture(handle, ctypes.byref(graph))       # reports the ended capture; there is no graph
    assert tp.STATUS_NAMES[code] == "TP_ERR_CUDA"


def entries():
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
    one = lambda *s: torch.ones(s, device=DEV)  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return {
        "quantize": lambda: tp.tp_fp8_quantize([b(4, 128)]),
        "quantize_weight": lambda: tp.tp_fp8_quantize_weight([b(4, 128)]),
        "rmsnorm": lambda: tp.tp_fp8_rmsnorm([b(4, 128)], b(128)),
        "few": lambda: tp.tp_fp8_linear_col(f8(4, 128), one(1, 4), [f8(64, 128)], [one(1, 1)]),
        "pairs": lambda: tp.tp_fp8_linear_col(f8(4096, 1024), one(8, 4096), [f8(2048, 1024)], [one(16, 8)]),
        "linear_col": lambda: tp.tp_linear_col(b(4, 128), [b(64, 128)]),
        "linear_col_many": lambda: tp.tp_linear_col(b(4096, 1024), [b(2048, 1024)]),
        "linear_row_split": lambda: tp.tp_linear_row([b(4, 128)] * 2, [b(64, 128)] * 2, mode="fused"),
        "small_mlp": lambda: tp.tp_mlp_forward(b(4, 256), [b(256, 256)], [b(256, 128)], mode="fused"),
        "reduce": lambda: tp.tp_shard_reduce([b(4, 128)] * 2),
        "reduce_ring": lambda: tp.tp_shard_reduce([b(4, 128)] * 2, mode="ring"),
        "replicate": lambda: tp.tp_shard_reduce([b(4, 128)] * 2, replicate=True, alloc_out=False),
        "gather": lambda: tp.tp_shard_gather([b(4, 128)] * 2),
        "norm": lambda: tp.tp_reduce_scatter_rmsnorm([b(4, 128)], b(128)),
        "embed": lambda: tp.vocab_parallel_embed(torch.zeros(4, dtype=torch.int32, device=DEV), [b(16, 128)], 16),
    }


@pytest.mark.parametrize("name", ["quantize", "quantize_weight", "rmsnorm", "few", "pairs", "linear_col", "linear_col_many", "linear_row_split",
                                  "small_mlp", "reduce", "reduce_ring", "replicate", "gather", "norm", "embed"])
def test_an_earlier_error_is_not_reported_again(name):
    call = entries()[name]
    call()
    torch.cuda.synchronize()
    failed_call()
    call()                                                   # raises TPError where the error is still there
    torch.cuda.synchronize()
    assert tp.tp_device_status() == 0

"""Tensors of another device than the current one are refused: the library launches on the current device, whose kernels cannot
read them.  Runs on the CPU, with tensors that say that they are on a device."""

import pytest
import torch

from megatron_tensor_layers_gb300 import _lib as tp


class On1(torch.Tensor):
    def get_device(self):
        return 1


def on1(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=torch.uint8 if dtype is tp.FP8 else dtype).view(dtype).as_subclass(On1)


@pytest.fixture
def launches(monkeypatch):
    made = []
    monkeypatch.setattr(tp, "_launch", lambda name, *a: made.append(name))
    monkeypatch.setattr(tp, "_stream", lambda s: s)
    return made


def calls():
    f8, f32 = tp.FP8, torch.float32
    return {
        "quantize": lambda: tp.tp_fp8_quantize([on1(4, 128)], codes=[on1(4, 128, dtype=f8)], scales=[on1(1, 4, dtype=f32)]),
        "linear_row": lambda: tp.tp_fp8_linear_row([on1(4, 128, dtype=f8)], [on1(1, 4, dtype=f32)], [on1(64, 128, dtype=f8)],
                                                   [on1(1, 1, dtype=f32)], mode="fused", y=on1(4, 64)),
        "reduce": lambda: tp.tp_shard_reduce([on1(8), on1(8)], out=on1(8)),
        "norm": lambda: tp.tp_reduce_scatter_rmsnorm([on1(4, 128)], on1(128), out=on1(4, 128)),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_another_device_is_refused(launches, monkeypatch, name):
    monkeypatch.setattr(tp, "_current_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
        calls()[name]()
    assert not launches


@pytest.mark.parametrize("name", list(calls()))
def test_the_current_device_is_taken(launches, monkeypatch, name):
    monkeypatch.setattr(tp, "_current_device", lambda: 1, raising=False)
    calls()[name]()
    assert len(launches) == 1

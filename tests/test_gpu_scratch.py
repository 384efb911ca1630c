"""Workspaces that the caller does not give: on another stream than the current one, and under prepared calls."""

import numpy as np
import pytest
import torch

from test_gpu_kv4 import Cache, DEV, cu_of
from test_gpu_kv_pages import dev, make_pools

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


def calls():
    """(call(stream) -> tensors) of every operator with a workspace."""
    c = Cache(2, 2, 128, 64, [3000, 257, 33], 91)
    q = [torch.randn((3, 1024), device=DEV).to(torch.bfloat16) for _ in range(2)]
    qc = [torch.randn((190, 64 * 128), device=DEV).to(torch.bfloat16) for _ in range(2)]
    cu = cu_of([100, 80, 10])
    table, lens, parents = dev(np.arange(24).reshape(8, 3)), dev([40] * 8), dev([0, 0, 1, 2, 2, 3, 7, 7])
    pools = make_pools(1, 1, 40, 1, 16, 64, 5)
    x, scores = torch.randn((8, 20000), device=DEV), torch.zeros((2, 4), device=DEV)
    w = [torch.randn((64, 512), device=DEV).to(torch.bfloat16) for _ in range(2)]
    return [
        lambda **kw: tp.tp_kv4_attention(q, c.pools, c.dtable, c.dlens, **kw),
        lambda **kw: tp.tp_kv4_attention(qc, c.pools, c.dtable, c.dlens, cu_rows=cu, **kw),
        lambda **kw: tp.tp_kv_fork(table, lens, parents, pools, **kw),
        lambda **kw: tp.tp_beam_select([x], scores, 4, **kw),
        lambda **kw: [tp.tp_linear_row([a[:, :512] for a in q], w, **kw)],
    ]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("which", range(5))
def test_on_a_stream_and_on_its_handle(which):
    """While the call waits on its stream, the current stream allocates and writes as much as it likes."""
    call = calls()[which]
    plain = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(stream=stream)
        noise = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(64)]
        torch.cuda.synchronize()
        assert same(plain, got) and all((n == 255).all() for n in noise)
    assert tp.tp_device_status() == 0


@pytest.mark.parametrize("which", range(5))
def test_a_prepared_call_has_its_workspace_to_itself(which):
    """Nothing allocated after the preparation is written by the call, nor does writing it change the call's results."""
    call = calls()[which]
    plain = [t.clone() for t in call()]
    step = tp.prepare(lambda: call())
    noise = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(64)]
    for _ in range(2):
        got = step()
        for n in noise:
            assert (n == 255).all()
            n.fill_(255)
    torch.cuda.synchronize()
    assert same(plain, got if isinstance(got, (list, tuple)) else [got])
    assert tp.tp_device_status() == 0

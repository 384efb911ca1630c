"""The decode loop's forward pass against the same model written down plainly, in
float64, with the cache's 4-bit rounding of keys and values.

The library rounds to bfloat16 between its operators (about ten times a layer, by
2^-9 of the norm on average), and a key or value that comes out on the other side of
a border between two codes is off by one of 15 steps.  Together that is some
hundredths of the logits' norm over two layers.  A column, head, shard, residual or
position in the wrong place makes the difference as large as the logits.  The bound
is a quarter of their norm."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu
loop = pytest.importorskip("megatron_tensor_layers_gb300.decode_loop")
from megatron_tensor_layers_gb300 import synth  # noqa: E402


def f64(x):
    return x.double().cpu().numpy()


def norm(x, w):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * f64(w)


def held(x):
    """What the cache stands for after rows x [n, hd]."""
    return K.values(*K.quantise(K.bf16(x.astype(np.float32))))


def plain(model, ids):
    """Logits [n, vocab] of every row of one sequence."""
    c = model.cfg
    group, hd, n = c.heads // c.kv_heads, c.head_dim, len(ids)
    table = np.concatenate([f64(x) for x in model.table])
    x = table[ids]
    for w in model.layers:
        y = norm(x, w["norm1"])
        add = np.zeros_like(x)
        for r in range(c.t):
            heads, kv = c.heads // c.t, c.kv_heads // c.t
            q, k, v = np.split(y @ f64(w["qkv"][r]).T, [heads * hd, (heads + kv) * hd], axis=1)
            out = np.empty((n, heads * hd))
            for h in range(heads):
                at = slice(h // group * hd, (h // group + 1) * hd)
                out[:, h * hd:(h + 1) * hd] = K.attention(q[:, h * hd:(h + 1) * hd], held(k[:, at]), held(v[:, at]),
                                                          np.arange(n), hd ** -0.5, c.window, c.sinks)
            add += out @ f64(w["o"][r]).T
        x = x + add
        y = norm(x, w["norm2"])
        add = np.zeros_like(x)
        for r in range(c.t):
            gate, up = np.split(y @ f64(w["gate_up"][r]).T, 2, axis=1)
            add += (gate / (1 + np.exp(-gate)) * up) @ f64(w["down"][r]).T
        x = x + add
    return norm(x, model.norm) @ table.T


@pytest.mark.parametrize("t,kv_heads,window,sinks", [(2, 4, 0, 0), (1, 2, 0, 0), (4, 4, 20, 3)])
def test_forward_is_the_model(t, kv_heads, window, sinks):
    cfg = loop.Config(t=t, kv_heads=kv_heads, window=window, sinks=sinks)
    model = loop.Model(cfg)
    prompts = [synth.uniform_ids(n, cfg.vocab, 7 + n, device="cuda") for n in (1, 30, 47)]
    lens = torch.tensor([1, 30, 47], dtype=torch.int32, device="cuda")
    cache = loop.Cache(cfg, 40, 8)
    cache.start(lens)
    cu = torch.tensor([0, 1, 31, 78], dtype=torch.int32, device="cuda")
    got = [f64(torch.cat(loop.forward(model, cache, torch.cat(prompts), cu_rows=cu), 1))]
    # then a token each, the sequences in another order
    order = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    cache.fork(order, 1)
    more = torch.tensor([5, 900, 77], dtype=torch.int32, device="cuda")
    step = f64(torch.cat(loop.forward(model, cache, more), 1))
    at = 0
    for i, p in enumerate(prompts):
        n = p.numel()
        row = order.tolist().index(i)
        want = plain(model, p.tolist() + [more[row].item()])
        for have, ref in ((got[0][at:at + n], want[:n]), (step[row:row + 1], want[n:])):
            err = np.linalg.norm(have - ref, axis=1) / np.linalg.norm(ref, axis=1)
            assert err.max() < 0.25, (i, err)
        at += n

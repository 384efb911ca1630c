"""The operators together: a beam search over the paged 4-bit cache."""

import pytest
import torch

pytestmark = pytest.mark.gpu
loop = pytest.importorskip("megatron_tensor_layers_gb300.decode_loop")
from megatron_tensor_layers_gb300 import synth  # noqa: E402


def run(cfg, steps=9, beams=4, **kw):
    model = loop.Model(cfg)
    prompts = [synth.uniform_ids(n, cfg.vocab, 7 + n, device="cuda") for n in (1, 30, 47)]
    return loop.generate(model, prompts, beams=beams, steps=steps, **kw)


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_where_pages_lie_does_not_matter(window, sinks):
    """Moving the pages, a pool with hardly a page to spare (so that freed ones come back), and other page sizes give
    the same tokens and scores, bit for bit: nothing but the place of the cached rows differs."""
    want = run(loop.Config(window=window, sinks=sinks))
    assert want[0].shape == (3, 4, 9) and (want[1][:, :-1] >= want[1][:, 1:]).all()
    for i in range(3):
        assert len({tuple(b) for b in want[0][i].tolist()}) == 4
    # 47 tokens and nine more are four pages of 16; shared fronts, a copied tail and a fresh page for each beam
    for kw in (dict(compact_every=1), dict(compact_every=3), dict(pages=40), dict(pages=40, compact_every=2)):
        got = run(loop.Config(window=window, sinks=sinks), **kw)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    for ps in (32, 64, 128):
        got = run(loop.Config(window=window, sinks=sinks, page_size=ps), compact_every=2)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_sequence_does_not_see_the_others():
    """A prompt alone gives the tokens it gives among others (the products of a row do not depend on other rows)."""
    cfg = loop.Config()
    model = loop.Model(cfg)
    prompts = [synth.uniform_ids(n, cfg.vocab, 7 + n, device="cuda") for n in (30, 47)]
    cache = loop.Cache(cfg, 40, 8)
    ids = torch.cat(prompts)
    cache.start(torch.tensor([30, 47], dtype=torch.int32, device="cuda"))
    x = torch.cat(loop.forward(model, cache, ids, cu_rows=torch.tensor([0, 30, 77], dtype=torch.int32, device="cuda")), 1)
    for a, b, p in ((0, 30, prompts[0]), (30, 77, prompts[1])):
        one = loop.Cache(cfg, 40, 8)
        one.start(torch.tensor([b - a], dtype=torch.int32, device="cuda"))
        y = torch.cat(loop.forward(model, one, p, cu_rows=torch.tensor([0, b - a], dtype=torch.int32, device="cuda")), 1)
        assert torch.isfinite(y).all() and y.std() > 0.1
        # the last row's best tokens agree where they are not next to each other
        top = y[-1].topk(2).values
        if top[0] - top[1] > 0.1:
            assert x[b - 1].argmax() == y[-1].argmax()


def test_pages_run_out_without_harm():
    """A pool that is too small: the rows that found no page are reported, nothing outside is touched."""
    with pytest.raises(RuntimeError, match="out of range"):
        run(loop.Config(), pages=9)

"""Beam selection over rows whose edges cut 16-byte words, many of them for each
thread block: against the oracle, tokens exactly."""

import pytest
import torch

from test_gpu_kv_pages import DEV, check_beams

tp = pytest.importorskip("megatron_tensor_layers_gb300")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [37, 4095, 4097])
def test_many_cut_rows_of_a_block(vocab, dtype):
    """700 rows of odd width: every ring slot is used for cut words and then for whole ones, several times."""
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.randn((100, 7, vocab), device=DEV, generator=g).to(dtype)
    scores = -torch.rand((100, 7), device=DEV, generator=g)
    check_beams(x, scores, 5, shards=[x.reshape(700, vocab)])
    wide = torch.randn((700, vocab + 3), device=DEV, generator=g).to(dtype)
    x = wide[:, 1:vocab + 1]
    check_beams(x.reshape(100, 7, vocab), scores, 5, shards=[x])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", [0, 1, 3])
@pytest.mark.parametrize("items,vocab", [(32, 151936), (5, 20011)])
def test_equal_beams_tie(items, vocab, extra, dtype):
    """Beams of the same logits and score: by logit, then beam, then token, wherever the rows lie in memory and
    whichever thread blocks read them."""
    beams, k = 8, 16
    g = torch.Generator(device=DEV).manual_seed(vocab + extra)
    one = (torch.randn((items, 1, vocab), device=DEV, generator=g) * 3).to(dtype)
    wide = torch.empty((items * beams, vocab + extra), dtype=dtype, device=DEV)
    x = wide[:, extra:]
    x.copy_(one.expand(items, beams, vocab).reshape(items * beams, vocab))
    scores = -torch.rand((items, 1), device=DEV, generator=g).expand(items, beams).contiguous()
    top = one[:, 0].float().sort(dim=1, descending=True, stable=True)
    want = [sorted((-x, b, t) for b in range(beams) for x, t in zip(top.values[i, :k].tolist(), top.indices[i, :k].tolist()))[:k]
            for i in range(items)]
    want_rows = [[i * beams + b for _, b, _ in w] for i, w in enumerate(want)]
    want_tokens = [[t for _, _, t in w] for w in want]
    per = -(-vocab // 3)
    for shards in ([x], [x[:, :per], x[:, per:2 * per], x[:, 2 * per:]]):
        s, rows, tokens = tp.tp_beam_select(shards, scores, k)
        assert rows.tolist() == want_rows and tokens.tolist() == want_tokens
        for i, w in enumerate(want):                         # equal logits, equal bits
            assert all(s[i, n] == s[i, n + 1] for n in range(k - 1) if w[n][0] == w[n + 1][0])
        s1, rows, tokens = tp.tp_beam_select(shards, scores, 1)
        assert rows.tolist() == [w[:1] for w in want_rows] and torch.equal(s1, s[:, :1])
        for i in (0, items - 1):                             # alone: the same bits as among others
            alone = tp.tp_beam_select([y[i * beams:(i + 1) * beams] for y in shards], scores[i:i + 1], k)
            assert torch.equal(alone[0][0], s[i]) and alone[2][0].tolist() == want_tokens[i]
    assert tp.tp_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabulary_of_many_chunks(dtype):
    """More chunks than the second kernel asks for at once, with the largest logits first, last, or in the middle, and
    chunks of nothing but -inf."""
    vocab, beams = 450001, 4
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn((1, beams, vocab), device=DEV, generator=g)
    ramp = torch.linspace(0, 30, vocab, device=DEV)
    x[0, 0] += ramp
    x[0, 1] += ramp.flip(0)
    x[0, 2, :200000] = -float("inf")
    x[0, 2, 250000:] = -float("inf")
    x = x.to(dtype)
    scores = -torch.rand((1, beams), device=DEV, generator=g)
    check_beams(x, scores, 10, shards=[x[0]])
    check_beams(x, scores, 3, 3)

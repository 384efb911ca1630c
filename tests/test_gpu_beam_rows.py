"""Beam selection over rows whose edges cut 16-byte words, many of them for each
thread block: against the oracle, tokens exactly."""

import pytest
import torch

from test_gpu_kv_pages import DEV, check_beams

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

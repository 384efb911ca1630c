"""What the decode loop refuses, before any call of the library."""

from types import SimpleNamespace

import pytest
import torch

from megatron_tensor_layers_gb300 import decode_loop as loop


@pytest.mark.parametrize("lengths,beams,steps", [([], 2, 2), ([3, 0], 2, 2), ([0], 2, 2), ([3], 0, 2), ([3], 2, 0), ([3], 2, -1)])
def test_generate_refuses(lengths, beams, steps):
    """A prompt without a token has no last row: its beams would begin with the logits of the prompt before it."""
    prompts = [torch.zeros(n, dtype=torch.int32) for n in lengths]
    with pytest.raises(ValueError, match="prompts|steps"):
        loop.generate(SimpleNamespace(cfg=loop.Config()), prompts, beams, steps)


def test_generate_refuses_other_shapes_and_types():
    for bad in (torch.zeros((2, 3), dtype=torch.int32), torch.zeros(3, dtype=torch.int64)):
        with pytest.raises(ValueError, match="prompts"):
            loop.generate(SimpleNamespace(cfg=loop.Config()), [bad], 2, 2)

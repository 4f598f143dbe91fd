"""The example's model: trains, and decodes token by token what its prompt computes (GPU)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_prompt_and_steps_agree():
    import hybrid_blocks as ex
    torch.manual_seed(1)
    model = ex.Model(vocab=128, pairs=1)
    tokens = torch.randint(0, 128, (3, 90), device="cuda")
    losses = ex.train(model, tokens, 12)
    assert losses[-1] < 0.8 * losses[0]
    with torch.no_grad():
        whole, _ = model.prompt(tokens)
        steps = ex.decode(model, tokens, 70)
    # each of the two blocks' outputs and projections is rounded to bf16 on either path
    assert (steps - whole).double().norm() <= 2e-2 * whole.double().norm()

"""The example's model with attention blocks: runs, gives every parameter a gradient, and decodes token by token what its prompt computes (GPU)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_training_prompt_and_steps():
    import hybrid_blocks as ex
    torch.manual_seed(1)
    model = ex.Model(vocab=128, pairs=1, attention=True)
    tokens = torch.randint(0, 128, (3, 150), device="cuda")
    losses = ex.train(model, tokens, 2)
    assert len(losses) == 2 and all(x == x for x in losses)
    for t in model.parameters():
        assert t.grad is not None and torch.isfinite(t.grad).all() and t.grad.any()
    with torch.no_grad():
        whole, _ = model.prompt(tokens)
        steps = ex.decode(model, tokens, 110)
    # each of the three blocks' outputs and projections is rounded to bf16 on either path
    assert (steps - whole).double().norm() <= 3e-2 * whole.double().norm()


"""The example's cache grows with its sequences: a prompt longer than the pages it starts with, and decoding past their end, compute what one
prompt does (GPU)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("page,pages,T,cut", [(16, 4, 150, 50), (16, 4, 150, 110), (64, 8, 540, 500), (64, 8, 600, 590)])
def test_past_the_first_pages(page, pages, T, cut):
    import hybrid_blocks as ex
    torch.manual_seed(1)
    model = ex.Model(vocab=128, pairs=1, attention=True)
    for b in model.blocks:
        if isinstance(b, ex.AttentionBlock):
            b.page, b.pages = page, pages
    tokens = torch.randint(0, 128, (3, T), device="cuda")
    with torch.no_grad():
        whole, _ = model.prompt(tokens)
        steps = ex.decode(model, tokens, cut)
    # each of the three blocks' outputs and projections is rounded to bf16 on either path
    assert (steps - whole).double().norm() <= 3e-2 * whole.double().norm()
    assert (steps[:, cut:] - whole[:, cut:]).double().norm() <= 3e-2 * whole[:, cut:].double().norm()

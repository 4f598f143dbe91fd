"""A backward keeps the offsets that its forward was called with, whatever becomes of the caller's (GPU)."""
import pytest
import torch

import chunked_gated_delta_05_gb300 as lib

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
T = 90      # both sets of offsets cut it into as many chunks and groups of tokens


def rn(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def rule(g, cu, per_channel):
    q, k, v = (rn(g, 1, T, 2, 128, std=0.5).requires_grad_() for _ in range(3))
    gate = -rn(g, 1, T, 2, *([128] if per_channel else []), dtype=F32).abs() * 0.1
    o, _ = lib.chunk_gated_delta_rule(q, k, v, gate, rn(g, 1, T, 2).sigmoid(), cu_seqlens=cu)
    return o, (q, k, v)


def conv(g, cu):
    x, w = rn(g, 1, T, 64).requires_grad_(), rn(g, 64, 4, dtype=F32).requires_grad_()
    return lib.causal_conv1d(x, w, cu_seqlens=cu), (x, w)


def scan(g, cu):
    u, delta = (rn(g, 1, T, 64).requires_grad_() for _ in range(2))
    B, C = rn(g, 1, T, 1, 8), rn(g, 1, T, 1, 8)
    y, _ = lib.selective_scan(u, delta, -rn(g, 64, 8, dtype=F32).abs(), B, C, cu_seqlens=cu)
    return y, (u, delta)


CALLS = {"gdn": lambda g, cu: rule(g, cu, False), "kda": lambda g, cu: rule(g, cu, True), "conv": conv, "scan": scan}


@pytest.mark.parametrize("as_list", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_offsets_changed_after_the_forward(name, as_list):
    def grads(change):
        g = torch.Generator().manual_seed(1)
        cu = [0, 30, T] if as_list else torch.tensor([0, 30, T], dtype=torch.int32)
        y, leaves = CALLS[name](g, cu)
        if change:
            cu[1] = 60
        return torch.autograd.grad(y, leaves, rn(g, *y.shape))

    for x, y in zip(grads(False), grads(True)):
        assert torch.equal(x, y)

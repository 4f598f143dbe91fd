"""Results do not depend on what workspaces and outputs held before a call, and outputs are written whole (GPU)."""
import contextlib

import pytest
import torch

from test_attention_autograd import freqs, lib, rn

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@contextlib.contextmanager
def filled():
    """New memory is filled with NaN, and with the largest whole numbers."""
    before = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    try:
        assert int(torch.empty(3, dtype=torch.uint8, device="cuda").min()) == 255
        yield
    finally:
        torch.use_deterministic_algorithms(before[0])
        torch.utils.deterministic.fill_uninitialized_memory = before[1]


def both(call):
    a = call()
    with filled():
        b = call()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("cu", [None, [0, 1, 130, 300], list(range(0, 301, 2))])
@pytest.mark.parametrize("D", [64, 128])
def test_whole_sequences(D, cu):
    g = torch.Generator().manual_seed(1)
    q, k, v, dO, dk = (rn(g, 1, 300, h, D) for h in (5, 1, 1, 5, 1))
    w, f = 1 + rn(g, D, dtype=F32, std=0.1), freqs(D)

    def call():
        a, b = lib().qk_norm_rope_fwd(q, k, w, w, f, cu_seqlens=cu)
        o, lse = lib().attention_fwd(a, b, v, cu_seqlens=cu)
        return (a, b, o, lse, *lib().attention_bwd(dO, a, b, v, o, lse, cu_seqlens=cu), *lib().qk_norm_rope_bwd(dO, dk, q, k, w, w, f, cu_seqlens=cu))

    both(call)


@pytest.mark.parametrize("lengths", [[5000], [300, 0, 17, -2, 900], [0, 0], [40] * 200])
@pytest.mark.parametrize("H,Hk,D", [(8, 2, 128), (24, 2, 64), (1, 1, 128)])
def test_steps(H, Hk, D, lengths):
    g = torch.Generator().manual_seed(2)
    B, page = len(lengths), 16
    width = -(-max(1, *lengths) // page) if B > 1 else -(-lengths[0] // page)
    pages = B * max(width, 1)
    kc, vc, q, k, v = rn(g, pages, page, Hk, D), rn(g, pages, page, Hk, D), rn(g, B, H, D), rn(g, B, Hk, D), rn(g, B, Hk, D)
    table = torch.randperm(pages, generator=g).to(I32).view(B, -1).cuda()
    n, w, f = torch.tensor(lengths, dtype=I32, device="cuda"), torch.ones(D, device="cuda"), freqs(D)

    def call():
        c = kc.clone(), vc.clone()
        a, b = lib().qk_norm_rope_store(q, k, v, w, w, f, *c, table, n)
        return a, b, *c, lib().attention_step(a, *c, table, n)

    both(call)

"""Attention where every CTA takes several output tiles, each of several tiles of keys or queries (GPU): rings, accumulators and the handing out of
tiles go on from one to the next. Against the elementwise bounds of the method's roundings, and a sequence in a large call against
the same sequence alone, to the bit."""
import numpy as np
import pytest
import torch

from test_parity_attention import check, lib, rn

pytestmark = pytest.mark.gpu


def documents(n, lo, hi, seed):
    """Mixed lengths, with single tiles and ragged ones among them."""
    lens = np.random.default_rng(seed).integers(lo, hi + 1, n)
    lens[:4] = 128, 1, 256, 129
    return [0, *(int(x) for x in np.cumsum(np.random.default_rng(seed + 1).permutation(lens)))]


def alone(q, k, v, dO, causal, starts, cu=None):
    """A call's outputs against those of each of its sequences by itself."""
    o, lse = lib().attention_fwd(q, k, v, causal=causal, cu_seqlens=cu)
    out = (o, lse, *lib().attention_bwd(dO, q, k, v, o, lse, causal=causal, cu_seqlens=cu))
    flat = [t.flatten(0, 1) for t in (q, k, v, dO, *out)]
    for a, b in zip(starts, starts[1:]):
        q1, k1, v1, dO1, *want = (t[a:b][None] for t in flat)
        o1, lse1 = lib().attention_fwd(q1, k1, v1, causal=causal)
        for x, y in zip(want, (o1, lse1, *lib().attention_bwd(dO1, q1, k1, v1, o1, lse1, causal=causal))):
            assert torch.equal(x, y), (a, b)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_documents(D, causal):
    g = torch.Generator().manual_seed(D)
    cu = documents(40, 100, 700, 1)
    alone(*(rn(g, 1, cu[-1], n, D) for n in (8, 2, 2, 8)), causal, cu, cu=cu)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,B,T,H,Hk", [(128, 12, 385, 16, 16), (64, 12, 385, 16, 4), (128, 20, 511, 5, 1), (64, 3, 1300, 16, 8)])
def test_batches(D, B, T, H, Hk, causal):
    g = torch.Generator().manual_seed(T)
    alone(*(rn(g, B, T, n, D) for n in (H, Hk, Hk, H)), causal, [b * T for b in range(B + 1)])


@pytest.mark.parametrize("D,causal", [(64, True), (128, True), (128, False)])
def test_documents_within_bounds(D, causal):
    cu = documents(30, 100, 600, 3)
    check(1, cu[-1], 8, 2, D, causal, cu=cu, seed=1)


@pytest.mark.parametrize("D,B,T,H,Hk,causal", [(64, 1, 1500, 16, 2, True), (128, 1, 1500, 16, 2, True), (64, 1, 1100, 16, 1, False), (128, 1, 1300, 12, 1, True),
                                               (64, 4, 600, 16, 8, True), (128, 6, 385, 16, 16, False)])
def test_batches_within_bounds(D, B, T, H, Hk, causal):
    """Few key heads over many tiles among them."""
    check(B, T, H, Hk, D, causal, seed=2)

"""What stands beside a sequence in a call (GPU)."""
import pytest
import torch

from test_parity_attention import lib, rn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cu", [[0, 200, 333], [0, 135, 400, 401], [0, 300, 700]])
def test_documents_have_the_bits_they_have_alone(cu, D, causal):
    """A document's last tile of queries is filled up with its neighbour's: large ones that would move a softmax's reference change no bit
    of a document of several tiles."""
    g = torch.Generator().manual_seed(cu[1] + D)
    R, H, Hk = cu[-1], 8, 2
    q, k, v, dO = (rn(g, 1, R, n, D) for n in (H, Hk, Hk, H))
    q[:, cu[1]:] *= 40
    o, lse = lib().attention_fwd(q, k, v, causal=causal, cu_seqlens=cu)
    grads = lib().attention_bwd(dO, q, k, v, o, lse, causal=causal, cu_seqlens=cu)
    for a, b in zip(cu, cu[1:]):
        part = [t[:, a:b].contiguous() for t in (q, k, v)]
        o1, lse1 = lib().attention_fwd(*part, causal=causal)
        for x, y in zip((o, lse, *grads), (o1, lse1, *lib().attention_bwd(dO[:, a:b].contiguous(), *part, o1, lse1, causal=causal))):
            assert torch.equal(x[:, a:b], y)

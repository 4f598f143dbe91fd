"""Offsets of packed documents are refused alike with and without gradients (CPU)."""
import pytest
import torch

import chunked_gated_delta_05_gb300 as lib


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("call", [lambda q, k, w, cu: lib.qk_norm_rope(q, k, w, w, torch.ones(32), cu_seqlens=cu), lambda q, k, w, cu: lib.attention(q, k, k, cu_seqlens=cu)],
                         ids=["qk_norm_rope", "attention"])
@pytest.mark.parametrize("cu", [torch.tensor([0, 4], dtype=torch.int16), torch.tensor([[0, 4]], dtype=torch.int32), torch.tensor([0.0, 4.0]), [0, 4.0], [True, 4], [0]],
                         ids=["int16", "two dimensions", "float", "float in a list", "bool", "one"])
def test_refused_with_and_without_gradients(call, cu, grad):
    q, k = (torch.zeros(1, 4, h, 64, dtype=torch.bfloat16, requires_grad=grad) for h in (2, 1))
    with pytest.raises(ValueError, match="cu_seqlens"):
        call(q, k, torch.ones(64), cu)


@pytest.mark.parametrize("grad", [False, True])
def test_offsets_on_a_device_are_refused(grad):
    q, k = (torch.zeros(1, 4, h, 64, dtype=torch.bfloat16, requires_grad=grad) for h in (2, 1))
    cu = torch.zeros(2, dtype=torch.int32, device="meta")
    for call in (lambda: lib.qk_norm_rope(q, k, None, None, torch.ones(32), cu_seqlens=cu), lambda: lib.attention(q, k, k, cu_seqlens=cu)):
        with pytest.raises(ValueError, match="cu_seqlens"):
            call()

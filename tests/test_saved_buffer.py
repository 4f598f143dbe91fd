"""A buffer of kept states that does not hold what its element count says is refused before the kernels read it."""
import pytest
import torch

import chunked_gated_delta_05_gb300 as lib
from chunked_gated_delta_05_gb300 import _lib, block_ops, ops

BF16 = torch.bfloat16


def short(n, device):
    """n elements in one byte of memory, and n in every second one of 2 n."""
    return [torch.zeros(1, dtype=torch.uint8, device=device).expand(n), torch.zeros(2 * n, dtype=torch.uint8, device=device)[::2]]


def test_selective_scan_bwd(monkeypatch):
    monkeypatch.setattr(block_ops, "_device", lambda name, t: -1)
    monkeypatch.setattr(block_ops, "_run", lambda *a: None)
    monkeypatch.setattr(_lib, "size", lambda name, d: 4096)
    u, A, B = torch.zeros(1, 4, 8, dtype=BF16), torch.zeros(8, 2), torch.zeros(1, 4, 1, 2, dtype=BF16)
    lib.selective_scan_bwd(u, u, A, B, B, u, saved=torch.zeros(4096, dtype=torch.uint8))
    for bad in short(4096, "cpu"):
        with pytest.raises(ValueError, match="saved"):
            lib.selective_scan_bwd(u, u, A, B, B, u, saved=bad)


def test_gdn_bwd(monkeypatch):
    class Host:     # the library with a saved size, and no kernels
        def __getattr__(self, name):
            return lambda *a: 4096

    monkeypatch.setattr(_lib, "load", Host)
    monkeypatch.setattr(ops, "_common_checks", lambda q, k, v, *a: (1, 4, 1, 1, 1, torch.device("cpu")))
    monkeypatch.setattr(ops, "_launch", lambda *a: None)
    q, g, beta = torch.zeros(1, 4, 1, 128, dtype=BF16), torch.zeros(1, 4, 1), torch.zeros(1, 4, 1, dtype=BF16)
    lib.gdn_bwd(q, q, q, g, beta, q, saved=torch.zeros(4096, dtype=torch.uint8))
    for bad in short(4096, "cpu"):
        with pytest.raises(ValueError, match="saved"):
            lib.gdn_bwd(q, q, q, g, beta, q, saved=bad)

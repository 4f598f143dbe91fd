"""Scores of minus infinity (GPU)."""
import math

import numpy as np
import pytest
import torch

from _util import f64
from oracle import attention as A
from test_parity_attention import lib, rn, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shut", [(0, 64), (0, 128), (0, 130), (0, 300), (0, 384), (40, 200), (128, 400)])
def test_scores_of_minus_infinity_weigh_nothing(shut, D):
    """Keys that an infinite channel shuts off, whole tiles of them at a row's beginning too: the others are weighed as if alone.
    Tolerance: weights and output rounded to bf16, scores fp32 sums of D products."""
    g = torch.Generator().manual_seed(D)
    T, H = 450, 2
    q, k, v = rn(g, 1, T, H, D), rn(g, 1, T, 1, D), rn(g, 1, T, 1, D)
    q[..., 5] = q[..., 5].abs() + 0.125
    k[0, shut[0]: shut[1], 0, 5] = -math.inf
    open_ = np.array([j for j in range(T) if not shut[0] <= j < shut[1]])
    for causal in (False, True):
        o, lse = lib().attention_fwd(q, k, v, causal=causal)
        Q, K, V = rows(q), rows(k), rows(v)
        for i in range(0, T, 7):
            keys = open_[open_ <= i] if causal else open_
            if len(keys) == 0:
                continue
            for h in range(H):
                P, L = A.weights(Q[i: i + 1, h], K[keys, 0], D ** -0.5, False)
                want, size = (P @ V[keys, 0])[0], (P @ np.abs(V[keys, 0]))[0]
                assert (np.abs(f64(o)[0, i, h] - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2e-4) * size).all(), (causal, i)
                assert abs(f64(lse)[0, i, h] - L[0]) <= 2e-4

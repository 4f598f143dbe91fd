"""Norm and rotation in calls whose offsets do not travel with the launch, and whose warps take several tokens each (GPU), with the
tolerances of the smaller calls."""
import numpy as np
import pytest

from test_parity_rope import check, check_store

pytestmark = pytest.mark.gpu


def lengths(n, most, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(1, most + 1, n)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [62, 63, 64, 65, 300])
def test_many_documents(n, D):
    cu = [0, *(int(x) for x in np.cumsum(lengths(n, 9, n)))]
    check(1, cu[-1], 3, 1, D, D, cu=cu)


@pytest.mark.parametrize("n", [62, 63, 64, 65, 300])
def test_many_prompts_into_a_cache(n):
    new = lengths(n, 4, n)
    before = lengths(n, 30, n + 1)
    total = [0 if i % 11 == 5 else a + b for i, (a, b) in enumerate(zip(new, before))]
    check_store(total, new, 2, 1, 64, 8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_many_tokens(packed, D):
    if packed:
        cu = [0, *(int(x) for x in np.cumsum(lengths(90, 190, 7)))]
        check(1, cu[-1], 2, 1, D, D // 2, cu=cu)
    else:
        check(2, 4001, 2, 1, D, D)


def test_many_tokens_into_a_cache():
    new = [2500, 1, 1700, 40]
    check_store([2600, 1, 1700, 90], new, 1, 1, 128, 64)

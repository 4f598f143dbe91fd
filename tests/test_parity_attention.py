"""Attention over whole sequences against its fp64 definition (GPU). Tolerances: the elementwise bounds of the roundings the method
makes (``oracle.attention.bounds``): the softmax's weights and their gradients rounded once to bf16, outputs once more, fp32 elsewhere."""
import numpy as np
import pytest
import torch

from _util import f64
from oracle import attention as A

pytestmark = pytest.mark.gpu


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def rn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def rows(t):
    return f64(t).reshape(-1, *t.shape[-2:])


def check(B, T, H, Hk, D, causal, cu=None, scale=None, seed=0, std=1.0, backward=True):
    g = torch.Generator().manual_seed(seed + 7 * T + H)
    q, k, v, dO = rn(g, B, T, H, D, std=std), rn(g, B, T, Hk, D, std=std), rn(g, B, T, Hk, D), rn(g, B, T, H, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(causal=causal, scale=scale, cu_seqlens=cu, status=status)
    o, lse = lib().attention_fwd(q, k, v, **kw)
    got = {"o": o, "lse": lse}
    if backward:
        got.update(zip(("dq", "dk", "dv"), lib().attention_bwd(dO, q, k, v, o, lse, **kw)))
    assert int(status.item()) == 0
    starts = [b * T for b in range(B + 1)] if cu is None else cu
    exact, bound = A.bounds(*(rows(t) for t in (dO, q, k, v)), starts, D ** -0.5 if scale is None else scale, causal, tile=128)
    for n, t in got.items():
        x = f64(t).reshape(exact[n].shape)
        assert np.isfinite(x).all(), n
        over = np.abs(x - exact[n]) - bound[n]
        assert over.max() <= 0, f"{n}: off by {over.max():.3e} more than allowed"
    return got


LENGTHS = [1, 2, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 384, 385, 513, 700]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, causal):
    check(1, T, 2, 1, 128, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T", [1, 100, 129, 300, 520])
def test_small_heads(T, causal):
    check(2, T, 4, 2, 64, causal)


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2), (7, 1), (8, 8), (16, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(H, Hk, D):
    check(1, 150, H, Hk, D, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cu", [[0, 1], [0, 1, 2, 3], [0, 1, 130, 131, 400], [0, 128, 256, 512], [0, 300, 301, 700], [0, 5, 260, 517, 518, 900]])
def test_documents(cu, causal):
    check(1, cu[-1], 4, 2, 128, causal, cu=cu)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_a_query_of_a_single_key_has_no_gradient_of_scores(D, causal):
    cu = [0, 1, 2, 3, 7, 8, 140, 141]
    got = check(1, cu[-1], 4, 2, D, causal, cu=cu, seed=3)
    for a, b in zip(cu, cu[1:]):
        if b - a == 1:
            assert not got["dq"][0, a].any() and not got["dk"][0, a].any()
        elif causal:
            assert not got["dq"][0, a].any()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_few_keys(D, causal):
    # D of a query with few keys is taken from its scores: with the rounded o's it lay outside these bounds
    check(1, 360, 6, 2, D, causal, cu=[0, 3, 7, 12, 40, 41, 43, 90, 218, 360], seed=5)


def test_many_documents():
    cu = np.concatenate([[0], np.cumsum(np.random.default_rng(0).integers(1, 9, 1500))]).tolist()      # tables of several uploads
    check(1, cu[-1], 2, 1, 64, True, cu=[int(x) for x in cu])


@pytest.mark.parametrize("D", [64, 128])
def test_own_scale(D):
    check(1, 190, 2, 2, D, True, scale=0.3)


@pytest.mark.parametrize("causal", [True, False])
def test_peaked_scores(causal):
    """Scores of tens: rows that look at one key, references that move from tile to tile."""
    check(1, 600, 2, 1, 128, causal, std=3.0)


def test_references_move_up_and_down():
    """Keys that grow, then shrink, along the sequence."""
    g = torch.Generator().manual_seed(3)
    T, H, D = 900, 2, 128
    q, k, v = rn(g, 1, T, H, D), rn(g, 1, T, 1, D), rn(g, 1, T, 1, D)
    grow = torch.cat([torch.linspace(0.1, 8, T // 2), torch.linspace(8, 0.1, T - T // 2)]).view(1, T, 1, 1).cuda()
    k = (k * grow).to(torch.bfloat16)
    o, lse = lib().attention_fwd(q, k, v, causal=False)
    exact, bound = A.bounds(np.zeros((T, H, D)), rows(q), rows(k), rows(v), [0, T], D ** -0.5, False)
    for n, t in (("o", o), ("lse", lse)):
        assert (np.abs(f64(t).reshape(exact[n].shape) - exact[n]) <= bound[n]).all(), n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [4, 16])
@pytest.mark.parametrize("at", [0, 100, 130, 200, 255, 256, 383, 399])
def test_a_key_far_above_the_others(at, far, D):
    """Some queries meet one key whose score moves their reference, in either half of any tile, the others do not."""
    g = torch.Generator().manual_seed(at + D)
    T, H = 400, 2
    q, k, v = rn(g, 1, T, H, D), rn(g, 1, T, 1, D), rn(g, 1, T, 1, D)
    k[0, at, 0] = q[0, T - 1, 0] * far      # a score of far sqrt(D) for that query (16: 2 to its power overflows fp32), less for the others
    q[0, ::7, 1] = q[0, T - 1, 0]
    for causal in (True, False):
        o, lse = lib().attention_fwd(q, k, v, causal=causal)
        exact, bound = A.bounds(np.zeros((T, H, D)), rows(q), rows(k), rows(v), [0, T], D ** -0.5, causal)
        for n, t in (("o", o), ("lse", lse)):
            assert (np.abs(f64(t).reshape(exact[n].shape) - exact[n]) <= bound[n]).all(), n


def test_strided_inputs():
    """q, k and v as slices of one projection give the bits of contiguous ones."""
    g = torch.Generator().manual_seed(5)
    B, T, H, Hk, D = 2, 333, 4, 2, 128
    mixed = rn(g, B, T, (H + 2 * Hk) * D + 24)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in mixed[..., 8: 8 + (H + 2 * Hk) * D].split([H * D, Hk * D, Hk * D], -1))
    dO = rn(g, B, T, H, D)
    o, lse = lib().attention_fwd(q, k, v)
    a = [o, lse, *lib().attention_bwd(dO, q, k, v, o, lse)]
    q, k, v = (t.contiguous() for t in (q, k, v))
    o, lse = lib().attention_fwd(q, k, v)
    for x, y in zip(a, [o, lse, *lib().attention_bwd(dO, q, k, v, o, lse)]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_neighbours_nan_stays_there(bad, causal):
    """Documents next to one full of NaN or infinities compute what they compute alone."""
    g = torch.Generator().manual_seed(6)
    cu, H, Hk, D = [0, 70, 200, 333], 4, 2, 128
    q, k, v, dO = (rn(g, 1, 333, n, D) for n in (H, Hk, Hk, H))
    for t in (q, k, v, dO):
        t[:, 70:200] = bad
    o, lse = lib().attention_fwd(q, k, v, causal=causal, cu_seqlens=cu)
    grads = lib().attention_bwd(dO, q, k, v, o, lse, causal=causal, cu_seqlens=cu)
    for a, b in ((0, 70), (200, 333)):
        part = [t[:, a:b].contiguous() for t in (q, k, v)]
        o1, lse1 = lib().attention_fwd(*part, causal=causal)
        for x, y in zip((o, lse, *grads), (o1, lse1, *lib().attention_bwd(dO[:, a:b].contiguous(), *part, o1, lse1, causal=causal))):
            assert torch.equal(x[:, a:b], y)


def test_batch_rows_are_independent_and_runs_repeat():
    g = torch.Generator().manual_seed(8)
    q, k, v, dO = rn(g, 3, 300, 8, 128), rn(g, 3, 300, 2, 128), rn(g, 3, 300, 2, 128), rn(g, 3, 300, 8, 128)
    o, lse = lib().attention_fwd(q, k, v)
    grads = lib().attention_bwd(dO, q, k, v, o, lse)
    for _ in range(3):
        o2, lse2 = lib().attention_fwd(q, k, v)
        for x, y in zip((o, lse, *grads), (o2, lse2, *lib().attention_bwd(dO, q, k, v, o2, lse2))):
            assert torch.equal(x, y)
    o1, _ = lib().attention_fwd(q[1:2].contiguous(), k[1:2].contiguous(), v[1:2].contiguous())
    assert torch.equal(o[1:2], o1)


def test_long_rows():
    """Thousands of keys: a few query rows against the definition."""
    g = torch.Generator().manual_seed(9)
    T, H, D = 5000, 2, 128
    q, k, v = rn(g, 1, T, H, D), rn(g, 1, T, 1, D), rn(g, 1, T, 1, D)
    o, lse = lib().attention_fwd(q, k, v)
    Q, K, V = rows(q), rows(k), rows(v)
    for i in (0, 127, 128, 255, 256, 2560, 4095, 4096, 4999):
        for h in range(H):
            P, L = A.weights(Q[i: i + 1, h], K[: i + 1, 0], D ** -0.5, False)
            want = P @ V[: i + 1, 0]
            # weights and output rounded to bf16; scores are fp32 sums of 128 products
            assert (np.abs(f64(o)[0, i, h] - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -8 + 2e-4) * (P @ np.abs(V[: i + 1, 0]))[0]).all()
            assert abs(f64(lse)[0, i, h] - L[0]) <= 2e-4

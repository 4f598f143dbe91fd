"""Pins of the attention blocks' fp64 definitions (CPU): closed forms, an independent torch computation, finite differences."""
import numpy as np
import pytest
import torch

from oracle import attention as A


def rng(seed):
    return np.random.default_rng(seed)


def test_turn_is_a_rotation_by_the_angle():
    x = np.zeros((3, 1, 8))
    x[:, 0, 0] = 1.0
    f = np.array([0.5, 0.25])
    y = A.turn(x, [0, 1, 4], f, False)
    np.testing.assert_allclose(y[:, 0, 0], np.cos([0, 0.5, 2.0]))
    np.testing.assert_allclose(y[:, 0, 2], np.sin([0, 0.5, 2.0]))
    y = A.turn(x, [0, 1, 4], f, True)
    np.testing.assert_allclose(y[:, 0, 1], np.sin([0, 0.5, 2.0]))
    z = rng(0).standard_normal((3, 2, 8))
    for inter in (False, True):
        np.testing.assert_allclose(A.turn(A.turn(z, [3, 9, 1], f, inter), [3, 9, 1], f, inter, back=True), z)
        np.testing.assert_allclose((A.turn(z, [3, 9, 1], f, inter) ** 2).sum(-1), (z ** 2).sum(-1))
        np.testing.assert_array_equal(A.turn(z, [3, 9, 1], f, inter)[..., 4:], z[..., 4:])


def test_products_of_turned_vectors_depend_on_the_distance():
    q, k = rng(1).standard_normal((2, 1, 1, 16))
    f = 1.0 / 100.0 ** (np.arange(8) / 8)
    dot = lambda i, j: (A.turn(q, [i], f, False) * A.turn(k, [j], f, False)).sum()  # noqa: E731
    np.testing.assert_allclose(dot(7, 3), dot(104, 100))


def differences(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("inter,norm", [(False, True), (True, True), (False, False)])
def test_norm_rope_adjoint(inter, norm):
    g = rng(2)
    x, dy, w = g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 8)), 1 + 0.1 * g.standard_normal(8)
    pos, f = [0, 3, 2, 900, 1], np.array([1.0, 0.3, 0.01])
    dx, dw, _ = A.norm_rope_bwd(dy, x, w if norm else None, pos, f, 1e-3, inter)
    loss = lambda x, w: (A.norm_rope(x, w if norm else None, pos, f, 1e-3, inter)[0] * dy).sum()  # noqa: E731
    e, ew = g.standard_normal(x.shape), g.standard_normal(8)
    np.testing.assert_allclose((dx * e).sum(), differences(lambda t: loss(t, w), x, e), rtol=1e-6)
    if norm:
        np.testing.assert_allclose((dw * ew).sum(), differences(lambda t: loss(x, t), w, ew), rtol=1e-6)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (3, 1)])
def test_attention_against_torch_and_differences(H, Hk, causal):
    g = rng(3)
    starts = [0, 1, 7, 12]
    q, dO = g.standard_normal((2, 12, H, 6))
    k, v = g.standard_normal((2, 12, Hk, 6))
    o, lse = A.attention(q, k, v, starts, 0.4, causal)
    for a, b in zip(starts, starts[1:]):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x[a:b].repeat(H // x.shape[1], 1).swapaxes(0, 1)))  # noqa: E731
        want = torch.nn.functional.scaled_dot_product_attention(t(q), t(k), t(v), is_causal=causal, scale=0.4)
        np.testing.assert_allclose(o[a:b].swapaxes(0, 1), want.numpy(), rtol=1e-10)
    np.testing.assert_allclose(lse[0], 0.4 * (q[0] * k[0].repeat(H // Hk, 0)).sum(-1))
    loss = lambda q, k, v: (A.attention(q, k, v, starts, 0.4, causal)[0] * dO).sum()  # noqa: E731
    for grad, name in zip(A.attention_bwd(dO, q, k, v, starts, 0.4, causal), "qkv"):
        x = {"q": q, "k": k, "v": v}
        d = g.standard_normal(x[name].shape)
        np.testing.assert_allclose((grad * d).sum(), differences(lambda t: loss(**{**x, name: t}), x[name], d), rtol=1e-6)


def test_step_is_the_last_row_of_the_prompt():
    g = rng(4)
    q, k, v = g.standard_normal((9, 4, 6)), g.standard_normal((9, 2, 6)), g.standard_normal((9, 2, 6))
    o, _ = A.attention(q, k, v, [0, 9], 0.3, True)
    kc, vc = np.full((2, 5, 4, 2, 6), np.nan)
    table = np.array([[3, 1, 4], [0, 0, 0]])
    for t in range(9):
        kc[table[0, t // 4], t % 4], vc[table[0, t // 4], t % 4] = k[t], v[t]
    out = A.attention_step(np.stack([q[8], q[8]]), kc, vc, table, [9, 0], 0.3)
    np.testing.assert_allclose(out[0], o[8])
    assert not out[1].any()


@pytest.mark.parametrize("causal", [True, False])
def test_bounds_hold_for_a_computation_in_rounded_operands(causal):
    """The method with bf16 weights and fp32 sums, emulated, stays inside the bounds the GPU tests use."""
    g = rng(5)
    bf = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()  # noqa: E731
    q, k, v, dO = (bf(x) for x in g.standard_normal((4, 60, 1, 32)))
    starts, scale = [0, 25, 60], 32 ** -0.5
    exact, bound = A.bounds(dO, q, k, v, starts, scale, causal)
    got = {n: np.zeros_like(exact[n]) for n in exact}
    for a, b in zip(starts, starts[1:]):
        Q, K, V, O = (x[a:b, 0] for x in (q, k, v, dO))
        P, lse = A.weights(Q, K, scale, causal)
        o = bf(bf(P) @ V)
        dS = bf(P * (O @ V.T - (O * o).sum(-1, keepdims=True)))
        for n, x in dict(o=o, dv=bf(bf(P).T @ O), dq=bf(scale * dS @ K), dk=bf(scale * dS.T @ Q)).items():
            got[n][a:b, 0] = x
        got["lse"][a:b, 0] = lse
    for n in exact:
        assert (np.abs(got[n] - exact[n]) <= bound[n]).all(), n

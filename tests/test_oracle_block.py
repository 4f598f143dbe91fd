"""Pins of the fp64 definitions in oracle/block.py (CPU): finite differences of every gradient, closed forms, and
consistency of packed sequences, groups and initial states."""
import numpy as np
import pytest

from oracle import block

rng = np.random.default_rng(7)


def fd(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def check_fd(f, args, grads, tol=1e-6):
    for name, g in grads.items():
        d = rng.standard_normal(args[name].shape)
        num = fd(lambda v: f(**{**args, name: v}), args[name], d)
        assert abs(num - (g * d).sum()) <= tol * max(1.0, abs(num)), name


@pytest.mark.parametrize("scale,with_res", [(0.7, True), (1.0, False)])
def test_add_norm_gradients(scale, with_res):
    a = {"x": rng.standard_normal((3, 5)), "weight": rng.standard_normal(5)}
    if with_res:
        a["residual"] = rng.standard_normal((3, 5))
    dy, ds = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def f(x, weight, residual=None):
        y, r = block.add_norm(x, residual, weight, 1e-3, scale)
        return (y * dy).sum() + (r * ds).sum()

    stream = block.add_norm(a["x"], a.get("residual"), a["weight"], 1e-3, scale)[1]
    dx, dr, dw = block.add_norm_bwd(dy, ds, stream, a["weight"], 1e-3, scale)
    check_fd(f, a, {"x": dx, "weight": dw, **({"residual": dr} if with_res else {})})


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gated_norm_gradients(act):
    a = {"x": rng.standard_normal((3, 5)), "gate": rng.standard_normal((3, 5)), "weight": rng.standard_normal(5)}
    dy = rng.standard_normal((3, 5))
    dx, dg, dw = block.gated_norm_bwd(a["x"], a["gate"], a["weight"], dy, 1e-3, act)
    check_fd(lambda x, gate, weight: (block.gated_norm(x, gate, weight, 1e-3, act) * dy).sum(), a, {"x": dx, "gate": dg, "weight": dw})


def test_norm_of_a_constant_row():
    y, r = block.add_norm(np.full((1, 4), 3.0), None, np.arange(4.0), 0.0, 1.0)
    assert np.allclose(y, np.arange(4.0)) and np.allclose(r, 3.0)
    assert np.allclose(block.gated_norm(np.zeros((1, 4)), np.ones((1, 4)), np.ones(4), 1e-6, "silu"), 0.0)


def scan_case(R, D, N, G, starts):
    a = {"u": rng.standard_normal((R, D)), "delta": rng.standard_normal((R, D)), "A": -np.exp(rng.standard_normal((D, N))),
         "B": rng.standard_normal((R, G, N)), "C": rng.standard_normal((R, G, N)), "D": rng.standard_normal(D),
         "z": rng.standard_normal((R, D)), "delta_bias": rng.standard_normal(D), "h0": rng.standard_normal((len(starts) - 1, D, N))}
    return a


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("G,starts", [(1, [0, 6]), (2, [0, 1, 4, 6])])
def test_scan_gradients(G, starts, softplus):
    a = scan_case(6, 4, 3, G, starts)
    if not softplus:    # step sizes as they are: positive
        a["delta"], a["delta_bias"] = np.abs(a["delta"]), np.abs(a["delta_bias"])
    dy, df = rng.standard_normal((6, 4)), rng.standard_normal(a["h0"].shape)

    def f(**kw):
        y, final, _ = block.scan(softplus=softplus, starts=starts, **kw)
        return (y * dy).sum() + (final * df).sum()

    g = block.scan_bwd(dy=dy, dfinal=df, softplus=softplus, starts=starts, **a)
    check_fd(f, a, {k: g["d" + k] for k in a}, tol=1e-5)


def test_scan_packed_is_separate_runs():
    a = scan_case(7, 4, 3, 1, [0, 3, 7])
    y, final, _ = block.scan(starts=[0, 3, 7], **a)
    for s, (lo, hi) in enumerate([(0, 3), (3, 7)]):
        part = {k: (v[lo:hi] if k in ("u", "delta", "B", "C", "z") else v) for k, v in a.items()}
        part["h0"] = a["h0"][s:s + 1]
        y1, f1, _ = block.scan(**part)
        assert np.allclose(y[lo:hi], y1) and np.allclose(final[s], f1[0])


def test_scan_closed_forms():
    # A = 0: the state is a running sum; one token: y = C . (dt u B) + D u
    one, two = np.ones((1, 1, 1)), 2 * np.ones((1, 1, 1))
    y, final, _ = block.scan(np.array([[3.0]]), np.array([[0.5]]), np.zeros((1, 1)), one, two, D=np.array([10.0]), softplus=False)
    assert np.allclose(y, 2 * 0.5 * 3 + 30) and np.allclose(final, 1.5)
    u = rng.standard_normal((5, 1))
    _, final, _ = block.scan(u, np.ones((5, 1)), np.zeros((1, 1)), np.ones((5, 1, 1)), np.ones((5, 1, 1)), softplus=False)
    assert np.allclose(final, u.sum())
    # softplus(0) = log 2, and exp(dt A) alone without input
    _, final, _ = block.scan(np.zeros((4, 1)), np.zeros((4, 1)), -np.ones((1, 1)), np.ones((4, 1, 1)), np.ones((4, 1, 1)), h0=np.ones((1, 1, 1)))
    assert np.allclose(final, 0.5 ** 4)


@pytest.mark.parametrize("dilation", [1, 2])
def test_conv_step_is_the_convolution(dilation):
    from oracle import conv
    T, C, W = 6, 3, 3
    x, w, b = rng.standard_normal((1, T, C)), rng.standard_normal((C, W)), rng.standard_normal(C)
    want = conv.causal_conv1d(x, w, b, dilation=dilation)
    state = np.zeros((1, (W - 1) * dilation, C))
    for t in range(T):
        y, state = block.conv_step(state, x[:, t], w, b, dilation)
        assert np.allclose(y, want[:, t])

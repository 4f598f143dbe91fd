"""fp64 definitions of the operators around the recurrence: the norms before and after a block and the selective
state space scan, forward and adjoint, written token by token from their formulas. The single-token forms are these on
sequences of one token."""
import numpy as np


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def add_norm(x, residual, weight, eps, scale, keep=lambda r: r):
    """``(y, stream)``: stream = keep(residual + scale x) (keep: the rounding to the stream's type), or x."""
    r = x if residual is None else keep(residual + scale * x)
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * weight, r


def add_norm_bwd(dy, dstream, stream, weight, eps, scale):
    """``(dx, dresidual, dweight)`` of <dy, y> + <dstream, stream>."""
    rstd = 1.0 / np.sqrt((stream * stream).mean(-1, keepdims=True) + eps)
    xh, d = stream * rstd, dy * weight
    dr = rstd * (d - xh * (d * xh).mean(-1, keepdims=True)) + (0.0 if dstream is None else dstream)
    return scale * dr, dr, (dy * xh).reshape(-1, dy.shape[-1]).sum(0)


def gated_norm(x, gate, weight, eps, activation):
    act = sigmoid(gate) * (gate if activation == "silu" else 1.0)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight * act


def gated_norm_bwd(x, gate, weight, dy, eps, activation):
    """``(dx, dgate, dweight)``."""
    sg = sigmoid(gate)
    act, dact = (gate * sg, sg * (1 + gate * (1 - sg))) if activation == "silu" else (sg, sg * (1 - sg))
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx, _, dw = add_norm_bwd(dy * act, None, x, weight, eps, 1.0)
    return dx, dy * n * weight * dact, dw


def scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, h0=None, starts=None):
    """Selective scan of rows ``u [R,D]``, ``B [R,G,N]``, cut into sequences at ``starts`` (offsets 0 .. R). Returns
    ``(y [R,D], final [S,D,N], tape)``."""
    R, Dc = u.shape
    N, G = A.shape[1], B.shape[1]
    starts = [0, R] if starts is None else list(starts)
    group = np.arange(Dc) // (Dc // G)
    x = delta if delta_bias is None else delta + delta_bias
    dt = np.logaddexp(x, 0.0) if softplus else x
    h_all, before = np.zeros((R, Dc, N)), np.zeros((R, Dc, N))
    final = np.zeros((len(starts) - 1, Dc, N))
    for s in range(len(starts) - 1):
        h = np.zeros((Dc, N)) if h0 is None else h0[s].copy()
        for t in range(starts[s], starts[s + 1]):
            before[t] = h
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * u[t])[:, None] * B[t][group]
            h_all[t] = h
        final[s] = h
    y0 = np.einsum("rdn,rdn->rd", h_all, C[:, group])
    if D is not None:
        y0 = y0 + D * u
    y = y0 if z is None else y0 * z * sigmoid(z)
    return y, final, (x, dt, before, h_all, y0)


def scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, softplus=True, h0=None, starts=None, dfinal=None):
    """Adjoint of :func:`scan`: a dict of du, ddelta, dA, dB, dC, dD, dz, ddelta_bias, dh0."""
    R, Dc = u.shape
    N, G = A.shape[1], B.shape[1]
    starts = [0, R] if starts is None else list(starts)
    group = np.arange(Dc) // (Dc // G)
    _, _, (x, dt, before, h_all, y0) = scan(u, delta, A, B, C, D, z, delta_bias, softplus, h0, starts)
    out = {"dA": np.zeros_like(A), "dB": np.zeros_like(B), "dC": np.zeros_like(C), "dh0": np.zeros((len(starts) - 1, Dc, N))}
    dy0 = dy
    if z is not None:
        sg = sigmoid(z)
        dy0 = dy * z * sg
        out["dz"] = dy * y0 * sg * (1 + z * (1 - sg))
    du, ddt = np.zeros_like(u), np.zeros_like(u)
    for s in range(len(starts) - 1):
        g = np.zeros((Dc, N)) if dfinal is None else dfinal[s].copy()
        for t in range(starts[s + 1] - 1, starts[s] - 1, -1):
            g = g + dy0[t][:, None] * C[t][group]
            np.add.at(out["dC"][t], group, dy0[t][:, None] * h_all[t])
            np.add.at(out["dB"][t], group, (dt[t] * u[t])[:, None] * g)
            gB = (g * B[t][group]).sum(-1)
            g = g * np.exp(dt[t][:, None] * A)
            w = g * before[t]
            out["dA"] += w * dt[t][:, None]
            du[t] = dt[t] * gB
            ddt[t] = u[t] * gB + (w * A).sum(-1)
        out["dh0"][s] = g
    if D is not None:
        du = du + D * dy0
        out["dD"] = (dy0 * u).sum(0)
    out["du"], out["ddelta"] = du, ddt * (sigmoid(x) if softplus else 1.0)
    out["ddelta_bias"] = out["ddelta"].sum(0)
    return out


def conv_step(state, x, weight, bias, dilation, silu=True):
    """One token of the short convolution: ``(y [B,C], new state [B,HW,C])`` for state rows oldest first."""
    seen = np.concatenate([state, x[:, None]], 1)
    z = np.einsum("bwc,cw->bc", seen[:, ::dilation], weight) + (0.0 if bias is None else bias)
    return (z * sigmoid(z) if silu else z), seen[:, 1:]

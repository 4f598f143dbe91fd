"""fp64 definitions of the attention blocks: norm and rotation of query and key heads with its adjoint, attention over whole
sequences with its adjoint, and a token's attention over a paged cache; written head by head from their formulas."""
import numpy as np


def turn(x, positions, inv_freq, interleaved, back=False):
    """x [R,H,D]: the first 2 len(inv_freq) channels in pairs, the i-th turned by positions inv_freq[i] (``back``: the other way)."""
    n = len(inv_freq)
    angle = np.multiply.outer(np.asarray(positions, np.float64), inv_freq) * (-1.0 if back else 1.0)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def norm_rope(x, weight, positions, inv_freq, eps, interleaved=False):
    """``(y, normed)`` of heads x [R,H,D]; weight None: no norm."""
    n = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    return turn(n, positions, inv_freq, interleaved), n


def norm_rope_bwd(dy, x, weight, positions, inv_freq, eps, interleaved=False):
    """``(dx, dweight, size of dx's terms)``."""
    d = turn(dy, positions, inv_freq, interleaved, back=True)
    if weight is None:
        return d, None, np.abs(d)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, g = x * r, d * weight
    mean = (g * xh).mean(-1, keepdims=True)
    return r * (g - xh * mean), (d * xh).sum((0, 1)), r * (np.abs(g) + np.abs(xh * mean))


def weights(q, k, scale, causal):
    """Softmax weights [Tq,Tk] and the logarithms of their denominators; with fewer queries than keys, the queries are the last tokens."""
    s = scale * (q @ k.T)
    if causal:
        s = np.where(np.arange(k.shape[0])[None] > np.arange(q.shape[0])[:, None] + k.shape[0] - q.shape[0], -np.inf, s)
    top = s.max(-1, keepdims=True)
    e = np.exp(s - top)
    total = e.sum(-1, keepdims=True)
    return e / total, (top + np.log(total))[:, 0]


def attention(q, k, v, starts, scale, causal):
    """``(o [R,H,D], lse [R,H])`` of rows cut into sequences at ``starts``; q [R,H,D], k, v [R,Hk,D]."""
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    o, lse = np.zeros_like(q), np.zeros(q.shape[:2])
    for a, b in zip(starts, starts[1:]):
        for h in range(H):
            P, lse[a:b, h] = weights(q[a:b, h], k[a:b, h // G], scale, causal)
            o[a:b, h] = P @ v[a:b, h // G]
    return o, lse


def attention_bwd(dO, q, k, v, starts, scale, causal):
    """Adjoint: ``(dq, dk, dv)``."""
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in zip(starts, starts[1:]):
        for h in range(H):
            g = h // G
            P, _ = weights(q[a:b, h], k[a:b, g], scale, causal)
            dP = dO[a:b, h] @ v[a:b, g].T
            dS = P * (dP - (P * dP).sum(-1, keepdims=True))
            dq[a:b, h] = scale * dS @ k[a:b, g]
            dk[a:b, g] += scale * dS.T @ q[a:b, h]
            dv[a:b, g] += P.T @ dO[a:b, h]
    return dq, dk, dv


def bounds(dO, q, k, v, starts, scale, causal, half=2.0 ** -8, tile=0):
    """How far results may lie from the exact ones when the weights and their gradients are rounded once to a type whose half step is
    ``half`` relative, outputs once more, and scores and products are fp32 sums of D terms in any order (each of at most D 2^-23 of
    the sum of their magnitudes): a dict of elementwise bounds for o, lse, dq, dk, dv. First-order in the roundings, plus 1% for the rest.

    The sum D of a row's weights times their gradients is taken from the rounded o, but from the weights themselves for the queries that
    see only the sequence's first ``tile`` keys by their place (its first ``tile`` queries if causal, all of it if it is no longer)."""
    D, H, G = q.shape[2], q.shape[1], q.shape[1] // k.shape[1]
    out = {"o": np.zeros_like(q), "lse": np.zeros(q.shape[:2]), "dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    exact = dict(zip(("o", "lse"), attention(q, k, v, starts, scale, causal)))
    exact.update(zip(("dq", "dk", "dv"), attention_bwd(dO, q, k, v, starts, scale, causal)))
    fp = 2.0 ** -23
    for a, b in zip(starts, starts[1:]):
        for h in range(H):
            g = h // G
            Q, K, V, O = q[a:b, h], k[a:b, g], v[a:b, g], dO[a:b, h]
            P, lse = weights(Q, K, scale, causal)
            S = scale * np.abs(Q) @ np.abs(K).T * (P > 0)
            # a score's error, the exponent's fp32 rounding (of the score and of the reference it is taken from), the exponential unit
            ds = (D * fp + 4 * fp) * S + 4 * fp * np.abs(lse)[:, None] + 8 * fp
            dl = (P * ds).sum(-1) + 16 * fp
            rel = ds + dl[:, None]                      # of a weight p / sum
            out["lse"][a:b, h] = dl + 4 * fp * np.abs(lse)
            eo = (P * (half + rel)) @ np.abs(V)
            out["o"][a:b, h] = eo
            eo = eo + half * np.abs(exact["o"][a:b, h])  # as it is read back
            dP = O @ V.T
            delta = (P * dP).sum(-1, keepdims=True)
            edelta = (np.abs(O) * eo).sum(-1, keepdims=True) + D * fp * (np.abs(O) * np.abs(exact["o"][a:b, h])).sum(-1, keepdims=True)
            own = np.arange(b - a) < (tile if causal or b - a <= tile else 0)
            # sum p dP / sum p: the weights' relative errors on dP - D, the products' errors, and at most `tile` + 8 roundings of the sums
            edelta[own] = ((P * rel * np.abs(dP - delta)).sum(-1, keepdims=True) + D * fp * (P * (np.abs(O) @ np.abs(V).T)).sum(-1, keepdims=True)
                           + (tile + 8) * fp * (P * np.abs(dP)).sum(-1, keepdims=True))[own]
            dS = np.abs(P * (dP - delta))
            edS = (half + rel) * dS + P * (D * fp * np.abs(O) @ np.abs(V).T + edelta + 2 * fp * (np.abs(dP) + np.abs(delta)))
            out["dq"][a:b, h] = scale * edS @ np.abs(K)
            out["dk"][a:b, g] += scale * edS.T @ np.abs(Q)
            out["dv"][a:b, g] += (P * (half + rel)).T @ np.abs(O)
    return exact, {n: 1.01 * e + (half * np.abs(exact[n]) if n != "lse" else 0.0) for n, e in out.items()}


def attention_step(q, k_cache, v_cache, page_table, lengths, scale):
    """q [B,H,D] over pages [pages,size,Hk,D]; rows of length 0 or less are zero."""
    B, H, _ = q.shape
    size, Hk = k_cache.shape[1:3]
    o = np.zeros_like(q)
    for b in range(B):
        n = int(lengths[b])
        if n <= 0:
            continue
        pages = page_table[b, : -(-n // size)]
        K, V = (c[pages].reshape(-1, Hk, c.shape[3])[:n] for c in (k_cache, v_cache))
        for h in range(H):
            g = h // (H // Hk)
            P, _ = weights(q[b, h][None], K[:, g], scale, False)
            o[b, h] = (P @ V[:, g])[0]
    return o

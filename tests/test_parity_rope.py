"""Norm and rotation of query and key heads against their fp64 definitions (GPU).

Tolerances: a bf16 result is rounded once (half a step, 2^-8 relative); the sine and cosine are within 2^-20 (the unit's 2^-20.9 and the
angle's rounding to fp32 at up to half a turn), which counts with the pair's size; fp32 norms within 1e-5 of the terms."""
import numpy as np
import pytest
import torch

from _util import f64, rel_l2
from oracle import attention as A

pytestmark = pytest.mark.gpu
I32 = torch.int32


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def rn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def freqs(rotary, theta=1e4):
    return None if rotary == 0 else (1 / theta ** (torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)).float().cuda()


def rows(t):
    return f64(t).reshape(-1, *t.shape[-2:])


def close(name, got, want, terms):
    x = f64(got).reshape(want.shape)
    size = np.abs(terms).max(-1, keepdims=True)
    over = np.abs(x - want) - (2.0 ** -8 * np.abs(want) + (2.0 ** -18 + 1e-5) * size)
    assert np.isfinite(x).all() and over.max() <= 0, f"{name}: off by {over.max():.3e} more than allowed"


def position_list(B, T, cu):
    starts = [b * T for b in range(B + 1)] if cu is None else cu
    return np.concatenate([np.arange(b - a) for a, b in zip(starts, starts[1:])])


def check(B, T, H, Hk, D, rotary, cu=None, positions=None, inter=False, norm=True, eps=1e-6, backward=True):
    g = torch.Generator().manual_seed(T * 11 + H + D + rotary)
    q, k = rn(g, B, T, H, D), rn(g, B, T, Hk, D)
    qw, kw = (1 + rn(g, D, dtype=torch.float32, std=0.2) for _ in range(2)) if norm else (None, None)
    f = freqs(rotary)
    kwargs = dict(positions=positions, cu_seqlens=cu, eps=eps, interleaved=inter)
    got = lib().qk_norm_rope_fwd(q, k, qw, kw, f, **kwargs)
    pos = position_list(B, T, cu) if positions is None else positions.flatten().tolist()
    freq = np.zeros(0) if f is None else f64(f)
    dy = [rn(g, *t.shape) for t in (q, k)]
    grads = lib().qk_norm_rope_bwd(*dy, q, k, qw, kw, f, **kwargs) if backward else None
    for i, (x, w) in enumerate(((q, qw), (k, kw))):
        y, n = A.norm_rope(rows(x), None if w is None else f64(w), pos, freq, eps, inter)
        close("qk"[i], got[i], y, n)
        if backward:
            dx, dw, terms = A.norm_rope_bwd(rows(dy[i]), rows(x), None if w is None else f64(w), pos, freq, eps, inter)
            close("d" + "qk"[i], grads[i], dx, terms)
            if norm:
                assert rel_l2(f64(grads[2 + i]), dw) <= 1e-5
            else:
                assert grads[2 + i] is None


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rotary", [(128, 128), (128, 64), (128, 96), (128, 16), (128, 0), (64, 64), (64, 32), (64, 48), (64, 16)])
def test_widths(D, rotary, inter):
    check(2, 37, 3, 1, D, rotary, inter=inter)


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1), (5, 5), (7, 1), (16, 4), (40, 8), (9, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(H, Hk, D):
    check(1, 9, H, Hk, D, D)


@pytest.mark.parametrize("B,T", [(1, 1), (5, 1), (1, 2), (1, 2500), (3, 700)])
def test_rows(B, T):
    check(B, T, 4, 2, 128, 64)


@pytest.mark.parametrize("cu", [[0, 1], [0, 1, 2, 40], [0, 30, 100, 101]])
def test_documents(cu):
    check(1, cu[-1], 4, 2, 128, 128, cu=cu)


def test_no_norm():
    check(1, 50, 4, 2, 128, 128, norm=False)


def test_large_eps():
    check(1, 20, 2, 1, 64, 64, eps=0.5)


@pytest.mark.parametrize("D", [64, 128])
def test_no_eps(D):
    """Heads that do not fill a warp leave lanes without one, whose zeros have no finite norm."""
    check(1, 20, 7, 1, D, 64, eps=0.0)


@pytest.mark.parametrize("inter", [False, True])
def test_positions_far_away(inter):
    """The same precision at any position, negative ones among them."""
    pos = torch.tensor([[0, 1, 1023, 8191, 131071, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -1, -77777, -(1 << 31)]], dtype=I32).cuda()
    check(1, pos.shape[1], 2, 1, 128, 128, positions=pos, inter=inter)


@pytest.mark.parametrize("f", [0.0, 1.0, 6.2831855, 100.0, 3e7, 1e-7, 1e-30, 1e-42, -0.7])
def test_any_frequency(f):
    """One frequency for all pairs against its exact turn."""
    q = torch.ones(1, 300, 1, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.full((32,), f, dtype=torch.float32, device="cuda")
    y, _ = lib().qk_norm_rope_fwd(q, q, None, None, inv)
    want = A.turn(rows(q), np.arange(300), f64(inv), False)
    assert np.abs(rows(y) - want).max() <= 2.0 ** -8 * 1.42 + 2.0 ** -18


def test_strided_inputs():
    g = torch.Generator().manual_seed(1)
    mixed = rn(g, 2, 21, 5 * 128 + 8)
    q, k = mixed[..., 8: 8 + 4 * 128].unflatten(-1, (4, 128)), mixed[..., 8 + 4 * 128:].unflatten(-1, (1, 128))
    w, f = 1 + rn(g, 128, dtype=torch.float32, std=0.1), freqs(128)
    dy = [rn(g, *t.shape) for t in (q, k)]
    a = (*lib().qk_norm_rope_fwd(q, k, w, w, f), *lib().qk_norm_rope_bwd(*dy, q, k, w, w, f))
    q, k = q.contiguous(), k.contiguous()
    for x, y in zip(a, (*lib().qk_norm_rope_fwd(q, k, w, w, f), *lib().qk_norm_rope_bwd(*dy, q, k, w, w, f))):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ into the cache

def store_case(lengths, new, H, Hk, D, page, seed=0, extra=2):
    """Sequences of ``lengths`` tokens whose last ``new`` ones are stored."""
    g = torch.Generator().manual_seed(seed + page + sum(new))
    R = sum(new)
    q, k, v = rn(g, 1, R, H, D), rn(g, 1, R, Hk, D), rn(g, 1, R, Hk, D)
    need = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).to(I32)
    table = torch.full((len(lengths), max(1, max(need)) + 1), -1, dtype=I32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at: at + n]
        at += n
    kc, vc = rn(g, pages, page, Hk, D), rn(g, pages, page, Hk, D)
    w = 1 + rn(g, D, dtype=torch.float32, std=0.1)
    return q, k, v, w, freqs(D), kc, vc, table.cuda(), torch.tensor(lengths, dtype=I32).cuda()


def check_store(lengths, new, H, Hk, D, page, single=False):
    q, k, v, w, f, kc, vc, table, n = store_case(lengths, new, H, Hk, D, page)
    kc0, vc0 = kc.clone(), vc.clone()
    status = torch.zeros(1, dtype=I32, device="cuda")
    cu = None if single else np.concatenate([[0], np.cumsum(new)]).tolist()
    args = [t[0] for t in (q, k, v)] if single else [q, k, v]
    qo, ko = lib().qk_norm_rope_store(*args, w, w, f, kc, vc, table, n, cu_seqlens=None if single else [int(x) for x in cu], status=status)
    assert int(status.item()) == 0
    # the outputs are the forward's at those positions
    pos = np.concatenate([np.arange(a - b, a) if a > 0 else np.zeros(b) for a, b in zip(lengths, new)])
    qf, kf = lib().qk_norm_rope_fwd(q, k, w, w, f, positions=torch.tensor(pos, dtype=I32).view(1, -1).cuda())
    row = 0
    for i, (a, b) in enumerate(zip(lengths, new)):
        for t in range(b):
            if a <= 0:
                qf[0, row], kf[0, row] = 0, 0
            else:
                p = a - b + t
                kc0[table[i, p // page], p % page], vc0[table[i, p // page], p % page] = kf[0, row], v[0, row]
            row += 1
    assert torch.equal(qo.reshape(qf.shape), qf) and torch.equal(ko.reshape(kf.shape), kf)
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)      # everything else as it was


@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_store_single_tokens(page):
    check_store([1, 2, 16, 17, 0, 63, 64, 65, -1, 200], [1] * 10, 4, 2, 128, page, single=True)


@pytest.mark.parametrize("page", [7, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_store_prompts(page, D):
    check_store([3, 80, 0, 130, 41], [3, 70, 2, 130, 1], 5, 1, D, page)


def test_store_dense_prompts():
    q, k, v, w, f, kc, vc, table, n = store_case([9, 9, 9], [9, 9, 9], 4, 2, 128, 4)
    kc2, vc2 = kc.clone(), vc.clone()
    a = lib().qk_norm_rope_store(q, k, v, w, w, f, kc, vc, table, n, cu_seqlens=[0, 9, 18, 27])
    b = lib().qk_norm_rope_store(*(t.view(3, 9, *t.shape[2:]) for t in (q, k, v)), w, w, f, kc2, vc2, table, n)
    assert torch.equal(a[0].view(-1), b[0].view(-1)) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_store_reports_bad_places():
    from chunked_gated_delta_05_gb300 import GDN_ERANGE
    for what in ("page", "negative", "table", "short"):
        q, k, v, w, f, kc, vc, table, n = store_case([20, 20, 20], [1, 1, 1], 4, 2, 128, 8)
        if what == "short":
            q, k, v, w, f, kc, vc, table, n = store_case([20, 20, 20], [3, 3, 3], 4, 2, 128, 8)
            n[1] = 2
        elif what == "table":
            n[1] = 8 * table.shape[1] + 1
        else:
            table[1, 2] = kc.shape[0] if what == "page" else -5
        new = q.shape[1] // 3
        kc0, vc0, st = kc.clone(), vc.clone(), torch.zeros(1, dtype=I32, device="cuda")
        shape = lambda t: t.view(3, new, *t.shape[2:])  # noqa: E731
        qo, ko = lib().qk_norm_rope_store(shape(q), shape(k), shape(v), w, w, f, kc, vc, table, n, status=st)
        assert int(st.item()) == GDN_ERANGE, what
        assert not qo[1].any() and not ko[1].any() and qo[0].any() and qo[2].any()
        changed = (kc != kc0).flatten(2).any(-1)
        assert int(changed.sum()) == 2 * new, what     # the other two sequences' rows

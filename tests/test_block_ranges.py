"""The operators around the recurrence at the ends of their ranges: the scan's plan (CPU), rows of large and small values, steps of
size zero, and parameters at odd addresses (GPU). Tolerances are those of the operators' other tests."""
import ctypes

import numpy as np
import pytest
import torch

from _util import f64, rel_l2
from chunked_gated_delta_05_gb300 import _lib
from oracle import block


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


# ------------------------------------------------------------------ the scan's plan, as the sizes show it (CPU)

def sizes(B, T, D, N, G=1, docs=None):
    d = _lib.SscanDesc(B=B, T=T, D=D, N=N, G=G, num_seqs=B, delta_softplus=1)
    if docs:
        keep = (ctypes.c_int32 * len(docs))(*docs)
        d.cu_seqlens, d.num_seqs = ctypes.cast(keep, ctypes.POINTER(ctypes.c_int32)), len(docs) - 1
    L = _lib.load()
    return tuple(getattr(L, f"gdn_sscan_{k}")(ctypes.byref(d)) for k in ("fwd_workspace_size", "saved_size", "bwd_workspace_size"))


def up(n):
    return (n + 255) // 256 * 256


def segments(fwd, D, N, tables):
    """Segments of a forward whose workspace holds the tables, a state and a step sum a segment and channel; 0 if it is not cut."""
    rest = fwd - up(tables)
    n = 0
    while n * D * (N + 1) * 4 <= rest:
        if up(n * N * D * 4) + up(n * D * 4) == rest:
            return n
        n += 1
    raise AssertionError("no whole number of segments")


@pytest.mark.parametrize("B,T,D,N,docs", [(1, 8192, 4096, 16, None), (1, 8192, 64, 16, None), (3, 1000, 200, 13, None), (1, 4093, 2048, 16, [0, 1, 700, 4093]),
                                          (1, 300, 128, 4, [0, 299, 300]), (1, 31, 64, 16, None), (1, 33, 64, 16, None), (64, 1, 4096, 16, None)])
def test_plan_covers_every_sequence(B, T, D, N, docs):
    fwd, saved, bwd = sizes(B, T, D, N, docs=docs)
    lengths = [b - a for a, b in zip(docs, docs[1:])] if docs else [T] * B
    assert saved == up(sum((n + 7) // 8 for n in lengths) * N * D * 4)      # a state before every 8th token
    n = segments(fwd, D, N, len(docs) * 3 * 4 if docs else 4)
    assert n == 0 or len(lengths) < n <= sum((x + 31) // 32 for x in lengths)
    assert bwd >= fwd + saved


def test_plan_cuts_few_sequences_and_leaves_many_whole():
    assert segments(sizes(1, 8192, 4096, 16)[0], 4096, 16, 4) > 1
    assert segments(sizes(256, 128, 4096, 16)[0], 4096, 16, 4) == 0
    assert segments(sizes(1, 32, 4096, 16)[0], 4096, 16, 4) == 0      # a shortest segment


# ------------------------------------------------------------------ on the device

def close_bf16(x, ref):
    x = f64(x)
    assert np.isfinite(x).all()
    bad = np.abs(x - ref) - (2.0 ** -8 * np.abs(ref) + 1e-5 * np.abs(ref).max())
    assert bad.max() <= 0, f"off by {bad.max():.3e} more than allowed"


def rng(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dtype=torch.bfloat16, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("width", [100, 2048, 8192])
@pytest.mark.parametrize("size", [1e-15, 1e-4, 1e6, 1e15])
def test_norms_of_large_and_small_rows(width, size):
    """Squares of 1e15 sum to 1e34 at most, in fp32's range; of rows under 1e-4 eps is most of the mean."""
    rn = rng(width)
    x, gate, dy, w = rn(5, width, std=size), rn(5, width), rn(5, width), 1 + rn(width, dtype=torch.float32, std=0.1)
    m = lib()
    close_bf16(m.gated_rms_norm_fwd(x, gate, w, eps=1e-5), block.gated_norm(f64(x), f64(gate), f64(w), 1e-5, "silu"))
    for got, want in zip(m.gated_rms_norm_bwd(x, gate, w, dy, eps=1e-5), block.gated_norm_bwd(f64(x), f64(gate), f64(w), f64(dy), 1e-5, "silu")):
        close_bf16(got, want) if got.dtype is torch.bfloat16 else None
        assert rel_l2(f64(got), want) <= (1e-5 if got.dtype is torch.float32 else 2.0 ** -8)
    res = rn(5, width, dtype=torch.float32, std=size)
    y, stream = m.add_rms_norm_fwd(x, res, w, eps=1e-5, residual_scale=0.7)
    want, r = block.add_norm(f64(x), f64(res), f64(w), 1e-5, 0.7)
    close_bf16(y, want)
    assert rel_l2(f64(stream), r) <= 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(1, 3000), (200, 40)])
def test_steps_of_size_zero_leave_the_state(B, T):
    """delta = 0 without softplus, cut into segments and whole: the state stays bit for bit, and so do its gradients' paths."""
    rn = rng(T)
    D, N = 64, 16
    u, dy, Bm, Cm, zero = rn(B, T, D), rn(B, T, D), rn(B, T, 1, N), rn(B, T, 1, N), torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda")
    A, Ds, h0, dfinal = -torch.exp(rn(D, N, dtype=torch.float32)), rn(D, dtype=torch.float32), rn(B, D, N, dtype=torch.float32), rn(B, D, N, dtype=torch.float32)
    m, kw = lib(), dict(D=Ds, delta_softplus=False, initial_state=h0)
    y, final = m.selective_scan_fwd(u, zero, A, Bm, Cm, output_final_state=True, **kw)
    assert torch.equal(final, h0)
    close_bf16(y, np.einsum("bdn,btn->btd", f64(h0), f64(Cm)[:, :, 0]) + f64(Ds) * f64(u))
    du, _, dA, dB, dC, dD, _, _, dh0 = m.selective_scan_bwd(u, zero, A, Bm, Cm, dy, dfinal=dfinal, **kw)
    close_bf16(du, f64(Ds) * f64(dy))
    assert (dA == 0).all() and (dB == 0).all()
    want = np.einsum("btd,bdn->btn", f64(dy), f64(h0))
    assert rel_l2(f64(dC)[:, :, 0], want) <= 2.0 ** -8
    assert rel_l2(f64(dh0), f64(dfinal) + np.einsum("btd,btn->bdn", f64(dy), f64(Cm)[:, :, 0])) <= 1e-5
    assert rel_l2(f64(dD), (f64(dy) * f64(u)).sum((0, 1))) <= 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 16])
def test_scan_step_takes_A_at_any_address(N):
    rn = rng(N)
    B, D = 5, 72
    u, z, Bm, Cm, state, A = rn(B, D), rn(B, D), rn(B, 1, N), rn(B, 1, N), rn(B, D, N, dtype=torch.float32), -torch.exp(rn(D, N, dtype=torch.float32))
    odd = torch.empty(D * N + 1, device="cuda")[1:].view(D, N).copy_(A)
    outs = []
    for a in (A, odd):
        s = state.clone()
        outs.append((lib().selective_scan_step(s, u, u, a, Bm, Cm, z=z), s))
    assert all(torch.equal(p, q) for p, q in zip(*outs))

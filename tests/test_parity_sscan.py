"""Selective scan against its fp64 definition (GPU).

Tolerances: y, du, ddelta and dz are one bf16 rounding (2^-8) of fp32 values whose recurrences of up
to some hundred tokens are within 1e-4 of the result's largest value; final states, dA, dD, ddelta_bias and dh0 are fp32, within
1e-5 rel-L2; dB and dC sum tf32 products (2^-11 each) over the channels and are rounded to bf16: rel-L2 4e-3."""
import numpy as np
import pytest
import torch

from _util import f64, rel_l2
from oracle import block

pytestmark = pytest.mark.gpu


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def make(B, T, D, N, G=1, docs=None, z=True, skip=True, bias=True, softplus=True, h0=False, strided=False, seed=0, dt=(1e-3, 0.1)):
    g = torch.Generator().manual_seed(seed * 1009 + B * 31 + T * 7 + D * 3 + N)

    def rn(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()

    step = torch.exp(torch.rand(D, generator=g) * np.log(dt[1] / dt[0]) + np.log(dt[0])).cuda()
    s = len(docs) - 1 if docs else B
    c = {"u": rn(B, T, D), "A": -torch.exp(rn(D, N, dtype=torch.float32, std=0.5)) * 4, "B": rn(B, T, G, N), "C": rn(B, T, G, N)}
    if softplus:
        c["delta"] = rn(B, T, D, std=0.5)
        c["delta_bias"] = (step + torch.log(-torch.expm1(-step))) if bias else None
    else:
        c["delta"] = (step * torch.exp(rn(B, T, D, dtype=torch.float32, std=0.5))).to(torch.bfloat16)
        c["delta_bias"] = step.clone() if bias else None
    c["D"] = rn(D, dtype=torch.float32) if skip else None
    c["z"] = rn(B, T, D) if z else None
    c["initial_state"] = rn(s, D, N, dtype=torch.float32) if h0 else None
    if strided:     # rows of wider projections
        for k, pad in (("u", 8), ("delta", 16), ("z", D), ("B", 5), ("C", 24)):
            if c[k] is not None:
                t = c[k]
                flat = t.reshape(B, T, -1)
                wide = rn(B, T, flat.shape[-1] + pad)
                wide[..., pad:] = flat
                c[k] = wide[..., pad:].view(t.shape)
                assert not c[k].is_contiguous() or B * T == 1
    c["cfg"] = dict(delta_softplus=softplus, cu_seqlens=docs)
    c["dy"] = rn(B, T, D)
    c["dfinal"] = rn(s, D, N, dtype=torch.float32)
    return c


def kwargs(c):
    return dict(D=c["D"], z=c["z"], delta_bias=c["delta_bias"], initial_state=c["initial_state"], **c["cfg"])


def reference(c, with_final=True):
    B, T, D = c["u"].shape
    flat = {k: (None if c[k] is None else f64(c[k]).reshape(B * T, *c[k].shape[2:])) for k in ("u", "delta", "B", "C", "z", "dy")}
    par = {k: None if c[k] is None else f64(c[k]) for k in ("A", "D", "delta_bias")}
    starts = c["cfg"]["cu_seqlens"] or [b * T for b in range(B + 1)]
    kw = dict(D=par["D"], z=flat["z"], delta_bias=par["delta_bias"], softplus=c["cfg"]["delta_softplus"],
              h0=None if c["initial_state"] is None else f64(c["initial_state"]), starts=starts)
    args = (flat["u"], flat["delta"], par["A"], flat["B"], flat["C"])
    y, final, _ = block.scan(*args, **kw)
    return y.reshape(B, T, D), final, block.scan_bwd(*args, flat["dy"], dfinal=f64(c["dfinal"]) if with_final else None, **kw)


def close_bf16(name, x, ref):
    x = f64(x).reshape(ref.shape)
    assert np.isfinite(x).all(), name
    bad = np.abs(x - ref) - (2.0 ** -8 * np.abs(ref) + 1e-4 * np.abs(ref).max())
    assert bad.max() <= 0, f"{name}: off by {bad.max():.3e} more than allowed"


def close_f32(name, x, ref):
    assert rel_l2(f64(x), ref) <= 1e-5, f"{name}: {rel_l2(f64(x), ref):.2e}"


def check(c):
    m = lib()
    args = (c["u"], c["delta"], c["A"], c["B"], c["C"])
    y, final, saved = m.selective_scan_fwd(*args, output_final_state=True, save=True, **kwargs(c))
    ry, rf, g = reference(c)
    close_bf16("y", y, ry)
    close_f32("final", final, rf)
    grads = m.selective_scan_bwd(*args, c["dy"], dfinal=c["dfinal"], saved=saved, **kwargs(c))
    again = m.selective_scan_bwd(*args, c["dy"], dfinal=c["dfinal"], **kwargs(c))
    names = ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dh0")
    for name, a, b in zip(names, grads, again):
        src = {"ddelta_bias": "delta_bias", "dh0": "initial_state"}.get(name, name[1:])
        if c[src] is None:
            assert a is None, name
            continue
        assert torch.equal(a, b), f"{name}: the kept states and the recomputed ones differ"
        assert a.shape == c[src].shape and a.is_contiguous()
        if name in ("dB", "dC"):
            assert rel_l2(f64(a).reshape(g[name].shape), g[name]) <= 4e-3, name
        elif a.dtype == torch.float32:
            close_f32(name, a, g[name])
        else:
            close_bf16(name, a, g[name])


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 33, 63, 64, 65, 100, 300])
def test_lengths(T):
    check(make(2, T, 40, 16, h0=True))


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 13, 15, 16])
def test_states(N):
    check(make(1, 70, 48, N, h0=True, seed=1))


@pytest.mark.parametrize("D,G", [(1, 1), (2, 1), (7, 1), (8, 1), (127, 1), (128, 1), (129, 1), (130, 1), (136, 1), (256, 2), (258, 2), (260, 4), (393, 3)])
def test_channels_and_groups(D, G):
    check(make(1, 75, D, 16, G=G, h0=True, seed=2))


@pytest.mark.parametrize("kw", [dict(z=False), dict(skip=False), dict(bias=False), dict(softplus=False), dict(softplus=False, bias=False),
                                dict(z=False, skip=False, bias=False), dict(h0=True, z=False)])
def test_optional_inputs(kw):
    check(make(2, 90, 64, 16, seed=3, **kw))


@pytest.mark.parametrize("docs", [[0, 1], [0, 1, 2, 3], [0, 5, 6, 90, 91, 300], [0, 64, 128, 320], [0, 300], list(range(0, 260, 2)) + [300]])
def test_packed_documents(docs):
    check(make(1, docs[-1], 72, 16, docs=docs, h0=True, seed=4))


@pytest.mark.parametrize("D,N,G", [(64, 16, 1), (66, 13, 2), (33, 8, 1)])
def test_strided_rows(D, N, G):
    check(make(2, 70, D, N, G=G, strided=True, h0=True, seed=5))


def test_unaligned_base_addresses():
    c = make(1, 70, 64, 16, seed=6)
    for k in ("u", "delta", "z", "dy", "B", "C"):
        t = c[k]
        c[k] = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    check(c)


@pytest.mark.parametrize("dt", [(1e-5, 1e-4), (0.5, 4.0)])
def test_slow_and_fast_decays(dt):
    check(make(1, 200, 32, 16, h0=True, seed=7, dt=dt))


def test_whole_and_cut_sequences_agree():
    """Enough sequences are walked whole, one alone is cut into segments: the same values either way."""
    c = make(160, 130, 128, 16, seed=8)
    args = (c["u"], c["delta"], c["A"], c["B"], c["C"])
    y, final = lib().selective_scan_fwd(*args, output_final_state=True, **kwargs(c))
    grads = lib().selective_scan_bwd(*args, c["dy"], dfinal=c["dfinal"], **kwargs(c))
    for b in (0, 159):
        one = {k: (v[b:b + 1].contiguous() if k in ("u", "delta", "B", "C", "z") else v) for k, v in c.items()}
        a1 = (one["u"], one["delta"], c["A"], one["B"], one["C"])
        y1, f1 = lib().selective_scan_fwd(*a1, output_final_state=True, **kwargs(one))
        g1 = lib().selective_scan_bwd(*a1, c["dy"][b:b + 1].contiguous(), dfinal=c["dfinal"][b:b + 1].contiguous(), **kwargs(one))
        assert rel_l2(f64(final[b:b + 1]), f64(f1)) <= 1e-5
        assert rel_l2(f64(y[b:b + 1]), f64(y1)) <= 1e-3
        for i in (0, 1, 3, 4, 6):      # du, ddelta, dB, dC, dz of that sequence
            assert rel_l2(f64(grads[i][b:b + 1]), f64(g1[i])) <= 1e-3


def test_nan_stays_in_its_document_and_channel():
    docs = [0, 70, 150]
    c = make(1, 150, 64, 16, docs=docs, seed=9)
    args = [c["u"], c["delta"], c["A"], c["B"], c["C"]]
    y0, f0 = lib().selective_scan_fwd(*args, output_final_state=True, **kwargs(c))
    c["u"][0, 10, 5] = float("nan")
    y, f = lib().selective_scan_fwd(*args, output_final_state=True, **kwargs(c))
    assert y[0, 10:70, 5].isnan().all() and f[0, 5].isnan().all()
    y[0, 10:70, 5], f[0, 5] = y0[0, 10:70, 5], f0[0, 5]
    assert torch.equal(y, y0) and torch.equal(f, f0)


def test_gradients_against_differences():
    """Directional differences of <dfinal, final> (fp32) in A, delta_bias and the initial state; central differences with
    relative steps of 1e-2 leave their third derivatives' 1e-4, and 1e-3 is allowed."""
    c = make(1, 120, 32, 16, h0=True, seed=10)
    args = [c["u"], c["delta"], c["A"], c["B"], c["C"]]
    kw = kwargs(c)
    zero = torch.zeros_like(c["dy"])
    g = lib().selective_scan_bwd(*args, zero, dfinal=c["dfinal"], **kw)

    def loss(A, bias, h0):
        f = lib().selective_scan_fwd(args[0], args[1], A, args[3], args[4], output_final_state=True, **{**kw, "delta_bias": bias, "initial_state": h0})[1]
        return (f.double() * c["dfinal"].double()).sum().item()

    base = [c["A"], c["delta_bias"], c["initial_state"]]
    for i, grad in ((0, g[2]), (1, g[7]), (2, g[8])):
        d = 1e-2 * base[i].abs() * grad.sign()
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + d, base[i] - d
        want = 2 * (grad.double() * d.double()).sum().item()
        assert abs(loss(*up) - loss(*down) - want) <= 1e-3 * abs(want), i


def test_autograd_and_side_stream():
    c = make(2, 70, 48, 16, G=2, h0=True, seed=11)
    names = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "initial_state")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        leaf = {k: c[k].clone().requires_grad_() for k in names}
        y, final = lib().selective_scan(leaf["u"], leaf["delta"], leaf["A"], leaf["B"], leaf["C"], D=leaf["D"], z=leaf["z"], delta_bias=leaf["delta_bias"],
                                        initial_state=leaf["initial_state"], output_final_state=True)
        torch.autograd.backward([y, final], [c["dy"], c["dfinal"]])
    torch.cuda.current_stream().wait_stream(s)
    want = lib().selective_scan_bwd(c["u"], c["delta"], c["A"], c["B"], c["C"], c["dy"], dfinal=c["dfinal"], **kwargs(c))
    for k, w in zip(("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "initial_state"), want):
        assert torch.equal(leaf[k].grad, w), k


def test_graph_capture():
    c = make(1, 200, 64, 16, seed=12)
    args = (c["u"], c["delta"], c["A"], c["B"], c["C"])
    want = lib().selective_scan_fwd(*args, output_final_state=True, **kwargs(c))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib().selective_scan_fwd(*args, output_final_state=True, **kwargs(c))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    c = make(1, 20, 16, 8, seed=13)
    m = lib()

    def call(**kw):
        x = {**c, **kw}
        cfg = {**c["cfg"], **kw.get("cfg", {})}
        return m.selective_scan_fwd(x["u"], x["delta"], x["A"], x["B"], x["C"], D=x["D"], z=x["z"], delta_bias=x["delta_bias"],
                                    initial_state=x["initial_state"], **cfg)

    call()
    h = torch.zeros(1, 16, 8, device="cuda")
    for kw in (dict(u=c["u"].float()), dict(delta=c["delta"][:, :10]), dict(A=c["A"].double()), dict(A=torch.zeros(16, 17, device="cuda"),
               B=torch.zeros(1, 20, 1, 17, dtype=torch.bfloat16, device="cuda"), C=torch.zeros(1, 20, 1, 17, dtype=torch.bfloat16, device="cuda")),
               dict(B=c["B"].expand(1, 20, 3, 8).contiguous(), C=c["C"].expand(1, 20, 3, 8).contiguous()), dict(C=c["C"][..., :4]),
               dict(z=c["z"].transpose(1, 2)), dict(u=c["u"][:, :, :1].expand(1, 20, 16)), dict(D=c["D"].half()), dict(initial_state=h[:, :8]),
               dict(cfg=dict(cu_seqlens=[0, 21])), dict(cfg=dict(cu_seqlens=[0, 5, 5, 20])), dict(delta=c["delta"].cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        m.selective_scan_bwd(c["u"], c["delta"], c["A"], c["B"], c["C"], c["dy"], saved=torch.zeros(8, dtype=torch.uint8, device="cuda"), **kwargs(c))


def test_without_gradients_is_the_forward():
    u, delta, A, B, C = (t.cuda() for t in (torch.randn(1, 21, 40).bfloat16(), torch.randn(1, 21, 40).bfloat16(), -torch.rand(40, 8) - 0.1,
                                             torch.randn(1, 21, 1, 8).bfloat16(), torch.randn(1, 21, 1, 8).bfloat16()))
    want, final = lib().selective_scan_fwd(u, delta, A, B, C, output_final_state=True)
    A.requires_grad_(True)
    with torch.no_grad():
        y, h = lib().selective_scan(u, delta, A, B, C, output_final_state=True)
    assert y.grad_fn is None and torch.equal(y, want) and torch.equal(h, final)
    y, h = lib().selective_scan(u, delta, A, B, C, output_final_state=True)
    assert y.grad_fn is not None and torch.equal(y, want) and torch.equal(h, final)

"""Norms before and after a block against their fp64 definitions (GPU).

Tolerances: a bf16 result is one rounding (at most 2^-8 of its value, the unit roundoff of 8 significant bits) of an fp32
evaluation of a few dozen roundings, at most 1e-5 of the result's largest value; dx is a difference of two terms, which cancel
entirely at width 1 (dx = dy w eps rstd^3), so it may also be off by four fp32 roundings (2^-22) of the terms; fp32 results (the stream, weight gradients over the rows) are within
1e-5 rel-L2 (fp32 sums of up to some thousand terms)."""
import numpy as np
import pytest
import torch

from _util import f64, rel_l2
from oracle import block

pytestmark = pytest.mark.gpu

WIDTHS = [1, 7, 8, 24, 64, 100, 128, 250, 1000, 2048, 2056, 4100, 4104, 8200, 16384]


def lib():
    import chunked_gated_delta_05_gb300 as m
    return m


def rn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close_bf16(name, x, ref, terms=0.0):
    x = f64(x)
    assert np.isfinite(x).all(), name
    bad = np.abs(x - ref) - (2.0 ** -8 * np.abs(ref) + 1e-5 * np.abs(ref).max() + 2.0 ** -22 * np.abs(terms).max())
    assert bad.max() <= 0, f"{name}: off by {bad.max():.3e} more than allowed"


def close_f32(name, x, ref):
    assert rel_l2(f64(x), ref) <= 1e-5, f"{name}: {rel_l2(f64(x), ref):.2e}"


def round_like(kind):
    return lambda r: torch.from_numpy(r).to(kind).double().numpy()


def close_stream(x, ref, kind):
    close_f32("stream", x, ref) if kind is torch.float32 else close_bf16("stream", x, ref)


@pytest.mark.parametrize("kind", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", [(r, w) for w in WIDTHS for r in ((1, 37) if w < 4000 else (3,))])
def test_add_norm(rows, width, kind):
    g = gen(rows * 100003 + width)
    x, w = rn(g, rows, width), 1 + rn(g, width, dtype=torch.float32, std=0.1)
    res = None if kind is None else rn(g, rows, width, dtype=kind, std=2.0)
    scale = 1.0 if kind is None else 0.7
    y, stream = lib().add_rms_norm_fwd(x, res, w, eps=1e-5, residual_scale=scale)
    keep = f64(stream)
    if kind is not None:
        assert stream.dtype == kind
        close_stream(stream, f64(res) + scale * f64(x), kind)
    ry, _ = block.add_norm(keep, None, f64(w), 1e-5, 1.0)     # of the stream as it is kept
    close_bf16("y", y, ry)
    dy, ds = rn(g, rows, width), rn(g, rows, width, dtype=kind or torch.bfloat16)
    for d in (ds, None):
        dx, dres, dw = lib().add_rms_norm_bwd(dy, d, stream, w, eps=1e-5, residual_scale=scale, has_residual=kind is not None)
        rx, rr, rw = block.add_norm_bwd(f64(dy), None if d is None else f64(d), keep, f64(w), 1e-5, scale)
        rstd = 1 / np.sqrt((keep * keep).mean(-1, keepdims=True) + 1e-5)
        close_bf16("dx", dx, rx, scale * rstd * f64(dy) * f64(w))
        close_f32("dweight", dw, rw)
        if kind is None:
            assert dres is None
        else:
            assert dres.dtype == kind
            close_stream(dres, rr, kind) if width > 1 or d is not None else None


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("rows,width", [(r, w) for w in WIDTHS for r in ((1, 37) if w < 4000 else (3,))] + [(5000, 128), (3001, 24)])
def test_gated_norm(rows, width, act):
    g = gen(rows * 7 + width)
    x, gate, w, dy = rn(g, rows, width), rn(g, rows, width), 1 + rn(g, width, dtype=torch.float32, std=0.1), rn(g, rows, width)
    y = lib().gated_rms_norm_fwd(x, gate, w, eps=1e-5, activation=act)
    close_bf16("y", y, block.gated_norm(f64(x), f64(gate), f64(w), 1e-5, act))
    dx, dg, dw = lib().gated_rms_norm_bwd(x, gate, w, dy, eps=1e-5, activation=act)
    rx, rg, rw = block.gated_norm_bwd(f64(x), f64(gate), f64(w), f64(dy), 1e-5, act)
    close_bf16("dx", dx, rx)
    close_bf16("dgate", dg, rg)
    close_f32("dweight", dw, rw)


def shifted(t):
    """The same values at an address that is no multiple of 16 bytes."""
    return torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape).copy_(t)


@pytest.mark.parametrize("width", [64, 2048, 8192])
def test_unaligned_tensors_give_the_same(width):
    g = gen(width)
    x, gate, w, dy = rn(g, 9, width), rn(g, 9, width), rn(g, width, dtype=torch.float32), rn(g, 9, width)
    for a, b in zip(lib().gated_rms_norm_bwd(x, gate, w, dy), lib().gated_rms_norm_bwd(shifted(x), shifted(gate), w, shifted(dy))):
        assert rel_l2(f64(a), f64(b)) <= 1e-3      # another order of the same fp32 sums: a bf16 rounding here and there
    assert rel_l2(f64(lib().gated_rms_norm_fwd(x, gate, w)), f64(lib().gated_rms_norm_fwd(shifted(x), shifted(gate), w))) <= 1e-3


def test_leading_dimensions_zero_rows_and_nan_rows():
    g = gen(5)
    x, gate, w = rn(g, 2, 3, 5, 128), rn(g, 2, 3, 5, 128), torch.ones(128, device="cuda")
    x[0, 0, 0] = 0
    clean = lib().gated_rms_norm_fwd(x, gate, w)
    assert clean.shape == x.shape and (clean[0, 0, 0] == 0).all()
    x[1, 2, 4] = float("nan")
    y = lib().gated_rms_norm_fwd(x, gate, w)
    assert y[1, 2, 4].isnan().all()
    y[1, 2, 4] = clean[1, 2, 4]
    assert torch.equal(y, clean)
    inf = x.clone()
    inf[1, 2, 4] = 0
    gate[0, 1, 2] = float("-inf")       # the gate shuts: sigmoid gives 0
    assert (lib().gated_rms_norm_fwd(inf, gate, w, activation="sigmoid")[0, 1, 2] == 0).all()


def test_repeated_backwards_agree_bit_for_bit():
    g = gen(6)
    x, gate, w, dy = rn(g, 9001, 128), rn(g, 9001, 128), rn(g, 128, dtype=torch.float32), rn(g, 9001, 128)
    for a, b in zip(lib().gated_rms_norm_bwd(x, gate, w, dy), lib().gated_rms_norm_bwd(x, gate, w, dy)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    rows, width = 270000, 8192        # 2.2 G elements
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    gate = torch.zeros_like(x)
    x[-1], gate[-1] = 2.0, 100.0
    y = lib().gated_rms_norm_fwd(x, gate, torch.ones(width, device="cuda"), activation="sigmoid")
    assert (y[-1] == 1).all() and (y[-2] == 0).all() and (y[0] == 0).all()


def test_side_stream():
    g = gen(8)
    x, w = rn(g, 300, 512), rn(g, 512, dtype=torch.float32)
    want, _ = lib().add_rms_norm_fwd(x, None, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = lib().add_rms_norm_fwd(x, None, w)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_autograd():
    g = gen(9)
    x, res, w = rn(g, 4, 6, 256), rn(g, 4, 6, 256, dtype=torch.float32), 1 + rn(g, 256, dtype=torch.float32, std=0.1)
    gate = rn(g, 4, 6, 256)
    leaves = [t.clone().requires_grad_() for t in (x, res, w, gate)]
    y, stream = lib().add_rms_norm(leaves[0], leaves[1], leaves[2], residual_scale=0.5)
    o = lib().gated_rms_norm(y, leaves[3], leaves[2], activation="sigmoid")
    do, ds = rn(g, 4, 6, 256), rn(g, 4, 6, 256, dtype=torch.float32)
    (o.float() * do.float()).sum().backward(retain_graph=True)
    alone = [t.grad.clone() for t in leaves]
    for t in leaves:
        t.grad = None
    torch.autograd.backward([o, stream], [do, ds])
    dy, dgate, dw2 = lib().gated_rms_norm_bwd(y.detach(), gate, w, do, activation="sigmoid")
    for with_ds, got in ((None, alone), (ds, [t.grad for t in leaves])):
        dx, dres, dw1 = lib().add_rms_norm_bwd(dy, with_ds, stream.detach(), w, residual_scale=0.5)
        for a, b in zip(got, (dx, dres, dw1 + dw2, dgate)):
            assert torch.equal(a, b)
    # without a residual the stream is the input itself
    leaf = x.clone().requires_grad_()
    y, stream = lib().add_rms_norm(leaf, None, w)
    assert stream is leaf
    torch.autograd.backward([y, stream], [do, do])
    dx, _, _ = lib().add_rms_norm_bwd(do, None, x, w, has_residual=False)
    assert rel_l2(f64(leaf.grad), f64(dx) + f64(do)) <= 2 ** -8


def test_gradients_against_differences():
    """Directional differences of <dy, y>. With 32768 outputs the bf16 roundings of y leave about 1e-2 / (2 h) of the loss's
    scale at h = 0.05: 5% of the derivative's is allowed."""
    g = gen(10)
    x, gate, w, dy = rn(g, 64, 512), rn(g, 64, 512), 1 + rn(g, 512, dtype=torch.float32, std=0.1), rn(g, 64, 512)
    dx, dgate, dw = lib().gated_rms_norm_bwd(x, gate, w, dy)
    h = 0.0625

    def loss(x, gate, w):
        return (lib().gated_rms_norm_fwd(x.contiguous(), gate.contiguous(), w).double() * dy.double()).sum()

    for i, (t, grad) in enumerate(((x, dx), (gate, dgate), (w, dw))):
        d = grad.double().sign()
        args = [x, gate, w]
        vals = []
        for s in (1, -1):
            moved = (t.double() + s * h * d).to(t.dtype)
            vals.append((moved.double(), loss(*(args[:i] + [moved] + args[i + 1:]))))
        want = ((vals[0][0] - vals[1][0]) * grad.double()).sum()      # the steps as they were rounded
        assert abs((vals[0][1] - vals[1][1]) - want) <= 0.05 * abs(want), i


def test_refusals():
    g = gen(11)
    x, w = rn(g, 4, 64), rn(g, 64, dtype=torch.float32)
    m = lib()
    for bad in (lambda: m.add_rms_norm_fwd(x.float(), None, w), lambda: m.add_rms_norm_fwd(x, None, w[:-1].contiguous()),
                lambda: m.add_rms_norm_fwd(x, x.half(), w), lambda: m.add_rms_norm_fwd(x, x[:2], w), lambda: m.add_rms_norm_fwd(x.t(), None, w),
                lambda: m.add_rms_norm_fwd(x, None, w, residual_scale=2.0), lambda: m.add_rms_norm_fwd(x, None, w, eps=-1.0),
                lambda: m.add_rms_norm_fwd(rn(g, 1, 16392), None, rn(g, 16392, dtype=torch.float32)), lambda: m.add_rms_norm_fwd(x[:0], None, w),
                lambda: m.gated_rms_norm_fwd(x, x, w, activation="gelu"), lambda: m.gated_rms_norm_fwd(x, x[:, :32], w),
                lambda: m.add_rms_norm_bwd(x, x.float(), x, w), lambda: m.add_rms_norm_bwd(x, None, x.float(), w, has_residual=False)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("rows,width", [(1300, 2568), (1300, 4096), (1300, 5000), (700, 8192), (700, 8200)])
def test_many_wide_rows(rows, width):
    """More rows than blocks, of more than one vector a thread: the weight gradients gather over a block's rows."""
    g = gen(rows + width)
    x, gate, w, dy, ds = rn(g, rows, width), rn(g, rows, width), 1 + rn(g, width, dtype=torch.float32, std=0.1), rn(g, rows, width), rn(g, rows, width, dtype=torch.float32)
    for act in ("silu", "sigmoid"):
        got = lib().gated_rms_norm_bwd(x, gate, w, dy, eps=1e-5, activation=act)
        want = block.gated_norm_bwd(f64(x), f64(gate), f64(w), f64(dy), 1e-5, act)
        close_bf16("dx", got[0], want[0])
        close_bf16("dgate", got[1], want[1])
        close_f32("dweight", got[2], want[2])
    for stream, d in ((ds, ds.flip(0).contiguous()), (ds, None), (x, gate)):
        dx, dres, dw = lib().add_rms_norm_bwd(dy, d, stream, w, eps=1e-5, residual_scale=0.7)
        rx, rr, rw = block.add_norm_bwd(f64(dy), None if d is None else f64(d), f64(stream), f64(w), 1e-5, 0.7)
        close_bf16("dx", dx, rx)
        close_stream(dres, rr, stream.dtype)
        close_f32("dweight", dw, rw)

"""The operators around the recurrence under autograd's other modes (CPU: the kernels' calls are replaced by stand-ins)."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import chunked_gated_delta_05_gb300 as lib
from chunked_gated_delta_05_gb300 import block_ops, ops


@pytest.fixture
def scan_calls(monkeypatch):
    """The arguments ``save`` of the forwards that a stand-in answers."""
    calls = []

    def fwd(u, *args, save=False, **kw):
        calls.append(save)
        y = u.detach() * 2
        return (y, None, torch.zeros(1)) if save else (y, None)

    monkeypatch.setattr(block_ops, "selective_scan_fwd", fwd)
    return calls


def scan_inputs():
    return [torch.ones(1, 4, 8), torch.ones(1, 4, 8), torch.ones(8, 2), torch.ones(1, 4, 1, 2), torch.ones(1, 4, 1, 2)]


@pytest.mark.parametrize("i", range(5))
@pytest.mark.parametrize("grad", [True, False])
def test_scan_refuses_tangents(scan_calls, i, grad):
    """A forward-mode tangent is refused, not dropped, with and without reverse mode."""
    args = scan_inputs()
    with torch.set_grad_enabled(grad), fwad.dual_level():
        args[i] = fwad.make_dual(args[i], torch.ones_like(args[i]))
        with pytest.raises(NotImplementedError):
            lib.selective_scan(*args)


@pytest.mark.parametrize("name", ["D", "z", "delta_bias", "initial_state"])
def test_scan_refuses_tangents_of_optional_inputs(scan_calls, name):
    with fwad.dual_level():
        t = torch.ones(8)
        with pytest.raises(NotImplementedError):
            lib.selective_scan(*scan_inputs(), **{name: fwad.make_dual(t, t)})


def test_scan_refuses_jvp(scan_calls):
    args = scan_inputs()
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda u: lib.selective_scan(u, *args[1:])[0], (args[0],), (torch.ones_like(args[0]),))


def test_scan_keeps_states_only_for_a_backward(scan_calls):
    args = scan_inputs()
    lib.selective_scan(*args)
    with fwad.dual_level():     # no tangent among the inputs
        y, _ = lib.selective_scan(*args)
        assert fwad.unpack_dual(y).tangent is None
    args[2].requires_grad_()
    with torch.no_grad():
        lib.selective_scan(*args)
    assert scan_calls == [False] * 3
    assert lib.selective_scan(*args)[0].grad_fn is not None and scan_calls[-1] is True


@pytest.fixture
def host_steps(monkeypatch):
    """The step wrappers on CPU tensors, their kernels' calls replaced by nothing."""
    monkeypatch.setattr(block_ops, "_device", lambda name, t: -1)
    monkeypatch.setattr(block_ops, "_run", lambda *a: None)


def step_calls():
    """``(state, call on it)`` of the four steps."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, g, beta = bf(2, 1, 128), torch.zeros(2, 1), bf(2, 1)
    x, w, A, B = bf(2, 8), torch.zeros(8, 4), torch.zeros(8, 2), bf(2, 1, 2)
    return [
        (bf(2, 3, 8), lambda s: lib.causal_conv1d_step(s, x, w)),
        (torch.zeros(2, 1, 128, 128), lambda s: lib.gdn_step(s, q, q, q, g, beta)),
        (torch.zeros(2, 1, 128, 128), lambda s: lib.kda_step(s, q, q, q, g[..., None].expand(2, 1, 128).contiguous(), beta)),
        (torch.zeros(2, 8, 2), lambda s: lib.selective_scan_step(s, x, x, A, B, B)),
    ]


@pytest.mark.parametrize("i", range(4))
def test_steps_count_as_changes_of_their_state(host_steps, i):
    state, call = step_calls()[i]
    before = state._version
    call(state)
    assert state._version > before

    class Keep(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, s):
            ctx.save_for_backward(s)
            return x * 1

        @staticmethod
        def backward(ctx, dy):
            return dy, ctx.saved_tensors[0]

    y = Keep.apply(torch.ones(2, requires_grad=True), state)
    call(state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("i", range(4))
def test_steps_take_states_made_in_inference_mode(host_steps, i):
    """Those have no version to raise."""
    with torch.inference_mode():
        state, call = step_calls()[i]
        call(state)
    call(state)
    state, call = step_calls()[i]
    with torch.inference_mode():
        call(state)


@pytest.mark.gpu
def test_a_step_on_a_saved_halo_is_noticed():
    x, w = torch.randn(2, 6, 16, device="cuda").bfloat16(), torch.randn(16, 4, device="cuda", requires_grad=True)
    state = torch.randn(2, 3, 16, device="cuda").bfloat16()
    y = lib.causal_conv1d(x, w, halo=state)
    y.sum().backward(retain_graph=True)
    lib.causal_conv1d_step(state, x[:, 0].contiguous(), w.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def ones(*shape, dtype=torch.float32):
    return torch.ones(*shape, dtype=dtype)


@pytest.mark.parametrize("name", ["add_rms_norm", "add_rms_norm alone", "gated_rms_norm", "selective_scan", "gdn", "causal_conv1d"])
def test_second_derivatives_are_refused(monkeypatch, name):
    """A gradient taken with create_graph=True has no derivative of its own: it must not pass for a constant."""
    bf = torch.bfloat16
    monkeypatch.setattr(block_ops, "add_rms_norm_fwd", lambda x, r, w, **kw: (x * 2, x if r is None else r + x))
    monkeypatch.setattr(block_ops, "add_rms_norm_bwd", lambda dy, ds, s, w, **kw: (dy * 2, None if not kw["has_residual"] else dy.to(s.dtype), torch.zeros_like(w)))
    monkeypatch.setattr(block_ops, "gated_rms_norm_fwd", lambda x, g, w, **kw: x * 2)
    monkeypatch.setattr(block_ops, "gated_rms_norm_bwd", lambda x, g, w, dy, **kw: (dy * 2, dy * 2, torch.zeros_like(w)))
    monkeypatch.setattr(block_ops, "selective_scan_fwd", lambda u, *a, **kw: (u * 2, None, torch.zeros(1)))
    monkeypatch.setattr(block_ops, "selective_scan_bwd", lambda u, delta, A, B, C, dy, **kw: (dy * 2, dy * 2, torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(C),
                                                                                               None, None, None, None))
    monkeypatch.setattr(ops, "_fwd", lambda kda, q, k, v, *a, **kw: (v * 2, None, torch.zeros(1)))
    monkeypatch.setattr(ops, "_bwd", lambda kda, q, k, v, g, beta, dO, *a: tuple(t * 2 for t in (q, k, v, beta, g)) + (None,))
    monkeypatch.setattr(ops, "causal_conv1d_fwd", lambda x, w, *a, **kw: x * 2)
    monkeypatch.setattr(ops, "causal_conv1d_bwd", lambda x, w, b, dy, **kw: (dy * 2, torch.zeros_like(w), None, None))
    x = ones(1, 4, 8, dtype=bf).requires_grad_()
    q = ones(1, 4, 1, 128, dtype=bf).requires_grad_()
    leaf, y = {
        "add_rms_norm": lambda: (x, lib.add_rms_norm(x, ones(1, 4, 8), ones(8))[0]),
        "add_rms_norm alone": lambda: (x, lib.add_rms_norm(x, None, ones(8))[0]),
        "gated_rms_norm": lambda: (x, lib.gated_rms_norm(x, ones(1, 4, 8, dtype=bf), ones(8))),
        "selective_scan": lambda: (x, lib.selective_scan(x, ones(1, 4, 8, dtype=bf), ones(8, 2), ones(1, 4, 1, 2), ones(1, 4, 1, 2))[0]),
        "gdn": lambda: (q, lib.chunk_gated_delta_rule(q, q.detach(), q.detach(), ones(1, 4, 1), ones(1, 4, 1, dtype=bf))[0]),
        "causal_conv1d": lambda: (x, lib.causal_conv1d(x, ones(8, 4))),
    }[name]()
    for loss in (y.float().sum(), (y.float() ** 2).sum()):     # the incoming gradient depends on nothing, or on the leaf
        grad, = torch.autograd.grad(loss, leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            (grad.float() * leaf.float()).sum().backward(retain_graph=True)


@pytest.mark.gpu
def test_first_derivatives_with_create_graph():
    """They are the same with create_graph=True, and used alone they still give an error, not zeros."""
    x, w = torch.randn(4, 64, device="cuda").bfloat16().requires_grad_(), torch.ones(64, device="cuda")
    y = lib.gated_rms_norm(x, x.detach(), w)
    plain, = torch.autograd.grad(y.float().sum(), x, retain_graph=True)
    graph, = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    assert torch.equal(plain, graph.detach())
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        graph.float().sum().backward()

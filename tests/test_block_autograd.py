"""The operators around the recurrence under autograd's other modes (CPU: the kernels' calls are replaced by stand-ins)."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import chunked_gated_delta_05_gb300 as lib
from chunked_gated_delta_05_gb300 import block_ops


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

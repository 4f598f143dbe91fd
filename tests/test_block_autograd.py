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

"""Refusals of the operators around the recurrence, before any device is touched (CPU): the C entry points with made-up
addresses and the Python wrappers."""
import ctypes
import struct

import pytest
import torch

import chunked_gated_delta_05_gb300 as lib
from chunked_gated_delta_05_gb300 import _lib

MB = 1 << 20


def refused(name, desc, args, why):
    code = getattr(_lib.load(), name)(ctypes.byref(desc), ctypes.byref(args), None)
    assert code == _lib.GDN_EINVAL, code
    assert why in _lib.load().gdn_last_error().decode()


def reaches_device(name, desc, args):
    """The call passes every check of its arguments (and stops at the missing device)."""
    assert getattr(_lib.load(), name)(ctypes.byref(desc), ctypes.byref(args), None) == _lib.GDN_EUNSUPPORTED


@pytest.mark.parametrize("cls", [c for c in vars(_lib).values() if isinstance(c, type) and issubclass(c, ctypes.Structure) and c is not ctypes.Structure])
def test_packed_structures_have_the_c_layout(cls):
    """Every field lands at its ctypes offset."""
    pack = _lib.packer(cls)
    values = [i + 1 for i in range(len(cls._fields_))]
    raw = pack(*values)
    s = cls.from_buffer_copy(raw)
    for (name, t), v in zip(cls._fields_, values):
        got = getattr(s, name)
        if t is ctypes.POINTER(ctypes.c_int32):
            got = ctypes.cast(got, ctypes.c_void_p).value
        assert got == v, name
    assert struct.calcsize("P") == 8


def norm_desc(**kw):
    return _lib.NormDesc(**{**dict(rows=4, width=64, eps=1e-6, residual_scale=1.0, stream_kind=2, activation=1), **kw})


def norm_fwd(**kw):
    return _lib.NormFwdArgs(**{**dict(x=MB, residual=2 * MB, weight=3 * MB, y=4 * MB, stream=5 * MB), **kw})


def norm_bwd(**kw):
    return _lib.NormBwdArgs(**{**dict(x=MB, gate=None, weight=2 * MB, dy=3 * MB, dstream=4 * MB, dx=5 * MB, dgate=None, dresidual=6 * MB,
                                      dweight=7 * MB, workspace=8 * MB, workspace_bytes=1 << 40), **kw})


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: without a GPU only")
def test_complete_calls_pass_the_checks():
    reaches_device("gdn_add_norm_fwd", norm_desc(), norm_fwd())
    reaches_device("gdn_add_norm_fwd", norm_desc(), norm_fwd(stream=2 * MB))       # the stream may be updated in place
    reaches_device("gdn_add_norm_bwd", norm_desc(), norm_bwd(dstream=None, dresidual=None))
    reaches_device("gdn_gated_norm_fwd", norm_desc(), norm_fwd(stream=None))
    reaches_device("gdn_gated_norm_bwd", norm_desc(), norm_bwd(gate=4 * MB, dstream=None, dgate=6 * MB, dresidual=None))
    reaches_device("gdn_conv_step", conv_desc(), conv_args())
    reaches_device("gdn_step", step_desc(), step_args())
    reaches_device("kda_step", step_desc(use_gate_in_kernel=1, lower_bound=-5.0), step_args(A_log=60 * MB, dt_bias=61 * MB))
    reaches_device("gdn_sscan_fwd", scan_desc(), scan_fwd())
    reaches_device("gdn_sscan_bwd", scan_desc(), scan_bwd())
    reaches_device("gdn_sscan_step", scan_desc(), scan_step())


@pytest.mark.parametrize("kw,why", [(dict(rows=0), "rows"), (dict(width=0), "width"), (dict(width=16385), "width"), (dict(eps=-1.0), "eps"),
                                    (dict(eps=float("nan")), "eps"), (dict(stream_kind=3), "stream_kind"),
                                    (dict(residual_scale=float("inf")), "residual_scale"), (dict(stream_kind=0, residual_scale=0.5), "residual_scale")])
def test_norm_descriptions(kw, why):
    refused("gdn_add_norm_fwd", norm_desc(**kw), norm_fwd(), why)


def test_norm_arguments():
    refused("gdn_add_norm_fwd", norm_desc(), norm_fwd(x=None), "non-NULL")
    refused("gdn_add_norm_fwd", norm_desc(), norm_fwd(residual=None), "residual")
    refused("gdn_add_norm_fwd", norm_desc(), norm_fwd(y=MB + 16), "alias")
    refused("gdn_add_norm_fwd", norm_desc(), norm_fwd(stream=2 * MB + 16), "alias")
    refused("gdn_add_norm_fwd", norm_desc(stream_kind=0), norm_fwd(), "NULL")
    refused("gdn_gated_norm_fwd", norm_desc(activation=0), norm_fwd(), "activation")
    refused("gdn_gated_norm_fwd", norm_desc(), norm_fwd(residual=None), "gate")
    refused("gdn_add_norm_bwd", norm_desc(), norm_bwd(dx=3 * MB), "alias")
    refused("gdn_add_norm_bwd", norm_desc(), norm_bwd(dresidual=5 * MB), "alias")
    refused("gdn_add_norm_bwd", norm_desc(stream_kind=0), norm_bwd(), "dresidual")
    refused("gdn_add_norm_bwd", norm_desc(), norm_bwd(workspace_bytes=16), "workspace")
    refused("gdn_gated_norm_bwd", norm_desc(), norm_bwd(), "gate")


def conv_desc(**kw):
    return _lib.ConvStepDesc(**{**dict(B=2, C=16, W=4, dilation=1, activation=1, num_slots=2, x_stride=0), **kw})


def conv_args(**kw):
    return _lib.ConvStepArgs(**{**dict(x=MB, weight=2 * MB, bias=None, state=3 * MB, state_indices=None, y=4 * MB, status=None), **kw})


@pytest.mark.parametrize("dkw,akw,why", [
    (dict(C=12), {}, "C"), (dict(W=9), {}, "W"), (dict(dilation=0), {}, "dilation"), (dict(activation=2), {}, "activation"),
    (dict(x_stride=12), {}, "x_stride"), (dict(x_stride=8), {}, "x_stride"), (dict(num_slots=1), {}, "num_slots"), ({}, dict(state=None), "non-NULL"),
    ({}, dict(x=MB + 2), "aligned"), ({}, dict(y=3 * MB), "alias"), ({}, dict(state=MB), "alias")])
def test_conv_step(dkw, akw, why):
    refused("gdn_conv_step", conv_desc(**dkw), conv_args(**akw), why)


def step_desc(**kw):
    return _lib.StepDesc(**{**dict(B=2, H=4, num_k_heads=2, num_slots=2, scale=0.0, use_qk_l2norm=1), **kw})


def step_args(**kw):
    return _lib.StepArgs(**{**dict(q=MB, k=2 * MB, v=3 * MB, g=4 * MB, beta=5 * MB, state=16 * MB, o=6 * MB), **kw})


@pytest.mark.parametrize("dkw,akw,why", [
    (dict(B=0), {}, "positive"), (dict(num_k_heads=3), {}, "num_k_heads"), (dict(scale=float("nan")), {}, "scale"), (dict(num_slots=1), {}, "num_slots"),
    (dict(use_gate_in_kernel=1, lower_bound=-1.0), {}, "KDA"), (dict(q_stride=128), {}, "strides"), (dict(v_stride=514), {}, "strides"),
    ({}, dict(beta=None), "non-NULL"), ({}, dict(q=MB + 4), "aligned"), ({}, dict(state=16 * MB + 8), "aligned"), ({}, dict(o=3 * MB), "alias"),
    ({}, dict(state=3 * MB), "alias")])
def test_delta_step(dkw, akw, why):
    refused("gdn_step", step_desc(**dkw), step_args(**akw), why)


def test_kda_step_gate():
    refused("kda_step", step_desc(use_gate_in_kernel=1, lower_bound=-6.0), step_args(), "lower_bound")
    refused("kda_step", step_desc(use_gate_in_kernel=1, lower_bound=-5.0), step_args(), "A_log")


def scan_desc(cu=None, **kw):
    d = _lib.SscanDesc(**{**dict(B=1, T=40, D=24, N=8, G=2, num_seqs=1, delta_softplus=1), **kw})
    if cu is not None:
        d._keep = (ctypes.c_int32 * len(cu))(*cu)
        d.cu_seqlens = ctypes.cast(d._keep, ctypes.POINTER(ctypes.c_int32))
        d.num_seqs = len(cu) - 1
    return d


def scan_fwd(**kw):
    return _lib.SscanFwdArgs(**{**dict(u=MB, delta=2 * MB, A=3 * MB, Bm=4 * MB, Cm=5 * MB, z=6 * MB, y=7 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


def scan_bwd(**kw):
    return _lib.SscanBwdArgs(**{**dict(u=MB, delta=2 * MB, A=3 * MB, Bm=4 * MB, Cm=5 * MB, z=6 * MB, dy=7 * MB, du=8 * MB, ddelta=9 * MB, dA=10 * MB,
                                       dB=11 * MB, dC=12 * MB, dz=13 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


def scan_step(**kw):
    return _lib.SscanStepArgs(**{**dict(u=MB, delta=2 * MB, A=3 * MB, Bm=4 * MB, Cm=5 * MB, state=8 * MB, num_slots=1, y=7 * MB), **kw})


@pytest.mark.parametrize("dkw,why", [
    (dict(N=0), "N"), (dict(N=17), "N"), (dict(G=5), "G"), (dict(T=0), "positive"), (dict(u_stride=23), "stride"), (dict(B_stride=15), "stride"),
    (dict(cu=[0, 10, 41]), "end"), (dict(cu=[1, 40]), "start"), (dict(cu=[0, 10, 10, 40]), "increasing"), (dict(cu=[0, 40], B=2), "batch")])
def test_scan_descriptions(dkw, why):
    refused("gdn_sscan_fwd", scan_desc(**dkw), scan_fwd(), why)
    assert _lib.load().gdn_sscan_fwd_workspace_size(ctypes.byref(scan_desc(**dkw))) == 0
    refused("gdn_sscan_bwd", scan_desc(**dkw), scan_bwd(), why)


@pytest.mark.parametrize("akw,why", [(dict(A=None), "non-NULL"), (dict(y=MB), "alias"), (dict(y=6 * MB), "alias"), (dict(workspace_bytes=1), "workspace"),
                                     (dict(workspace=64 * MB + 8), "workspace"), (dict(saved=65 * MB, saved_bytes=4), "saved")])
def test_scan_forward_arguments(akw, why):
    refused("gdn_sscan_fwd", scan_desc(), scan_fwd(**akw), why)


@pytest.mark.parametrize("akw,why", [(dict(dB=None), "non-NULL"), (dict(dz=None), "dz"), (dict(dD=20 * MB), "input"), (dict(dh0=20 * MB), "input"),
                                     (dict(du=MB), "alias"), (dict(du=9 * MB), "alias"), (dict(workspace_bytes=1), "workspace")])
def test_scan_backward_arguments(akw, why):
    refused("gdn_sscan_bwd", scan_desc(), scan_bwd(**akw), why)


def test_scan_step_arguments():
    refused("gdn_sscan_step", scan_desc(B=2), scan_step(), "num_slots")
    refused("gdn_sscan_step", scan_desc(cu=[0, 40]), scan_step(), "cu_seqlens")
    refused("gdn_sscan_step", scan_desc(), scan_step(state=MB), "alias")


def test_backward_workspace_covers_the_saved_states():
    d = scan_desc(T=5000, D=256)
    L = _lib.load()
    saved = L.gdn_sscan_saved_size(ctypes.byref(d))
    assert saved == 625 * 8 * 256 * 4            # a state of 8 per channel for every 8 tokens
    assert L.gdn_sscan_bwd_workspace_size(ctypes.byref(d)) > saved


def test_conv_state_arguments():
    d = _lib.ConvDesc(B=1, T=8, C=16, W=4, dilation=1, num_seqs=1, activation=1)
    refused("gdn_conv_state", d, _lib.ConvFwdArgs(x=MB, workspace=2 * MB, workspace_bytes=1 << 30), "state")
    refused("gdn_conv_state", d, _lib.ConvFwdArgs(x=MB, y=MB + 16, workspace=2 * MB, workspace_bytes=1 << 30), "alias")


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: lib.add_rms_norm_fwd(bf(2, 8), None, torch.ones(8)),
    lambda: lib.gated_rms_norm_fwd(bf(2, 8), bf(2, 8), torch.ones(8)),
    lambda: lib.gated_rms_norm_fwd(bf(2, 8), bf(2, 8), torch.ones(8), activation="relu"),
    lambda: lib.causal_conv1d_step(bf(2, 3, 8), bf(2, 8), torch.ones(8, 4)),
    lambda: lib.gdn_step(torch.zeros(1, 1, 128, 128), bf(1, 1, 128), bf(1, 1, 128), bf(1, 1, 128), torch.zeros(1, 1), bf(1, 1)),
    lambda: lib.selective_scan_fwd(bf(1, 4, 8), bf(1, 4, 8), torch.ones(8, 4), bf(1, 4, 1, 4), bf(1, 4, 1, 4)),
    lambda: lib.selective_scan_step(torch.zeros(1, 8, 4), bf(1, 8), bf(1, 8), torch.ones(8, 4), bf(1, 1, 4), bf(1, 1, 4)),
    lambda: lib.add_rms_norm_fwd([1.0], None, torch.ones(8)),
])
def test_wrappers_refuse_what_is_not_on_a_gpu(call):
    with pytest.raises(ValueError):
        call()

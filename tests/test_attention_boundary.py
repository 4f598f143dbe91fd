"""Refusals of the attention blocks before any device is touched (CPU): the C entry points with made-up addresses and the Python
wrappers."""
import ctypes

import pytest
import torch

import chunked_gated_delta_05_gb300 as lib
from chunked_gated_delta_05_gb300 import _lib

MB = 1 << 20


def refused(name, desc, args, why):
    code = getattr(_lib.load(), name)(ctypes.byref(desc), ctypes.byref(args), None)
    assert code == _lib.GDN_EINVAL, code
    assert why in _lib.load().gdn_last_error().decode()


def packed(d, cu):
    if cu is not None:
        d._keep = (ctypes.c_int32 * len(cu))(*cu)
        d.cu_seqlens = ctypes.cast(d._keep, ctypes.POINTER(ctypes.c_int32))
        d.num_seqs = len(cu) - 1
    return d


def rope_desc(cu=None, **kw):
    return packed(_lib.RopeDesc(**{**dict(B=1, T=40, num_seqs=1, H=4, num_k_heads=2, head_dim=64, rotary_dim=64, eps=1e-6, num_pages=4, page_size=16, table_width=3), **kw}), cu)


def rope_args(**kw):
    return _lib.RopeArgs(**{**dict(q=MB, k=2 * MB, v=3 * MB, q_weight=4 * MB, k_weight=5 * MB, inv_freq=6 * MB, q_out=7 * MB, k_out=8 * MB, k_cache=9 * MB, v_cache=10 * MB,
                                   page_table=11 * MB, lengths=12 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


def rope_bwd(**kw):
    return _lib.RopeBwdArgs(**{**dict(dq_out=MB, dk_out=2 * MB, q=3 * MB, k=4 * MB, q_weight=5 * MB, k_weight=6 * MB, inv_freq=7 * MB, dq=8 * MB, dk=9 * MB, dq_weight=10 * MB,
                                      dk_weight=11 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


def attn_desc(cu=None, **kw):
    return packed(_lib.AttnDesc(**{**dict(B=1, T=40, num_seqs=1, H=4, num_k_heads=2, head_dim=128, causal=1), **kw}), cu)


def attn_fwd(**kw):
    return _lib.AttnFwdArgs(**{**dict(q=MB, k=2 * MB, v=3 * MB, o=4 * MB, lse=5 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


def attn_bwd(**kw):
    return _lib.AttnBwdArgs(**{**dict(q=MB, k=2 * MB, v=3 * MB, o=4 * MB, lse=5 * MB, dO=6 * MB, dq=7 * MB, dk=8 * MB, dv=9 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


def step_desc(**kw):
    return _lib.AttnStepDesc(**{**dict(B=3, H=4, num_k_heads=2, head_dim=128, num_pages=4, page_size=16, table_width=3), **kw})


def step_args(**kw):
    return _lib.AttnStepArgs(**{**dict(q=MB, k_cache=2 * MB, v_cache=3 * MB, page_table=4 * MB, lengths=5 * MB, o=6 * MB, workspace=64 * MB, workspace_bytes=1 << 40), **kw})


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: without a GPU only")
@pytest.mark.parametrize("name,desc,args", [
    ("gdn_qk_norm_rope_fwd", rope_desc(), rope_args(v=None, k_cache=None, v_cache=None, page_table=None, lengths=None)),
    ("gdn_qk_norm_rope_fwd", rope_desc(rotary_dim=0), rope_args(inv_freq=None, q_weight=None, k_weight=None, positions=13 * MB)),
    ("gdn_qk_norm_rope_store", rope_desc(cu=[0, 7, 40]), rope_args()), ("gdn_qk_norm_rope_bwd", rope_desc(), rope_bwd()),
    ("gdn_qk_norm_rope_bwd", rope_desc(), rope_bwd(q_weight=None, k_weight=None, dq_weight=None, dk_weight=None)),
    ("gdn_attn_fwd", attn_desc(), attn_fwd(workspace=None, workspace_bytes=0)), ("gdn_attn_fwd", attn_desc(cu=[0, 40]), attn_fwd()), ("gdn_attn_bwd", attn_desc(), attn_bwd()), ("gdn_attn_step", step_desc(), step_args())])
def test_complete_calls_pass_the_checks(name, desc, args):
    """They stop at the missing device."""
    assert getattr(_lib.load(), name)(ctypes.byref(desc), ctypes.byref(args), None) == _lib.GDN_EUNSUPPORTED


SHAPES = [(dict(H=0), "H"), (dict(num_k_heads=3), "num_k_heads"), (dict(num_k_heads=-1), "H"), (dict(head_dim=96), "head_dim"), (dict(q_stride=12), "strides"),
          (dict(q_stride=260), "strides"), (dict(k_stride=64), "strides")]
SEQUENCES = [(dict(B=0), "positive"), (dict(T=0), "positive"), (dict(B=1 << 16, T=1 << 16), "large"), (dict(cu=[0, 10, 41]), "end"), (dict(cu=[1, 40]), "start"),
             (dict(cu=[0, 10, 10, 40]), "increasing"), (dict(cu=[0, 40], B=2), "batch")]


@pytest.mark.parametrize("kw,why", [*SHAPES, *SEQUENCES, (dict(rotary_dim=72), "rotary"), (dict(rotary_dim=24), "rotary"), (dict(rotary_dim=-16), "rotary"),
                                    (dict(interleaved=2), "interleaved"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps")])
def test_rope_descriptions(kw, why):
    refused("gdn_qk_norm_rope_fwd", rope_desc(**kw), rope_args(), why)
    refused("gdn_qk_norm_rope_bwd", rope_desc(**kw), rope_bwd(), why)
    assert _lib.load().gdn_qk_norm_rope_workspace_size(ctypes.byref(rope_desc(**kw))) == 0


@pytest.mark.parametrize("kw,why", [(dict(q=None), "non-NULL"), (dict(q_weight=None), "both"), (dict(inv_freq=None), "inv_freq"), (dict(k=2 * MB + 8), "aligned"),
                                    (dict(q_out=MB), "alias"), (dict(k_out=7 * MB + 16), "alias")])
def test_rope_arguments(kw, why):
    refused("gdn_qk_norm_rope_fwd", rope_desc(), rope_args(**kw), why)


@pytest.mark.parametrize("kw", [dict(workspace=None), dict(workspace_bytes=8), dict(workspace=64 * MB + 8)])
def test_packed_calls_need_a_workspace(kw):
    """For the documents' offsets or tiles; dense ones need none."""
    refused("gdn_qk_norm_rope_fwd", rope_desc(cu=[0, 40]), rope_args(**kw), "workspace")
    refused("gdn_qk_norm_rope_store", rope_desc(cu=[0, 40]), rope_args(**kw), "workspace")
    refused("gdn_attn_fwd", attn_desc(cu=[0, 40]), attn_fwd(**kw), "workspace")


@pytest.mark.parametrize("dkw,kw,why", [({}, dict(v=None), "non-NULL"), ({}, dict(lengths=None), "non-NULL"), ({}, dict(positions=20 * MB), "positions"), (dict(page_size=0), {}, "page"),
                                        (dict(table_width=1 << 28), {}, "table"), ({}, dict(k_cache=MB), "alias"), ({}, dict(v_cache=9 * MB), "alias"),
                                        ({}, dict(v_cache=10 * MB + 2), "aligned"), (dict(v_stride=8), {}, "strides")])
def test_store_arguments(dkw, kw, why):
    refused("gdn_qk_norm_rope_store", rope_desc(**dkw), rope_args(**kw), why)


@pytest.mark.parametrize("kw,why", [(dict(dq=None), "non-NULL"), (dict(dq_weight=None), "weight"), (dict(q_weight=None), "both"), (dict(dq=MB), "alias"), (dict(dk=8 * MB), "alias"),
                                    (dict(dk_weight=10 * MB), "alias"), (dict(workspace=None), "workspace")])
def test_rope_backward_arguments(kw, why):
    refused("gdn_qk_norm_rope_bwd", rope_desc(), rope_bwd(**kw), why)


@pytest.mark.parametrize("kw,why", [*SHAPES, *SEQUENCES, (dict(causal=2), "causal"), (dict(scale=float("inf")), "scale"), (dict(B=1 << 10, T=1 << 20, H=1 << 13, num_k_heads=0), "large")])
def test_attention_descriptions(kw, why):
    refused("gdn_attn_fwd", attn_desc(**kw), attn_fwd(), why)
    refused("gdn_attn_bwd", attn_desc(**kw), attn_bwd(), why)
    assert _lib.load().gdn_attn_fwd_workspace_size(ctypes.byref(attn_desc(**kw))) == 0
    assert _lib.load().gdn_attn_bwd_workspace_size(ctypes.byref(attn_desc(**kw))) == 0


@pytest.mark.parametrize("kw,why", [(dict(lse=None), "non-NULL"), (dict(v=3 * MB + 2), "aligned"), (dict(o=MB), "alias"), (dict(lse=4 * MB), "alias")])
def test_attention_forward_arguments(kw, why):
    refused("gdn_attn_fwd", attn_desc(), attn_fwd(**kw), why)


@pytest.mark.parametrize("kw,why", [(dict(dO=None), "non-NULL"), (dict(dv=9 * MB + 8), "aligned"), (dict(dq=MB), "alias"), (dict(dk=9 * MB), "alias"), (dict(workspace_bytes=64), "workspace")])
def test_attention_backward_arguments(kw, why):
    refused("gdn_attn_bwd", attn_desc(), attn_bwd(**kw), why)


@pytest.mark.parametrize("kw,why", [*[s for s in SHAPES if "k_stride" not in s[0]], (dict(B=0), "positive"), (dict(num_pages=0), "page"), (dict(page_size=0), "page"),
                                    (dict(table_width=0), "table"), (dict(table_width=1 << 28), "table"), (dict(scale=float("nan")), "scale"), (dict(B=1 << 30), "large")])
def test_step_descriptions(kw, why):
    why = "q_stride" if why == "strides" else why
    refused("gdn_attn_step", step_desc(**kw), step_args(), why)
    assert _lib.load().gdn_attn_step_workspace_size(ctypes.byref(step_desc(**kw))) == 0


@pytest.mark.parametrize("kw,why", [(dict(lengths=None), "non-NULL"), (dict(k_cache=2 * MB + 8), "aligned"), (dict(o=MB), "alias"), (dict(workspace_bytes=0), "workspace")])
def test_step_arguments(kw, why):
    refused("gdn_attn_step", step_desc(), step_args(**kw), why)


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


I32 = torch.int32


@pytest.mark.parametrize("call", [
    lambda: lib.qk_norm_rope_fwd(bf(1, 4, 2, 64), bf(1, 4, 1, 64), torch.ones(64), torch.ones(64), torch.ones(32)),
    lambda: lib.qk_norm_rope_store(bf(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64), None, None, torch.ones(32), bf(2, 8, 1, 64), bf(2, 8, 1, 64), torch.zeros(4, 1, dtype=I32), torch.ones(4, dtype=I32)),
    lambda: lib.attention_fwd(bf(1, 4, 2, 64), bf(1, 4, 1, 64), bf(1, 4, 1, 64)),
    lambda: lib.attention(bf(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64)),
    lambda: lib.attention_step(bf(4, 2, 64), bf(2, 8, 1, 64), bf(2, 8, 1, 64), torch.zeros(4, 1, dtype=I32), torch.ones(4, dtype=I32)),
    lambda: lib.attention_step(None, bf(2, 8, 1, 64), bf(2, 8, 1, 64), torch.zeros(4, 1, dtype=I32), torch.ones(4, dtype=I32)),
])
def test_wrappers_refuse_what_is_not_on_a_gpu(call):
    with pytest.raises(ValueError):
        call()

"""PyTorch-facing wrappers of the attention blocks between recurrent ones: norm and rotation of query and key heads (also into a
paged cache), attention over whole sequences, and single tokens' attention over the cache. Like ops.py this is argument
marshalling only; without the built library or a GB300 these functions raise."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _lib
from .block_ops import _BF16, _F32, _I32, _changed, _device, _differentiated, _p, _rows_of, _run, _status, _want
from .ops import _first_order, _kept, _offsets

_rope_desc, _rope_args, _rope_bwd_args = _lib.packer(_lib.RopeDesc), _lib.packer(_lib.RopeArgs), _lib.packer(_lib.RopeBwdArgs)
_attn_desc, _attn_fwd_args, _attn_bwd_args = _lib.packer(_lib.AttnDesc), _lib.packer(_lib.AttnFwdArgs), _lib.packer(_lib.AttnBwdArgs)
_step_desc, _step_args = _lib.packer(_lib.AttnStepDesc), _lib.packer(_lib.AttnStepArgs)


def _rows(name, t, shape, dev, width):
    """Elements between tokens of ``t [..,heads,D]`` (0: contiguous)."""
    if type(t) is torch.Tensor and t.dtype is _BF16 and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return 0
        if len(shape) == 4:     # the usual cases: a prompt's rows, a step's
            b, row, head, one = t.stride()
            if one == 1 and head == shape[3] and row >= width and shape[1] > 1 and (shape[0] == 1 or b == shape[1] * row):
                return row
        else:
            row, head, one = t.stride()
            if one == 1 and head == shape[2] and row >= width and shape[0] > 1:
                return row
    return _rows_of(name, t, _BF16, shape, dev, 2, width)


def _heads(q, k, v):
    """Shapes and strides of q ``[..,H,D]`` and of k, v ``[..,Hk,D]`` (v or None): ``(device, lead, H, Hk, D, strides)``."""
    dev = _device("q", q)
    shape = q.shape
    if len(shape) not in (3, 4) or q.numel() == 0:
        raise ValueError("q must be [B,T,H,D] (or [B,H,D] for single tokens)")
    if not isinstance(k, torch.Tensor) or k.dim() != len(shape):
        raise ValueError("k must have q's dimensions")
    *lead, H, D = shape
    Hk = k.shape[-2]
    if Hk < 1 or H % Hk != 0:
        raise ValueError("the query heads must be a multiple of the key heads")
    keys = (*lead, Hk, D)
    return dev, lead, H, Hk, D, (_rows("q", q, shape, dev, H * D), _rows("k", k, keys, dev, Hk * D), 0 if v is None else _rows("v", v, keys, dev, Hk * D))


def _vectors(n, dev, *vectors):
    """Whether all are contiguous fp32 vectors of n on the device: one cheap test of the usual case ahead of _want's messages."""
    for t in vectors:
        if not (isinstance(t, torch.Tensor) and t.dtype is _F32 and t.numel() == n and t.dim() == 1 and t.get_device() == dev and t.is_contiguous()):
            return False
    return True


def _packed(offsets, n):
    return (0, n) if offsets is None else (ctypes.addressof(offsets[0]), offsets[1])


def _rope_inputs(q, k, v, q_weight, k_weight, inv_freq, positions, interleaved, eps, offsets, cache):
    """Checks a call's inputs; ``(device, sequences, packed description)``. ``cache``: (pages, page size, table width) or zeros."""
    dev, lead, H, Hk, D, st = _heads(q, k, v)
    B, T = (lead[0], 1) if len(lead) == 1 else lead
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight must both be given or both be None")
    if q_weight is not None and not _vectors(D, dev, q_weight, k_weight):
        _want("q_weight", q_weight, _F32, (D,), dev)
        _want("k_weight", k_weight, _F32, (D,), dev)
    rotary = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rotary/2]")
        rotary = 2 * len(inv_freq)
        if not _vectors(rotary // 2, dev, inv_freq):
            _want("inv_freq", inv_freq, _F32, inv_freq.shape, dev)
    if positions is not None:
        _want("positions", positions, _I32, tuple(lead), dev)
    cu, n = _packed(offsets, B)
    return dev, n, _rope_desc(B, T, cu, n, H, Hk, D, rotary, 1 if interleaved else 0, eps, *st, *cache)


def _workspace(name, desc, like):
    """``(buffer, its address, its bytes)``."""
    n = _lib.size(name, desc)
    ws = torch.empty(n, dtype=torch.uint8, device=like.device)
    return ws, ws.data_ptr(), n


_NONE = (None, 0, 0)    # calls on dense batches that need no workspace


def _new(t):
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, *, positions=None, cu_seqlens: Optional[Sequence[int]] = None, eps=1e-6, interleaved=False):
    """RMS norm of every query and key head and its rotation by position, in one pass: ``n = x * rsqrt(mean(x^2) + eps) * weight``,
    then the first ``2 len(inv_freq)`` channels of ``n`` in pairs, the i-th turned by ``position * inv_freq[i]``. Pairs are
    ``(i, i + len(inv_freq))``, or ``(2i, 2i + 1)`` when ``interleaved``.

    q ``[B,T,H,D]``, k ``[B,T,Hk,D]`` bf16 (D 64 or 128; tokens may be strided slices of a wider projection), weights fp32 ``[D]`` (None,
    None: no norm), inv_freq fp32 and finite (None: no rotation; its rotary width must be a multiple of 16). Positions count from the start
    of the sequence (or document, by ``cu_seqlens``) or are given as int32 ``[B,T]``; angles keep their precision at any
    position. Returns ``(q, k)``, contiguous."""
    offsets = _offsets(cu_seqlens, 0)       # the packed description points into it
    dev, _, d = _rope_inputs(q, k, None, q_weight, k_weight, inv_freq, positions, interleaved, eps, offsets, (0, 0, 0))
    ws, *space = _NONE if offsets is None else _workspace("gdn_qk_norm_rope_workspace_size", d, q)
    qo, ko = _new(q), _new(k)
    _run("gdn_qk_norm_rope_fwd", d, _rope_args(q.data_ptr(), k.data_ptr(), 0, _p(q_weight), _p(k_weight), _p(inv_freq), _p(positions), qo.data_ptr(), ko.data_ptr(),
                                               0, 0, 0, 0, *space, 0), dev)
    return qo, ko


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, *, positions=None, cu_seqlens=None, eps=1e-6, interleaved=False):
    """Gradients ``(dq, dk, dq_weight, dk_weight)`` of ``<dq_out, q_out> + <dk_out, k_out>`` of :func:`qk_norm_rope_fwd` (the weights'
    fp32, None without a norm; summed in a fixed order)."""
    offsets = _offsets(cu_seqlens, 0)
    dev, _, d = _rope_inputs(q, k, None, q_weight, k_weight, inv_freq, positions, interleaved, eps, offsets, (0, 0, 0))
    _want("dq_out", dq_out, _BF16, q.shape, dev)
    _want("dk_out", dk_out, _BF16, k.shape, dev)
    ws, *space = _workspace("gdn_qk_norm_rope_workspace_size", d, q)
    dq, dk = _new(q), _new(k)
    dqw, dkw = (None, None) if q_weight is None else (torch.empty_like(q_weight), torch.empty_like(k_weight))
    _run("gdn_qk_norm_rope_bwd", d, _rope_bwd_args(dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), _p(q_weight), _p(k_weight), _p(inv_freq), _p(positions),
                                                   dq.data_ptr(), dk.data_ptr(), _p(dqw), _p(dkw), *space), dev)
    return dq, dk, dqw, dkw


def _cache(k_cache, v_cache, page_table, lengths, n, Hk, D, dev):
    """Checks a paged cache ``[pages,page size,Hk,D]`` and its tables; ``(pages, page size, table width)``."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages,page_size,Hk,D]")
    shape = k_cache.shape
    pages, page, heads, width = shape
    if not (heads == Hk and width == D and isinstance(v_cache, torch.Tensor) and v_cache.shape == shape and k_cache.dtype is v_cache.dtype is _BF16 and
            k_cache.get_device() == v_cache.get_device() == dev and k_cache.is_contiguous() and v_cache.is_contiguous()):     # which of these it is
        _want("k_cache", k_cache, _BF16, (pages, page, Hk, D), dev)
        _want("v_cache", v_cache, _BF16, (pages, page, Hk, D), dev)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [sequences,pages of a sequence]")
    rows, columns = page_table.shape
    if not (rows == n and isinstance(lengths, torch.Tensor) and lengths.dim() == 1 and lengths.numel() == n and page_table.dtype is lengths.dtype is _I32 and
            page_table.get_device() == lengths.get_device() == dev and page_table.is_contiguous() and lengths.is_contiguous()):
        _want("page_table", page_table, _I32, (n, columns), dev)
        _want("lengths", lengths, _I32, (n,), dev)
    return pages, page, columns


def qk_norm_rope_store(q, k, v, q_weight, k_weight, inv_freq, k_cache, v_cache, page_table, lengths, *, cu_seqlens: Optional[Sequence[int]] = None, eps=1e-6,
                       interleaved=False, status=None):
    """:func:`qk_norm_rope_fwd` of tokens that enter a paged cache: single tokens (q ``[B,H,D]``, k, v ``[B,Hk,D]``), prompts
    (``[B,T,..]``) or packed prompts (``cu_seqlens``). ``lengths`` (int32 ``[sequences]`` on the device) counts each sequence's tokens, the
    new ones among them: those are its last ones, and their positions follow. The turned keys and the values go to
    ``k_cache, v_cache [pages,page_size,Hk,D]`` (bf16, changed in place): token p to row ``p % page_size`` of page
    ``page_table[sequence, p // page_size]`` (int32). A length of 0 or less marks a padding sequence: zero outputs, nothing
    stored. So do tokens whose page lies outside the table or the cache, recorded as GDN_ERANGE in ``status`` (int32 [1] on the
    device). No place may be written twice in a call. Returns ``(q, k)`` turned; there are no gradients, and a backward that saved a
    cache before it changed raises."""
    offsets = _offsets(cu_seqlens, 0)
    if not isinstance(k, torch.Tensor) or k.dim() not in (3, 4):
        raise ValueError("k must be [B,T,Hk,D] or [B,Hk,D]")
    dev = _device("q", q)
    n = offsets[1] if offsets is not None else q.shape[0]
    cache = _cache(k_cache, v_cache, page_table, lengths, n, k.shape[-2], k.shape[-1], dev)
    _, _, d = _rope_inputs(q, k, v, q_weight, k_weight, inv_freq, None, interleaved, eps, offsets, cache)
    _status(status, dev)
    ws, *space = _NONE if offsets is None else _workspace("gdn_qk_norm_rope_workspace_size", d, q)
    qo, ko = _new(q), _new(k)
    _run("gdn_qk_norm_rope_store", d, _rope_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(q_weight), _p(k_weight), _p(inv_freq), 0, qo.data_ptr(), ko.data_ptr(),
                                                 k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr(), *space, _p(status)), dev)
    _changed(k_cache)
    _changed(v_cache)
    return qo, ko


def _scale(scale):
    """The description's scale: 0 for the default. One that fp32 holds as zero or infinite is refused."""
    if scale is None:
        return 0.0
    scale = ctypes.c_float(scale).value
    if not 0 < scale < math.inf:
        raise ValueError("scale must be positive and finite in fp32")
    return scale


def _attn_inputs(q, k, v, causal, scale, offsets):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B,T,H,D]")
    dev, lead, H, Hk, D, st = _heads(q, k, v)
    cu, n = _packed(offsets, lead[0])
    return dev, (*lead, H), _attn_desc(lead[0], lead[1], cu, n, H, Hk, D, 1 if causal else 0, _scale(scale), *st)


def attention_fwd(q, k, v, *, causal=True, scale=None, cu_seqlens: Optional[Sequence[int]] = None, status=None):
    """Attention over whole sequences: ``o = softmax(scale q k^T) v`` per head, every query seeing its sequence up to itself, or all
    of it (``causal=False``). q ``[B,T,H,D]``, k, v ``[B,T,Hk,D]`` bf16, D 64 or 128, Hk dividing H (head h reads key head
    ``h // (H // Hk)``); tokens may be strided slices of a wider projection. ``scale`` defaults to ``D**-0.5``. Packed documents by
    ``cu_seqlens``. Returns ``(o bf16 [B,T,H,D], lse fp32 [B,T,H])``, lse the logarithm of the softmax's denominator."""
    offsets = _offsets(cu_seqlens, 0)       # the packed description points into it
    dev, shape, d = _attn_inputs(q, k, v, causal, scale, offsets)
    _status(status, dev)
    ws, *space = _NONE if offsets is None else _workspace("gdn_attn_fwd_workspace_size", d, q)
    o, lse = _new(q), torch.empty(shape, dtype=_F32, device=q.device)
    _run("gdn_attn_fwd", d, _attn_fwd_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), *space, _p(status)), dev)
    return o, lse


def attention_bwd(dO, q, k, v, o, lse, *, causal=True, scale=None, cu_seqlens=None, status=None):
    """Gradients ``(dq, dk, dv)`` (bf16, contiguous) of ``<dO, o>``, given the inputs and results of :func:`attention_fwd`."""
    offsets = _offsets(cu_seqlens, 0)
    dev, shape, d = _attn_inputs(q, k, v, causal, scale, offsets)
    _want("dO", dO, _BF16, q.shape, dev)
    _want("o", o, _BF16, q.shape, dev)
    _want("lse", lse, _F32, shape, dev)
    _status(status, dev)
    ws, *space = _workspace("gdn_attn_bwd_workspace_size", d, q)
    dq, dk, dv = _new(q), _new(k), _new(v)
    _run("gdn_attn_bwd", d, _attn_bwd_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dO.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                           *space, _p(status)), dev)
    return dq, dk, dv


def attention_step(q, k_cache, v_cache, page_table, lengths, *, scale=None, status=None):
    """One token's attention per sequence over a paged cache (see :func:`qk_norm_rope_store`): row b of q ``[B,H,D]`` (bf16, rows may
    be strided) attends to the first ``lengths[b]`` keys of its pages. A length of 0 or less gives a zero row; so does one
    beyond the table, and a page outside the cache counts as absent keys, both recorded as GDN_ERANGE in ``status``. A cache of
    one slot a sequence is one page each. Steps have no gradients. Returns ``o [B,H,D]`` bf16."""
    dev = _device("q", q)
    if q.dim() != 3 or q.numel() == 0:
        raise ValueError("q must be [B,H,D]")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages,page_size,Hk,D]")
    B, H, D = q.shape
    Hk = k_cache.shape[2]
    if Hk < 1 or H % Hk != 0:
        raise ValueError("the query heads must be a multiple of the key heads")
    qs = _rows_of("q", q, _BF16, (B, H, D), dev, 2, H * D)
    pages, page, width = _cache(k_cache, v_cache, page_table, lengths, B, Hk, D, dev)
    _status(status, dev)
    d = _step_desc(B, H, Hk, D, _scale(scale), pages, page, width, qs)
    ws, *space = _workspace("gdn_attn_step_workspace_size", d, q)
    o = _new(q)
    _run("gdn_attn_step", d, _step_args(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr(), o.data_ptr(), *space, _p(status)), dev)
    return o


class QkNormRope(torch.autograd.Function):
    """Autograd wrapper of the head norms and rotation."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, eps, interleaved):
        out = qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions=positions, cu_seqlens=cu_seqlens, eps=eps, interleaved=interleaved)
        ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq, positions)
        ctx.cfg = dict(cu_seqlens=_kept(cu_seqlens), eps=eps, interleaved=interleaved)
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @_first_order
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, inv_freq, positions = ctx.saved_tensors
        whole = lambda g, t: torch.zeros(t.shape, dtype=_BF16, device=t.device) if g is None else g.contiguous()  # noqa: E731
        return (*qk_norm_rope_bwd(whole(dq, q), whole(dk, k), q, k, q_weight, k_weight, inv_freq, positions=positions, **ctx.cfg), None, None, None, None, None)


class Attention(torch.autograd.Function):
    """Autograd wrapper of attention over whole sequences."""

    @staticmethod
    def forward(ctx, q, k, v, causal, scale, cu_seqlens):
        o, lse = attention_fwd(q, k, v, causal=causal, scale=scale, cu_seqlens=cu_seqlens)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.cfg = dict(causal=causal, scale=scale, cu_seqlens=_kept(cu_seqlens))
        return o

    @staticmethod
    @_first_order
    def backward(ctx, dO):
        return (*attention_bwd(dO.contiguous(), *ctx.saved_tensors, **ctx.cfg), None, None, None)


def qk_norm_rope(q, k, q_weight, k_weight, inv_freq, *, positions=None, cu_seqlens=None, eps=1e-6, interleaved=False):
    """Differentiable head norms and rotation (see :func:`qk_norm_rope_fwd`): ``(q, k)``. ``inv_freq`` has no gradient."""
    if inv_freq is not None and _differentiated((inv_freq,)):
        raise ValueError("inv_freq has no gradient")
    if not _differentiated((q, k, q_weight, k_weight)):
        return qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions=positions, cu_seqlens=cu_seqlens, eps=eps, interleaved=interleaved)
    return QkNormRope.apply(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, eps, interleaved)


def attention(q, k, v, *, causal=True, scale=None, cu_seqlens=None):
    """Differentiable attention over whole sequences (see :func:`attention_fwd`): ``o``. Reverse mode only. As for any differentiable
    call, a step is captured into a graph while no eager graph of the same leaves lives (the autograd engine would join the stream
    that made that one, which a capture does not allow)."""
    if not _differentiated((q, k, v)):
        return attention_fwd(q, k, v, causal=causal, scale=scale, cu_seqlens=cu_seqlens)[0]
    return Attention.apply(q, k, v, causal, scale, cu_seqlens)

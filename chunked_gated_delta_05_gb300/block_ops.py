"""PyTorch-facing wrappers of the operators around the recurrence: the norms before and after a block, the selective
state space scan, and the single-token steps of the convolution, the delta rule and the scan. Like ops.py this is
argument marshalling only; without the built library or a GB300 these functions raise."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch
import torch.autograd.forward_ad as forward_ad

from . import _lib
from .ops import K_DIM, _check_tensor, _conv_checks, _conv_desc, _first_order, _gate_checks, _kept, _launch, _offsets

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_ACTIVATIONS = {"silu": 1, "sigmoid": 2}


def _want(name, t, dtype, shape, dev):
    """_check_tensor behind one cheap test of the usual case. ``dev``: the device's index."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        _check_tensor(name, t, dtype, shape, torch.device("cuda", dev))


def _p(t):
    return 0 if t is None else t.data_ptr()


_norm_desc = _lib.packer(_lib.NormDesc)
_norm_fwd_args, _norm_bwd_args = _lib.packer(_lib.NormFwdArgs), _lib.packer(_lib.NormBwdArgs)
_conv_step_desc, _conv_step_args = _lib.packer(_lib.ConvStepDesc), _lib.packer(_lib.ConvStepArgs)
_step_desc, _step_args = _lib.packer(_lib.StepDesc), _lib.packer(_lib.StepArgs)
_scan_desc, _scan_step_args = _lib.packer(_lib.SscanDesc), _lib.packer(_lib.SscanStepArgs)


def _run(name, desc, args, dev):
    _launch(_lib.entry(name), desc, args, dev)


def _device(name, t):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError("inputs must be CUDA tensors")
    return dev


def _rows_of(name, t, dtype, shape, dev, inner, width):
    """Elements between the rows (of ``width`` elements) of ``t``, whose last ``inner`` dimensions are contiguous and whose
    leading ones follow each other at one stride (a slice of a wider projection qualifies)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _check_tensor(name, t, dtype, shape, torch.device("cuda", dev))
    if t.is_contiguous():
        return width
    st, lead = t.stride(), len(shape) - inner
    if lead == 1 and st[-1] == 1 and st[0] >= width and (inner == 1 or st[1] == shape[2]):    # a step's usual case
        return st[0] if shape[0] > 1 else width
    w = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != w:
            raise ValueError(f"{name}'s rows must be contiguous")
        w *= shape[i]
    row = None
    for i in range(lead - 1, -1, -1):       # from the innermost leading dimension of more than one row
        if shape[i] == 1:
            continue
        if row is None:
            row, n = st[i], shape[i]
            if row < w:
                raise ValueError(f"{name}'s rows must not overlap (an expanded tensor must be made contiguous)")
        elif st[i] != n * row:
            raise ValueError(f"{name}'s rows must follow each other at one stride")
        else:
            n *= shape[i]
    return w if row is None else row


def _like(t):
    """An empty contiguous tensor of t's shape (None of None)."""
    return None if t is None else torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _pool(state_indices, B, slots, dev):
    if state_indices is not None:
        _want("state_indices", state_indices, _I32, (B,), dev)
    elif slots < B:
        raise ValueError("the state must have a slot for every row")


def _status(status, dev):
    if status is not None:
        _want("status", status, _I32, (1,), dev)


# ---------------------------------------------------------------- norms

def _norm_workspace(rows, width, like):
    n = _lib.size("gdn_norm_bwd_workspace_size", _norm_desc(rows, width, 0.0, 1.0, 0, 0))
    return torch.empty(n, dtype=torch.uint8, device=like.device), n


def _norm_shape(x):
    dev = _device("x", x)
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError("x must have at least one row")
    _want("x", x, _BF16, x.shape, dev)
    width = x.shape[-1]
    return dev, x.numel() // width, width


def add_rms_norm_fwd(x, residual, weight, *, eps=1e-6, residual_scale=1.0):
    """Residual sum and RMS norm before a block: ``stream = residual + residual_scale * x`` (kept in the residual's type,
    fp32 or bf16), ``y = stream * rsqrt(mean(stream^2) + eps) * weight`` over the last dimension of ``x`` (bf16), with
    ``weight`` fp32. Without a residual (None) the stream is x itself. Returns ``(y bf16, stream)``."""
    dev, rows, width = _norm_shape(x)
    _want("weight", weight, _F32, (width,), dev)
    kind = 0
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (_BF16, _F32):
            raise ValueError("residual must be a float32 or bfloat16 tensor")
        _want("residual", residual, residual.dtype, x.shape, dev)
        kind = 2 if residual.dtype is _F32 else 1
    y = torch.empty_like(x)
    stream = x if residual is None else torch.empty_like(residual)
    _run("gdn_add_norm_fwd", _norm_desc(rows, width, eps, residual_scale, kind, 0),
         _norm_fwd_args(x.data_ptr(), _p(residual), weight.data_ptr(), y.data_ptr(), stream.data_ptr() if kind else 0), dev)
    return y, stream


def add_rms_norm_bwd(dy, dstream, stream, weight, *, eps=1e-6, residual_scale=1.0, has_residual=True):
    """Gradients of :func:`add_rms_norm_fwd` from ``dy`` (bf16) and ``dstream`` (the stream's type, or None), given the
    forward's ``stream``. Returns ``(dx bf16, dresidual (the stream's type) or None, dweight fp32)``."""
    dev, rows, width = _norm_shape(dy)
    if not isinstance(stream, torch.Tensor) or stream.dtype not in ((_BF16, _F32) if has_residual else (_BF16,)):
        raise ValueError("stream must be the tensor returned by the forward")
    _want("stream", stream, stream.dtype, dy.shape, dev)
    _want("weight", weight, _F32, (width,), dev)
    if dstream is not None:
        _want("dstream", dstream, stream.dtype, dy.shape, dev)
    kind = 0 if not has_residual else 2 if stream.dtype is _F32 else 1
    ws, ws_bytes = _norm_workspace(rows, width, weight)
    dx = torch.empty_like(dy)
    dres = torch.empty_like(stream) if has_residual else None
    dw = torch.empty_like(weight)
    _run("gdn_add_norm_bwd", _norm_desc(rows, width, eps, residual_scale, kind, 0),
         _norm_bwd_args(stream.data_ptr(), 0, weight.data_ptr(), dy.data_ptr(), _p(dstream), dx.data_ptr(), 0, _p(dres), dw.data_ptr(), ws.data_ptr(), ws_bytes), dev)
    return dx, dres, dw


def _act(activation):
    if activation not in _ACTIVATIONS:
        raise ValueError('activation must be "silu" or "sigmoid"')
    return _ACTIVATIONS[activation]


def gated_rms_norm_fwd(x, gate, weight, *, eps=1e-6, activation="silu"):
    """Gated RMS norm after the recurrence: ``y = x * rsqrt(mean(x^2) + eps) * weight * act(gate)`` over the last dimension
    (a head, or a whole row), x and gate bf16, weight fp32, act "silu" or "sigmoid". Returns ``y`` (bf16)."""
    act = _act(activation)
    dev, rows, width = _norm_shape(x)
    _want("gate", gate, _BF16, x.shape, dev)
    _want("weight", weight, _F32, (width,), dev)
    y = torch.empty_like(x)
    _run("gdn_gated_norm_fwd", _norm_desc(rows, width, eps, 1.0, 0, act), _norm_fwd_args(x.data_ptr(), gate.data_ptr(), weight.data_ptr(), y.data_ptr(), 0), dev)
    return y


def gated_rms_norm_bwd(x, gate, weight, dy, *, eps=1e-6, activation="silu"):
    """Gradients ``(dx bf16, dgate bf16, dweight fp32)`` of ``<dy, gated_rms_norm_fwd(...)>``."""
    act = _act(activation)
    dev, rows, width = _norm_shape(x)
    _want("gate", gate, _BF16, x.shape, dev)
    _want("weight", weight, _F32, (width,), dev)
    _want("dy", dy, _BF16, x.shape, dev)
    ws, ws_bytes = _norm_workspace(rows, width, weight)
    dx, dgate, dw = torch.empty_like(x), torch.empty_like(gate), torch.empty_like(weight)
    _run("gdn_gated_norm_bwd", _norm_desc(rows, width, eps, 1.0, 0, act),
         _norm_bwd_args(x.data_ptr(), gate.data_ptr(), weight.data_ptr(), dy.data_ptr(), 0, dx.data_ptr(), dgate.data_ptr(), 0, dw.data_ptr(), ws.data_ptr(), ws_bytes), dev)
    return dx, dgate, dw


class AddRmsNorm(torch.autograd.Function):
    """Autograd wrapper of the residual sum and norm."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps, residual_scale):
        y, stream = add_rms_norm_fwd(x, residual, weight, eps=eps, residual_scale=residual_scale)
        ctx.save_for_backward(stream, weight)
        ctx.cfg = (eps, residual_scale, residual is not None)
        ctx.set_materialize_grads(False)
        return (y, stream) if residual is not None else y

    @staticmethod
    @_first_order
    def backward(ctx, dy, dstream=None):
        stream, weight = ctx.saved_tensors
        eps, scale, has_residual = ctx.cfg
        dy = torch.zeros_like(stream, dtype=_BF16) if dy is None else dy.contiguous()
        dx, dres, dw = add_rms_norm_bwd(dy, None if dstream is None else dstream.contiguous(), stream, weight, eps=eps,
                                        residual_scale=scale, has_residual=has_residual)
        return dx, dres, dw, None, None


class GatedRmsNorm(torch.autograd.Function):
    """Autograd wrapper of the gated norm."""

    @staticmethod
    def forward(ctx, x, gate, weight, eps, activation):
        ctx.save_for_backward(x, gate, weight)
        ctx.cfg = (eps, activation)
        return gated_rms_norm_fwd(x, gate, weight, eps=eps, activation=activation)

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, gate, weight = ctx.saved_tensors
        eps, activation = ctx.cfg
        return (*gated_rms_norm_bwd(x, gate, weight, dy.contiguous(), eps=eps, activation=activation), None, None)


def add_rms_norm(x, residual, weight, *, eps=1e-6, residual_scale=1.0):
    """Differentiable residual sum and norm (see :func:`add_rms_norm_fwd`): ``(y, stream)``."""
    if residual is None:
        return AddRmsNorm.apply(x, None, weight, eps, residual_scale), x
    return AddRmsNorm.apply(x, residual, weight, eps, residual_scale)


def gated_rms_norm(x, gate, weight, *, eps=1e-6, activation="silu"):
    """Differentiable gated norm (see :func:`gated_rms_norm_fwd`)."""
    return GatedRmsNorm.apply(x, gate, weight, eps, activation)


# ---------------------------------------------------------------- single-token steps

def _changed(state):
    """Tells autograd that a kernel wrote to the state, so that a backward that had saved it raises."""
    if not state.is_inference():
        torch.autograd.graph.increment_version(state)


def causal_conv1d_state(x, weight, *, dilation=1, cu_seqlens: Optional[Sequence[int]] = None, halo=None):
    """The state that a prompt ``x [B,T,C]`` leaves for :func:`causal_conv1d_step`: the last ``(W-1)*dilation`` inputs of
    every sequence (from its halo, or zeros, where it is shorter), bf16 ``[N,(W-1)*dilation,C]``."""
    lib = _lib.load()
    offsets = _offsets(cu_seqlens, x.shape[1] if x.dim() == 3 else 0)
    desc = _conv_desc(x, weight, dilation, False, offsets)
    N, HW = desc.num_seqs, (weight.shape[1] - 1) * dilation
    _conv_checks(x, weight, None, halo, N, HW)
    dev = x.get_device()
    ws_bytes = lib.gdn_conv_fwd_workspace_size(desc)
    if ws_bytes == 0:
        _lib.check(_lib.GDN_EINVAL)
    state = torch.empty((N, HW, x.shape[2]), dtype=_BF16, device=x.device)
    if HW == 0:
        return state
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    a = _lib.ConvFwdArgs(x=x.data_ptr(), halo=_p(halo), y=state.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=ws_bytes)
    _launch(lib.gdn_conv_state, desc, a, dev)
    return state


def causal_conv1d_step(state, x, weight, bias=None, *, dilation=1, activation=True, state_indices=None, status=None):
    """One token of the short convolution: ``x [B,C]`` (bf16, rows may be strided) against ``state
    [slots,(W-1)*dilation,C]``, which is updated in place. ``state_indices`` (int32 [B] on the device) names each row's slot;
    a negative one marks a padding row (zero output, no state touched), and no slot may be named twice. A row whose slot lies
    outside the state is treated as padding and recorded as GDN_ERANGE in ``status`` (int32 [1] on the device). Steps have no
    gradients; a backward that saved ``state`` before it changed raises. Returns ``y [B,C]``."""
    dev = _device("x", x)
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [B,C] and weight [C,W]")
    B, C = x.shape
    W = weight.shape[1]
    xs = _rows_of("x", x, _BF16, (B, C), dev, 1, C)
    _want("weight", weight, _F32, (C, W), dev)
    if bias is not None:
        _want("bias", bias, _F32, (C,), dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be [slots,(W-1)*dilation,C]")
    slots = state.shape[0]
    _want("state", state, _BF16, (slots, (W - 1) * dilation, C), dev)
    _pool(state_indices, B, slots, dev)
    _status(status, dev)
    y = _like(x)
    _run("gdn_conv_step", _conv_step_desc(B, C, W, dilation, 1 if activation else 0, slots, xs),
         _conv_step_args(x.data_ptr(), weight.data_ptr(), _p(bias), state.data_ptr(), _p(state_indices), y.data_ptr(), _p(status)), dev)
    _changed(state)
    return y


def _delta_step(per_channel, state, q, k, v, g, beta, state_indices, l2, sig, scale, gate, status):
    dev = _device("q", q)
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q and v must have shape [B,H,128]")
    B, Hk, _ = q.shape
    H = v.shape[1]
    if Hk < 1 or H % Hk != 0:
        raise ValueError("the value heads must be a multiple of the q/k heads")
    qk = (B, Hk, K_DIM)
    qs = _rows_of("q", q, _BF16, qk, dev, 2, Hk * K_DIM)
    ks = _rows_of("k", k, _BF16, qk, dev, 2, Hk * K_DIM)
    vs = _rows_of("v", v, _BF16, (B, H, K_DIM), dev, 2, H * K_DIM)
    _want("g", g, _F32, (B, H, K_DIM) if per_channel else (B, H), dev)
    _want("beta", beta, _BF16, (B, H), dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [slots,H,128,128]")
    slots = state.shape[0]
    _want("state", state, _F32, (slots, H, K_DIM, K_DIM), dev)
    A_log, dt_bias = (None, None) if gate is None else _gate_checks(gate, H, q.device)
    _pool(state_indices, B, slots, dev)
    _status(status, dev)
    o = _like(v)
    _run("kda_step" if per_channel else "gdn_step",
         _step_desc(B, H, Hk, slots, 0.0 if scale is None else scale, 1 if l2 else 0, 1 if sig else 0,
                    0 if gate is None else 1, 0.0 if gate is None else gate[2], qs, ks, vs),
         _step_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(), _p(state_indices), o.data_ptr(), _p(A_log), _p(dt_bias), _p(status)), dev)
    _changed(state)
    return o


def gdn_step(state, q, k, v, g, beta, *, state_indices=None, use_qk_l2norm=True, use_beta_sigmoid=False, scale=None, status=None):
    """One token of Gated DeltaNet per batch row: q, k ``[B,Hk,128]``, v ``[B,H,128]`` (bf16, rows may be strided, Hk
    dividing H), g ``[B,H]`` fp32, beta ``[B,H]`` bf16, and ``state [slots,H,128,128]`` fp32, updated in place (the final state
    of :func:`gdn_fwd` is one). ``state_indices`` as for :func:`causal_conv1d_step`. Returns ``o [B,H,128]`` bf16."""
    return _delta_step(False, state, q, k, v, g, beta, state_indices, use_qk_l2norm, use_beta_sigmoid, scale, None, status)


def kda_step(state, q, k, v, g, beta, *, state_indices=None, use_qk_l2norm=True, use_beta_sigmoid=True, scale=None, status=None,
             A_log=None, dt_bias=None, lower_bound=None):
    """One token of Kimi Delta Attention per batch row: as :func:`gdn_step` with the per-channel gate g ``[B,H,128]``, or
    its logits with ``A_log``, ``dt_bias`` and ``lower_bound`` (see :func:`kda_fwd`)."""
    gate = None if A_log is None else (A_log, dt_bias, lower_bound)
    return _delta_step(True, state, q, k, v, g, beta, state_indices, use_qk_l2norm, use_beta_sigmoid, scale, gate, status)


# ---------------------------------------------------------------- selective scan

def _sscan_desc(u, delta, A, Bm, Cm, D, z, delta_bias, softplus, lead, offsets):
    """Checks the inputs of a scan (lead = 2: [B,T,..]) or a step (lead = 1: [B,..]); ``(device, sequences, D, N, packed description)``."""
    dev = _device("u", u)
    if u.dim() != lead + 1 or u.numel() == 0:
        raise ValueError("u must be [B,T,D]" if lead == 2 else "u must be [B,D]")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [D,N]")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != lead + 2:
        raise ValueError("B must be [B,T,G,N]" if lead == 2 else "B must be [B,G,N]")
    shape, head = u.shape, u.shape[:lead]
    Dc, N, G = shape[lead], A.shape[1], Bm.shape[lead]
    vectors = (*head, G, N)
    us = _rows_of("u", u, _BF16, shape, dev, 1, Dc)
    ds = _rows_of("delta", delta, _BF16, shape, dev, 1, Dc)
    zs = _rows_of("z", z, _BF16, shape, dev, 1, Dc) if z is not None else 0
    bs = _rows_of("B", Bm, _BF16, vectors, dev, 2, G * N)
    cs = _rows_of("C", Cm, _BF16, vectors, dev, 2, G * N)
    _want("A", A, _F32, (Dc, N), dev)
    if D is not None:
        _want("D", D, _F32, (Dc,), dev)
    if delta_bias is not None:
        _want("delta_bias", delta_bias, _F32, (Dc,), dev)
    B, T = head[0], head[1] if lead == 2 else 1
    cu, n = (0, B) if offsets is None else (ctypes.addressof(offsets[0]), offsets[1])
    return dev, n, Dc, N, _scan_desc(B, T, Dc, N, G, cu, n, 1 if softplus else 0, us, ds, zs, bs, cs)


_scan_fwd_args, _scan_bwd_args = _lib.packer(_lib.SscanFwdArgs), _lib.packer(_lib.SscanBwdArgs)


def selective_scan_fwd(u, delta, A, B, C, *, D=None, z=None, delta_bias=None, delta_softplus=True, initial_state=None,
                       output_final_state=False, cu_seqlens: Optional[Sequence[int]] = None, save=False):
    """Selective state space scan. For every channel with N <= 16 states:
    ``dt = softplus(delta + delta_bias)`` (or without softplus), ``h = exp(dt A) h + dt u B_t``, ``y = (C_t . h + D u) silu(z)``.

    u, delta, z: bf16 ``[B,T,D]``; B, C: bf16 ``[B,T,G,N]``, shared by the D/G channels of a group (rows of all five may be
    strided slices of wider projections); A fp32 ``[D,N]`` (negative); D, delta_bias fp32 ``[D]``; states fp32
    ``[sequences,D,N]``. Packed documents by ``cu_seqlens``. Returns ``(y bf16, final_state or None)``; with ``save=True``
    also the buffer to hand to :func:`selective_scan_bwd`."""
    offsets = _offsets(cu_seqlens, 0)       # the packed description points into it
    dev, *state_shape, d = _sscan_desc(u, delta, A, B, C, D, z, delta_bias, delta_softplus, 2, offsets)
    state_shape = tuple(state_shape)
    if initial_state is not None:
        _want("initial_state", initial_state, _F32, state_shape, dev)
    ws_bytes = _lib.size("gdn_sscan_fwd_workspace_size", d)
    y = _like(u)
    final = torch.empty(state_shape, dtype=_F32, device=A.device) if output_final_state else None
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=u.device)
    saved_bytes, saved = 0, None
    if save:
        saved_bytes = _lib.size("gdn_sscan_saved_size", d)
        saved = torch.empty(saved_bytes, dtype=torch.uint8, device=u.device)
    _run("gdn_sscan_fwd", d, _scan_fwd_args(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(delta_bias), _p(z), _p(initial_state),
                                            y.data_ptr(), _p(final), ws.data_ptr(), ws_bytes, _p(saved), saved_bytes), dev)
    return (y, final, saved) if save else (y, final)


def selective_scan_bwd(u, delta, A, B, C, dy, *, D=None, z=None, delta_bias=None, delta_softplus=True, initial_state=None,
                       dfinal=None, cu_seqlens=None, saved=None):
    """Gradients of ``<dy, y> + <dfinal, final_state>``: ``(du, ddelta, dA, dB, dC, dD, dz, ddelta_bias, dh0)``, None where the
    input is None. ``saved`` is the buffer of a ``save=True`` forward on the same inputs (else its states are recomputed)."""
    offsets = _offsets(cu_seqlens, 0)       # the packed description points into it
    dev, *state_shape, d = _sscan_desc(u, delta, A, B, C, D, z, delta_bias, delta_softplus, 2, offsets)
    state_shape = tuple(state_shape)
    _want("dy", dy, _BF16, u.shape, dev)
    for name, t in (("initial_state", initial_state), ("dfinal", dfinal)):
        if t is not None:
            _want(name, t, _F32, state_shape, dev)
    ws_bytes = _lib.size("gdn_sscan_bwd_workspace_size", d)
    saved_bytes = 0
    if saved is not None:
        saved_bytes = _lib.size("gdn_sscan_saved_size", d)
        if not isinstance(saved, torch.Tensor) or saved.get_device() != dev or not saved.is_contiguous() or saved.numel() * saved.element_size() < saved_bytes:
            raise ValueError("saved must be the buffer returned by the forward with save=True")
        ws_bytes -= saved_bytes

    du, ddelta, dz = torch.empty_like(dy), torch.empty_like(dy), None if z is None else torch.empty_like(dy)
    dA, dB, dC, dD, dbias, dh0 = torch.empty_like(A), _like(B), _like(C), _like(D), _like(delta_bias), _like(initial_state)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=u.device)
    _run("gdn_sscan_bwd", d, _scan_bwd_args(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(delta_bias), _p(z), _p(initial_state),
                                            dy.data_ptr(), _p(dfinal), du.data_ptr(), ddelta.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _p(dD), _p(dbias), _p(dz),
                                            _p(dh0), ws.data_ptr(), ws_bytes, _p(saved), saved_bytes), dev)
    return du, ddelta, dA, dB, dC, dD, dz, dbias, dh0


def selective_scan_step(state, u, delta, A, B, C, *, D=None, z=None, delta_bias=None, delta_softplus=True, state_indices=None,
                        status=None):
    """One token of the selective scan per batch row: u, delta, z ``[B,D]``, B, C ``[B,G,N]`` (bf16, rows may be strided) and
    ``state [slots,D,N]`` fp32, updated in place (the final state of :func:`selective_scan_fwd` is one). ``state_indices`` as
    for :func:`causal_conv1d_step`. Returns ``y [B,D]`` bf16."""
    dev, rows, Dc, N, d = _sscan_desc(u, delta, A, B, C, D, z, delta_bias, delta_softplus, 1, None)
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be [slots,D,N]")
    slots = state.shape[0]
    _want("state", state, _F32, (slots, Dc, N), dev)
    _pool(state_indices, rows, slots, dev)
    _status(status, dev)
    y = _like(u)
    _run("gdn_sscan_step", d, _scan_step_args(u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(delta_bias), _p(z), state.data_ptr(),
                                              _p(state_indices), slots, y.data_ptr(), _p(status)), dev)
    _changed(state)
    return y


class SelectiveScan(torch.autograd.Function):
    """Autograd wrapper of the selective scan: the forward keeps a state every 8 tokens, the backward starts from them."""

    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, initial_state, delta_softplus, output_final_state, cu_seqlens):
        y, final, saved = selective_scan_fwd(u, delta, A, B, C, D=D, z=z, delta_bias=delta_bias, delta_softplus=delta_softplus,
                                             initial_state=initial_state, output_final_state=output_final_state,
                                             cu_seqlens=cu_seqlens, save=True)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, initial_state, saved)
        ctx.cfg = (delta_softplus, _kept(cu_seqlens))
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @_first_order
    def backward(ctx, dy, dfinal):
        u, delta, A, B, C, D, z, delta_bias, h0, saved = ctx.saved_tensors
        softplus, cu = ctx.cfg
        dy = torch.zeros(u.shape, dtype=_BF16, device=u.device) if dy is None else dy.contiguous()
        du, ddelta, dA, dB, dC, dD, dz, dbias, dh0 = selective_scan_bwd(
            u, delta, A, B, C, dy, D=D, z=z, delta_bias=delta_bias, delta_softplus=softplus, initial_state=h0,
            dfinal=None if dfinal is None else dfinal.contiguous(), cu_seqlens=cu, saved=saved)
        return du, ddelta, dA, dB, dC, dD, dz, dbias, dh0, None, None, None


def _differentiated(tensors):
    """Whether one of the tensors asks for gradients or carries a forward-mode tangent (which the autograd function refuses)."""
    tensors = [t for t in tensors if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        return True
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def selective_scan(u, delta, A, B, C, *, D=None, z=None, delta_bias=None, delta_softplus=True, initial_state=None,
                   output_final_state=False, cu_seqlens=None):
    """Differentiable selective scan (see :func:`selective_scan_fwd`): ``(y, final_state or None)``. Reverse mode only."""
    if not _differentiated((u, delta, A, B, C, D, z, delta_bias, initial_state)):
        return selective_scan_fwd(u, delta, A, B, C, D=D, z=z, delta_bias=delta_bias, delta_softplus=delta_softplus,
                                  initial_state=initial_state, output_final_state=output_final_state, cu_seqlens=cu_seqlens)
    return SelectiveScan.apply(u, delta, A, B, C, D, z, delta_bias, initial_state, delta_softplus, output_final_state, cu_seqlens)

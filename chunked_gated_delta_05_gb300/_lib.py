"""ctypes view of libgdn's C ABI (include/gdn.h): struct layouts, loading and error mapping."""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

GDN_OK, GDN_EINVAL, GDN_EUNSUPPORTED, GDN_ECUDA, GDN_ETIMEOUT, GDN_ERANGE = 0, 1, 2, 3, 4, 5

c_int, c_float, c_size_t, c_void_p = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
c_ll = ctypes.c_longlong


class Desc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("H", c_int), ("K", c_int), ("V", c_int),
                ("chunk_size", c_int), ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)),
                ("num_seqs", c_int), ("scale", c_float), ("use_qk_l2norm", c_int),
                ("use_beta_sigmoid", c_int), ("output_final_state", c_int), ("num_k_heads", c_int),
                ("use_gate_in_kernel", c_int), ("lower_bound", c_float)]


class FwdArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("g", c_void_p),
                ("beta", c_void_p), ("initial_state", c_void_p), ("o", c_void_p),
                ("final_state", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("status", c_void_p), ("saved", c_void_p), ("saved_bytes", c_size_t),
                ("A_log", c_void_p), ("dt_bias", c_void_p)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("g", c_void_p),
                ("beta", c_void_p), ("initial_state", c_void_p), ("dO", c_void_p),
                ("dht", c_void_p), ("dq", c_void_p), ("dk", c_void_p), ("dv", c_void_p),
                ("dbeta", c_void_p), ("dg", c_void_p), ("dh0", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("status", c_void_p),
                ("saved", c_void_p), ("saved_bytes", c_size_t), ("A_log", c_void_p), ("dt_bias", c_void_p),
                ("dA_log", c_void_p), ("ddt_bias", c_void_p)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("C", c_int), ("W", c_int), ("dilation", c_int),
                ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)), ("num_seqs", c_int), ("activation", c_int)]


class ConvFwdArgs(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("weight", c_void_p), ("bias", c_void_p), ("halo", c_void_p),
                ("y", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t)]


class ConvBwdArgs(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("weight", c_void_p), ("bias", c_void_p), ("halo", c_void_p),
                ("dy", c_void_p), ("dx", c_void_p), ("dweight", c_void_p), ("dbias", c_void_p),
                ("dhalo", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t)]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", c_ll), ("width", c_int), ("eps", c_float), ("residual_scale", c_float),
                ("stream_kind", c_int), ("activation", c_int)]


class NormFwdArgs(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("residual", c_void_p), ("weight", c_void_p), ("y", c_void_p), ("stream", c_void_p)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("gate", c_void_p), ("weight", c_void_p), ("dy", c_void_p), ("dstream", c_void_p),
                ("dx", c_void_p), ("dgate", c_void_p), ("dresidual", c_void_p), ("dweight", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t)]


class ConvStepDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("C", c_int), ("W", c_int), ("dilation", c_int), ("activation", c_int),
                ("num_slots", c_int), ("x_stride", c_ll)]


class ConvStepArgs(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("weight", c_void_p), ("bias", c_void_p), ("state", c_void_p),
                ("state_indices", c_void_p), ("y", c_void_p), ("status", c_void_p)]


class StepDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("H", c_int), ("num_k_heads", c_int), ("num_slots", c_int), ("scale", c_float),
                ("use_qk_l2norm", c_int), ("use_beta_sigmoid", c_int), ("use_gate_in_kernel", c_int),
                ("lower_bound", c_float), ("q_stride", c_ll), ("k_stride", c_ll), ("v_stride", c_ll)]


class StepArgs(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("g", c_void_p), ("beta", c_void_p),
                ("state", c_void_p), ("state_indices", c_void_p), ("o", c_void_p), ("A_log", c_void_p),
                ("dt_bias", c_void_p), ("status", c_void_p)]


class SscanDesc(ctypes.Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("D", c_int), ("N", c_int), ("G", c_int),
                ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)), ("num_seqs", c_int), ("delta_softplus", c_int),
                ("u_stride", c_ll), ("delta_stride", c_ll), ("z_stride", c_ll), ("B_stride", c_ll), ("C_stride", c_ll)]


class SscanFwdArgs(ctypes.Structure):
    _fields_ = [("u", c_void_p), ("delta", c_void_p), ("A", c_void_p), ("Bm", c_void_p), ("Cm", c_void_p),
                ("D", c_void_p), ("delta_bias", c_void_p), ("z", c_void_p), ("initial_state", c_void_p),
                ("y", c_void_p), ("final_state", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("saved", c_void_p), ("saved_bytes", c_size_t)]


class SscanBwdArgs(ctypes.Structure):
    _fields_ = [("u", c_void_p), ("delta", c_void_p), ("A", c_void_p), ("Bm", c_void_p), ("Cm", c_void_p),
                ("D", c_void_p), ("delta_bias", c_void_p), ("z", c_void_p), ("initial_state", c_void_p),
                ("dy", c_void_p), ("dfinal", c_void_p), ("du", c_void_p), ("ddelta", c_void_p), ("dA", c_void_p),
                ("dB", c_void_p), ("dC", c_void_p), ("dD", c_void_p), ("ddelta_bias", c_void_p), ("dz", c_void_p),
                ("dh0", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("saved", c_void_p),
                ("saved_bytes", c_size_t)]


class SscanStepArgs(ctypes.Structure):
    _fields_ = [("u", c_void_p), ("delta", c_void_p), ("A", c_void_p), ("Bm", c_void_p), ("Cm", c_void_p),
                ("D", c_void_p), ("delta_bias", c_void_p), ("z", c_void_p), ("state", c_void_p),
                ("state_indices", c_void_p), ("num_slots", c_int), ("y", c_void_p), ("status", c_void_p)]


def _call(desc, args):
    return ([ctypes.POINTER(desc), ctypes.POINTER(args), c_void_p], c_int)


def packer(cls):
    """``pack(*fields) -> bytes`` of a structure with the C layout of ``cls`` (pointers as integers). Building the bytes
    takes a fraction of the time of filling a ctypes structure, which is much of a small call's."""
    codes = {c_int: "i", c_float: "f", c_size_t: "N", c_ll: "q", c_void_p: "P"}
    fmt = struct.Struct("@" + "".join(codes.get(t, "P") for _, t in cls._fields_) + "0P")
    if fmt.size != ctypes.sizeof(cls):
        raise RuntimeError(f"packed layout of {cls.__name__} differs from its C layout")
    return fmt.pack


# Every symbol include/gdn.h declares, with its ctypes signature.
SIGNATURES = {
    "gdn_strerror": ([c_int], ctypes.c_char_p),
    "gdn_last_error": ([], ctypes.c_char_p),
    "gdn_device_supported": ([c_int], c_int),
    "gdn_fwd_workspace_size": ([ctypes.POINTER(Desc)], c_size_t),
    "gdn_bwd_workspace_size": ([ctypes.POINTER(Desc)], c_size_t),
    "kda_fwd_workspace_size": ([ctypes.POINTER(Desc)], c_size_t),
    "kda_bwd_workspace_size": ([ctypes.POINTER(Desc)], c_size_t),
    "gdn_saved_size": ([ctypes.POINTER(Desc)], c_size_t),
    "kda_saved_size": ([ctypes.POINTER(Desc)], c_size_t),
    "gdn_fwd": ([ctypes.POINTER(Desc), ctypes.POINTER(FwdArgs), c_void_p], c_int),
    "gdn_bwd": ([ctypes.POINTER(Desc), ctypes.POINTER(BwdArgs), c_void_p], c_int),
    "kda_fwd": ([ctypes.POINTER(Desc), ctypes.POINTER(FwdArgs), c_void_p], c_int),
    "kda_bwd": ([ctypes.POINTER(Desc), ctypes.POINTER(BwdArgs), c_void_p], c_int),
    "gdn_fwd_noalloc": ([ctypes.POINTER(Desc), ctypes.POINTER(FwdArgs), c_void_p], c_int),
    "gdn_fwd_noalloc_capacity": ([], c_size_t),
    "gdn_set_chain_segment": ([c_int], c_int),
    "gdn_chain_plan": ([ctypes.POINTER(Desc), ctypes.POINTER(c_int), ctypes.POINTER(c_int)], c_int),
    "gdn_set_head_groups": ([c_int], c_int),
    "gdn_conv_fwd_workspace_size": ([ctypes.POINTER(ConvDesc)], c_size_t),
    "gdn_conv_bwd_workspace_size": ([ctypes.POINTER(ConvDesc)], c_size_t),
    "gdn_conv_fwd": ([ctypes.POINTER(ConvDesc), ctypes.POINTER(ConvFwdArgs), c_void_p], c_int),
    "gdn_conv_bwd": ([ctypes.POINTER(ConvDesc), ctypes.POINTER(ConvBwdArgs), c_void_p], c_int),
    "gdn_conv_state": _call(ConvDesc, ConvFwdArgs),
    "gdn_conv_step": _call(ConvStepDesc, ConvStepArgs),
    "gdn_norm_bwd_workspace_size": ([ctypes.POINTER(NormDesc)], c_size_t),
    "gdn_add_norm_fwd": _call(NormDesc, NormFwdArgs),
    "gdn_add_norm_bwd": _call(NormDesc, NormBwdArgs),
    "gdn_gated_norm_fwd": _call(NormDesc, NormFwdArgs),
    "gdn_gated_norm_bwd": _call(NormDesc, NormBwdArgs),
    "gdn_step": _call(StepDesc, StepArgs),
    "kda_step": _call(StepDesc, StepArgs),
    "gdn_sscan_fwd_workspace_size": ([ctypes.POINTER(SscanDesc)], c_size_t),
    "gdn_sscan_bwd_workspace_size": ([ctypes.POINTER(SscanDesc)], c_size_t),
    "gdn_sscan_saved_size": ([ctypes.POINTER(SscanDesc)], c_size_t),
    "gdn_sscan_fwd": _call(SscanDesc, SscanFwdArgs),
    "gdn_sscan_bwd": _call(SscanDesc, SscanBwdArgs),
    "gdn_sscan_step": _call(SscanDesc, SscanStepArgs),
    "gdn_timing_enable": ([c_int], c_int),
    "gdn_timing_kinds": ([], c_int),
    "gdn_timing_name": ([c_int], ctypes.c_char_p),
    "gdn_timing_read": ([c_int, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int)], c_int),
    "gdn_wait_selftest": ([c_void_p, ctypes.c_longlong, c_void_p, c_void_p], c_int),
}

_lock = threading.Lock()
_lib = None
_entries = {}


def entry(name: str):
    """The (desc, args, stream) entry point ``name``, taking packed structures (bytes) and the stream as an integer."""
    fn = _entries.get(name)
    if fn is None:
        fn = ctypes.CFUNCTYPE(c_int, c_void_p, c_void_p, c_void_p)((name, load()))
        _entries[name] = fn
    return fn


def size(name: str, desc: bytes) -> int:
    """What the size query ``name`` says of a packed description; raises where it is invalid (0)."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = ctypes.CFUNCTYPE(c_size_t, c_void_p)((name, load()))
    n = fn(desc)
    if n == 0:
        check(GDN_EINVAL)
    return n


def load(build_if_missing: bool = True):
    """Load libgdn.so (building it first when missing or stale). Raises if it cannot."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_missing:
                path = _build.build()
            else:
                path = _build.LIB
                if not os.path.exists(path):
                    raise RuntimeError("libgdn.so is not built; run chunked_gated_delta_05_gb300.build")
            lib = ctypes.CDLL(path)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(msg)
        self.code = code


def check(code: int) -> None:
    if code == GDN_OK:
        return
    lib = load()
    detail = lib.gdn_last_error().decode() or lib.gdn_strerror(code).decode()
    if code == GDN_EINVAL:
        raise ValueError(detail)
    raise GdnError(code, f"{lib.gdn_strerror(code).decode()}: {detail}")


def timing_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with CUDA events (profiling aid)."""
    check(load().gdn_timing_enable(int(bool(on))))


def timing_read() -> dict:
    """Per-kernel {name: (total_ms, launches)} since the last read; synchronizes the events."""
    lib = load()
    out = {}
    for kind in range(lib.gdn_timing_kinds()):
        ms = ctypes.c_double()
        n = c_int()
        check(lib.gdn_timing_read(kind, ctypes.byref(ms), ctypes.byref(n)))
        out[lib.gdn_timing_name(kind).decode()] = (ms.value, n.value)
    return out

"""causal_depthwise_conv1d_amd -- Python binding of libccv (the causal depthwise
conv1d forward for AMD gfx950).

Argument marshalling only: every step of the computation runs in the HIP kernels
behind the C ABI of ``include/ccv.h``; PyTorch provides device memory and
streams.  There is no CPU fallback: without the built library, or with tensors
that are not on a GPU, calls raise.

Low level (same names as the C ABI):
    ccv_fwd(args, stream=None), ccv_fwd_check(args), ccv_fwd_plan(args),
    ccv_update(args, stream=None), ccv_update_check(args), ccv_update_plan(args),
    ccv_bwd(args, stream=None), ccv_bwd_check(args), ccv_bwd_plan(args),
    ccv_bwd_workspace_size(args),
    ccv_status_str(code), ccv_abi_version()
    ccv_delta_fwd, ccv_delta_bwd, ccv_delta_update, ccv_linrec_fwd, ccv_linrec_bwd,
    ccv_linrec_update, ccv_norm_fwd, ccv_norm_bwd, ccv_group_norm_fwd, ccv_group_norm_bwd,
    ccv_rotary and
    ccv_seq_tables (args, stream=None), their ccv_*_check(args) and, where they need a
    workspace, ccv_*_workspace_size(args)
High level (the full-sequence contract of Ch.4 "Dao interface and source map",
section "Contract of the full-sequence interface"; and the update kernel of the
same page's section "Reading the source along the call chain"):
    causal_conv1d_fwd(x, weight, bias=None, seq_idx=None, initial_states=None,
                      return_final_states=False, final_states_out=None,
                      activation=None)
    causal_conv1d_update(x, conv_state, weight, bias=None, activation=None)
    causal_conv1d_bwd(x, weight, bias, dout, seq_idx=None, initial_states=None,
                      dfinal_states=None, activation=None, ...)
    causal_conv1d_fn(x, weight, bias=None, seq_idx=None, initial_states=None,
                     return_final_states=False, final_states_out=None, activation=None)
        (differentiable: a torch.autograd.Function over the forward and backward)
The operators of a gated linear-attention layer around the conv:
    gated_delta_rule_fwd(q, k, v, g, beta, scale=None, cu_seqlens=None,
                         initial_state=None, return_final_state=False, ...)
    gated_delta_rule_bwd(q, k, v, g, beta, dout, ...)
    gated_delta_rule_fn(...)            (differentiable)
    gated_delta_rule_update(q, k, v, g, beta, state, state_indices=None, ...)
    gated_linear_recurrence_fwd(x, g, cu_seqlens=None, initial_state=None,
                                return_final_state=False, normalize=False, ...)
    gated_linear_recurrence_bwd(x, g, dout, ...)
    gated_linear_recurrence_fn(...)     (differentiable)
    gated_linear_recurrence_update(x, g, state, state_indices=None, normalize=False, ...)
    layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, ...), layer_norm_bwd(...),
    layer_norm_fn(...)                  (differentiable)
    group_norm_fwd(x, num_groups, weight=None, bias=None, gate=None, activation=None, ...),
    group_norm_bwd(...), group_norm_fn(...)     (differentiable)
    rotary_fwd(q, k, positions, frequencies, interleaved=False, scale=1.0, ...),
    rotary_fn(...)                      (differentiable)
    rotary_frequencies(turned, base=10000.0, scaling=None, ...)     -> (frequencies, scale)
    sequence_tables(lengths, total)     -> (cu_seqlens, seq_idx, positions)
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libccv.so")
CALIB_LIB_PATH = os.path.join(_HERE, "libccv_calib.so")

CCV_ABI_VERSION = 1
CCV_F32, CCV_F16, CCV_BF16 = 0, 1, 2
CCV_ACT_NONE, CCV_ACT_SILU = 0, 1
CCV_PATH_NONE, CCV_PATH_CHANNEL_FIRST, CCV_PATH_CHANNEL_LAST, CCV_PATH_UPDATE, CCV_PATH_BACKWARD = 0, 1, 2, 3, 4
STATUS = {
    0: "CCV_OK", -1: "CCV_E_NULL", -2: "CCV_E_SHAPE", -3: "CCV_E_KSIZE", -4: "CCV_E_DTYPE",
    -5: "CCV_E_LAYOUT", -6: "CCV_E_UNSUPPORTED", -7: "CCV_E_ALIAS", -8: "CCV_E_HIP",
    -9: "CCV_E_INTERNAL", -10: "CCV_E_ABI", -11: "CCV_E_SCRATCH",
}
CCV_BWD_STATIC_SCRATCH_BYTES = 64 << 20
DTYPE_CODE = {torch.float32: CCV_F32, torch.float16: CCV_F16, torch.bfloat16: CCV_BF16}

_I64x2 = ctypes.c_int64 * 2
_I64x3 = ctypes.c_int64 * 3


class ccv_fwd_args_t(ctypes.Structure):
    """Mirror of ``ccv_fwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [
        ("struct_size", ctypes.c_int64),
        ("B", ctypes.c_int64), ("C", ctypes.c_int64), ("L", ctypes.c_int64),
        ("K", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("x_stride", _I64x3),
        ("weight", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("seq_idx", ctypes.c_void_p),
        ("initial_states", ctypes.c_void_p), ("init_stride", _I64x3),
        ("final_states_out", ctypes.c_void_p), ("final_stride", _I64x3),
        ("out", ctypes.c_void_p), ("out_stride", _I64x3),
    ]

    def __init__(self, **kw):
        super().__init__(**kw)
        self.struct_size = ctypes.sizeof(ccv_fwd_args_t)


class ccv_update_args_t(ctypes.Structure):
    """Mirror of ``ccv_update_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [
        ("struct_size", ctypes.c_int64),
        ("B", ctypes.c_int64), ("C", ctypes.c_int64), ("L", ctypes.c_int64),
        ("K", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("x_stride", _I64x3),
        ("weight", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("state", ctypes.c_void_p), ("state_stride", _I64x3),
        ("out", ctypes.c_void_p), ("out_stride", _I64x3),
    ]

    def __init__(self, **kw):
        super().__init__(**kw)
        self.struct_size = ctypes.sizeof(ccv_update_args_t)


class ccv_bwd_args_t(ctypes.Structure):
    """Mirror of ``ccv_bwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [
        ("struct_size", ctypes.c_int64),
        ("B", ctypes.c_int64), ("C", ctypes.c_int64), ("L", ctypes.c_int64),
        ("K", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("x_stride", _I64x3),
        ("weight", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("seq_idx", ctypes.c_void_p),
        ("initial_states", ctypes.c_void_p), ("init_stride", _I64x3),
        ("dout", ctypes.c_void_p), ("dout_stride", _I64x3),
        ("dfinal_states", ctypes.c_void_p), ("dfinal_stride", _I64x3),
        ("dx", ctypes.c_void_p), ("dx_stride", _I64x3),
        ("dweight", ctypes.c_void_p),
        ("dbias", ctypes.c_void_p),
        ("dinitial_states", ctypes.c_void_p), ("dinit_stride", _I64x3),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]

    def __init__(self, **kw):
        super().__init__(**kw)
        self.struct_size = ctypes.sizeof(ccv_bwd_args_t)


class ccv_plan_t(ctypes.Structure):
    """Mirror of ``ccv_plan_t`` in include/ccv.h."""
    _fields_ = [
        ("path", ctypes.c_int32), ("vector", ctypes.c_int32),
        ("elems_per_lane", ctypes.c_int32), ("unroll", ctypes.c_int32),
        ("grid", ctypes.c_int64), ("block", ctypes.c_int32), ("waves_per_group", ctypes.c_int32),
        ("work_items", ctypes.c_int64), ("span", ctypes.c_int64), ("channels_per_item", ctypes.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class _Args(ctypes.Structure):
    """A struct whose first field is its own size."""

    def __init__(self, **kw):
        super().__init__(**kw)
        self.struct_size = ctypes.sizeof(type(self))


def _strided(*names):
    """(pointer, three strides) field pairs."""
    out = []
    for n, s in names:
        out += [(n, ctypes.c_void_p), (s, _I64x3)]
    return out


_DELTA_SIZES = [("Hk", ctypes.c_int64), ("Hv", ctypes.c_int64), ("Dk", ctypes.c_int64), ("Dv", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32), ("beta_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]
_DELTA_INPUTS = _strided(("q", "q_stride"), ("k", "k_stride"), ("v", "v_stride"), ("g", "g_stride"),
                         ("beta", "beta_stride"))


class ccv_delta_fwd_args_t(_Args):
    """Mirror of ``ccv_delta_fwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("B", ctypes.c_int64), ("L", ctypes.c_int64), ("N", ctypes.c_int64),
                *_DELTA_SIZES, *_DELTA_INPUTS, ("cu_seqlens", ctypes.c_void_p),
                *_strided(("initial_state", "init_stride"), ("final_state", "final_stride"), ("out", "out_stride")),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ccv_delta_bwd_args_t(_Args):
    """Mirror of ``ccv_delta_bwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("B", ctypes.c_int64), ("L", ctypes.c_int64), ("N", ctypes.c_int64),
                *_DELTA_SIZES, *_DELTA_INPUTS, ("cu_seqlens", ctypes.c_void_p),
                *_strided(("initial_state", "init_stride"), ("dout", "dout_stride"), ("dfinal_state", "dfinal_stride"),
                          ("dq", "dq_stride"), ("dk", "dk_stride"), ("dv", "dv_stride"), ("dg", "dg_stride"),
                          ("dbeta", "dbeta_stride"), ("dinitial_state", "dinit_stride")),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ccv_delta_update_args_t(_Args):
    """Mirror of ``ccv_delta_update_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("B", ctypes.c_int64), ("L", ctypes.c_int64),
                ("slots", ctypes.c_int64), *_DELTA_SIZES, *_DELTA_INPUTS, ("state_indices", ctypes.c_void_p),
                *_strided(("state", "state_stride"), ("out", "out_stride"))]


class ccv_norm_fwd_args_t(_Args):
    """Mirror of ``ccv_norm_fwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("n0", ctypes.c_int64), ("n1", ctypes.c_int64),
                ("width", ctypes.c_int64), ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_stride", _I64x2), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_stride", _I64x2), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class ccv_norm_bwd_args_t(_Args):
    """Mirror of ``ccv_norm_bwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("n0", ctypes.c_int64), ("n1", ctypes.c_int64),
                ("width", ctypes.c_int64), ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_stride", _I64x2), ("weight", ctypes.c_void_p),
                ("dout", ctypes.c_void_p), ("dout_stride", _I64x2), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dx_stride", _I64x2), ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ccv_seq_tables_args_t(_Args):
    """Mirror of ``ccv_seq_tables_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("N", ctypes.c_int64), ("total", ctypes.c_int64),
                ("lengths", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("seq_idx", ctypes.c_void_p),
                ("positions", ctypes.c_void_p)]


_LINREC_SIZES = [("struct_size", ctypes.c_int64), ("B", ctypes.c_int64), ("L", ctypes.c_int64), ("C", ctypes.c_int64)]
_LINREC_TYPES = [("x_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32), ("normalize", ctypes.c_int32), ("reserved", ctypes.c_int32),
                 ("x", ctypes.c_void_p), ("x_stride", _I64x2), ("g", ctypes.c_void_p), ("g_stride", _I64x2)]


class ccv_linrec_fwd_args_t(_Args):
    """Mirror of ``ccv_linrec_fwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [*_LINREC_SIZES, ("N", ctypes.c_int64), *_LINREC_TYPES, ("cu_seqlens", ctypes.c_void_p),
                ("initial_state", ctypes.c_void_p), ("init_stride", ctypes.c_int64),
                ("final_state", ctypes.c_void_p), ("final_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride", _I64x2), ("carries", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ccv_linrec_bwd_args_t(_Args):
    """Mirror of ``ccv_linrec_bwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [*_LINREC_SIZES, ("N", ctypes.c_int64), *_LINREC_TYPES, ("cu_seqlens", ctypes.c_void_p),
                ("initial_state", ctypes.c_void_p), ("init_stride", ctypes.c_int64),
                ("dout", ctypes.c_void_p), ("dout_stride", _I64x2),
                ("dfinal_state", ctypes.c_void_p), ("dfinal_stride", ctypes.c_int64), ("carries", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dx_stride", _I64x2), ("dg", ctypes.c_void_p), ("dg_stride", _I64x2),
                ("dinitial_state", ctypes.c_void_p), ("dinit_stride", ctypes.c_int64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ccv_linrec_update_args_t(_Args):
    """Mirror of ``ccv_linrec_update_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [*_LINREC_SIZES, ("slots", ctypes.c_int64), *_LINREC_TYPES, ("state_indices", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("state_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("out_stride", _I64x2)]


class ccv_group_norm_fwd_args_t(_Args):
    """Mirror of ``ccv_group_norm_fwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("width", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class ccv_group_norm_bwd_args_t(_Args):
    """Mirror of ``ccv_group_norm_bwd_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("width", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64), ("dout", ctypes.c_void_p), ("dout_stride", ctypes.c_int64),
                ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dx_stride", ctypes.c_int64), ("dgate", ctypes.c_void_p), ("dgate_stride", ctypes.c_int64),
                ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class ccv_rotary_args_t(_Args):
    """Mirror of ``ccv_rotary_args_t`` in include/ccv.h (field order and types)."""
    _fields_ = [("struct_size", ctypes.c_int64), ("B", ctypes.c_int64), ("L", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hk", ctypes.c_int64), ("D", ctypes.c_int64), ("turned", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32), ("scale", ctypes.c_float),
                *_strided(("q", "q_stride"), ("k", "k_stride")), ("positions", ctypes.c_void_p), ("pos_stride", _I64x2),
                ("frequencies", ctypes.c_void_p), *_strided(("q_out", "q_out_stride"), ("k_out", "k_out_stride"))]


_LAYER_CALLS = {
    "ccv_delta_fwd": (ccv_delta_fwd_args_t, True), "ccv_delta_bwd": (ccv_delta_bwd_args_t, True),
    "ccv_delta_update": (ccv_delta_update_args_t, False), "ccv_norm_fwd": (ccv_norm_fwd_args_t, False),
    "ccv_norm_bwd": (ccv_norm_bwd_args_t, True), "ccv_seq_tables": (ccv_seq_tables_args_t, False),
    "ccv_linrec_fwd": (ccv_linrec_fwd_args_t, True), "ccv_linrec_bwd": (ccv_linrec_bwd_args_t, True),
    "ccv_linrec_update": (ccv_linrec_update_args_t, False),
    "ccv_group_norm_fwd": (ccv_group_norm_fwd_args_t, False), "ccv_group_norm_bwd": (ccv_group_norm_bwd_args_t, True),
    "ccv_rotary": (ccv_rotary_args_t, False),
}


class CcvError(RuntimeError):
    def __init__(self, status: int, where: str = "ccv_fwd"):
        self.status = status
        super().__init__(f"{where} failed: {STATUS.get(status, status)}")


class CcvArgumentError(CcvError, ValueError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libccv.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m causal_depthwise_conv1d_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(ccv_fwd_args_t)
        L.ccv_fwd.argtypes = [P, ctypes.c_void_p]
        L.ccv_fwd.restype = ctypes.c_int
        L.ccv_fwd_check.argtypes = [P]
        L.ccv_fwd_check.restype = ctypes.c_int
        L.ccv_fwd_plan.argtypes = [P, ctypes.POINTER(ccv_plan_t)]
        L.ccv_fwd_plan.restype = ctypes.c_int
        U = ctypes.POINTER(ccv_update_args_t)
        L.ccv_update.argtypes = [U, ctypes.c_void_p]
        L.ccv_update.restype = ctypes.c_int
        L.ccv_update_check.argtypes = [U]
        L.ccv_update_check.restype = ctypes.c_int
        L.ccv_update_plan.argtypes = [U, ctypes.POINTER(ccv_plan_t)]
        L.ccv_update_plan.restype = ctypes.c_int
        G = ctypes.POINTER(ccv_bwd_args_t)
        L.ccv_bwd.argtypes = [G, ctypes.c_void_p]
        L.ccv_bwd.restype = ctypes.c_int
        L.ccv_bwd_check.argtypes = [G]
        L.ccv_bwd_check.restype = ctypes.c_int
        L.ccv_bwd_plan.argtypes = [G, ctypes.POINTER(ccv_plan_t)]
        L.ccv_bwd_plan.restype = ctypes.c_int
        L.ccv_bwd_static.argtypes = [G, ctypes.c_void_p]
        L.ccv_bwd_static.restype = ctypes.c_int
        L.ccv_bwd_workspace_size.argtypes = [G]
        L.ccv_bwd_workspace_size.restype = ctypes.c_int64
        L.ccv_status_str.argtypes = [ctypes.c_int]
        L.ccv_status_str.restype = ctypes.c_char_p
        L.ccv_abi_version.argtypes = []
        L.ccv_abi_version.restype = ctypes.c_int
        for name, (args_t, workspace) in _LAYER_CALLS.items():
            A = ctypes.POINTER(args_t)
            call, check = getattr(L, name), getattr(L, name + "_check")
            call.argtypes, call.restype = [A, ctypes.c_void_p], ctypes.c_int
            check.argtypes, check.restype = [A], ctypes.c_int
            if workspace:
                size = getattr(L, name + "_workspace_size")
                size.argtypes, size.restype = [A], ctypes.c_int64
        if L.ccv_abi_version() != CCV_ABI_VERSION:
            raise RuntimeError("libccv ABI version mismatch")
        _lib = L
    return _lib


# ---- the C ABI, one to one ----------------------------------------------------------

def _stream_handle(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def ccv_fwd(args: ccv_fwd_args_t, stream=None) -> int:
    """Enqueue the forward on `stream` (a torch stream, a raw hipStream_t int, or None
    for torch's current stream).  Returns the status code."""
    return lib().ccv_fwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_fwd_check(args: ccv_fwd_args_t) -> int:
    return lib().ccv_fwd_check(ctypes.byref(args))


def ccv_fwd_plan(args: ccv_fwd_args_t):
    """(status, ccv_plan_t) without touching the device."""
    p = ccv_plan_t()
    st = lib().ccv_fwd_plan(ctypes.byref(args), ctypes.byref(p))
    return st, p


def ccv_update(args: ccv_update_args_t, stream=None) -> int:
    """Enqueue one update (decode) call on `stream`; returns the status code."""
    return lib().ccv_update(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_update_check(args: ccv_update_args_t) -> int:
    return lib().ccv_update_check(ctypes.byref(args))


def ccv_update_plan(args: ccv_update_args_t):
    """(status, ccv_plan_t) of an update call, without touching the device."""
    p = ccv_plan_t()
    st = lib().ccv_update_plan(ctypes.byref(args), ctypes.byref(p))
    return st, p


def ccv_bwd(args: ccv_bwd_args_t, stream=None) -> int:
    """Enqueue the backward (two kernels) on `stream`; returns the status code."""
    return lib().ccv_bwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_bwd_static(args: ccv_bwd_args_t, stream=None) -> int:
    """ccv_bwd with the partial sums in the library's fixed device array (no
    workspace, nothing allocated)."""
    return lib().ccv_bwd_static(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_bwd_check(args: ccv_bwd_args_t) -> int:
    return lib().ccv_bwd_check(ctypes.byref(args))


def ccv_bwd_plan(args: ccv_bwd_args_t):
    """(status, ccv_plan_t) of a backward call, without touching the device."""
    p = ccv_plan_t()
    st = lib().ccv_bwd_plan(ctypes.byref(args), ctypes.byref(p))
    return st, p


def ccv_bwd_workspace_size(args: ccv_bwd_args_t) -> int:
    """Workspace bytes the backward needs (>= 0), or a negative status."""
    return lib().ccv_bwd_workspace_size(ctypes.byref(args))


def ccv_status_str(status: int) -> str:
    return lib().ccv_status_str(int(status)).decode()


def ccv_abi_version() -> int:
    return lib().ccv_abi_version()


def ccv_delta_fwd(args: ccv_delta_fwd_args_t, stream=None) -> int:
    """Enqueue the gated delta rule's forward on `stream`; returns the status code."""
    return lib().ccv_delta_fwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_delta_fwd_check(args: ccv_delta_fwd_args_t) -> int:
    return lib().ccv_delta_fwd_check(ctypes.byref(args))


def ccv_delta_fwd_workspace_size(args: ccv_delta_fwd_args_t) -> int:
    """Workspace bytes the forward needs (>= 0), or a negative status."""
    return lib().ccv_delta_fwd_workspace_size(ctypes.byref(args))


def ccv_delta_bwd(args: ccv_delta_bwd_args_t, stream=None) -> int:
    """Enqueue the gated delta rule's backward on `stream`; returns the status code."""
    return lib().ccv_delta_bwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_delta_bwd_check(args: ccv_delta_bwd_args_t) -> int:
    return lib().ccv_delta_bwd_check(ctypes.byref(args))


def ccv_delta_bwd_workspace_size(args: ccv_delta_bwd_args_t) -> int:
    """Workspace bytes the backward needs (>= 0), or a negative status."""
    return lib().ccv_delta_bwd_workspace_size(ctypes.byref(args))


def ccv_delta_update(args: ccv_delta_update_args_t, stream=None) -> int:
    """Enqueue new steps against cached states on `stream`; returns the status code."""
    return lib().ccv_delta_update(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_delta_update_check(args: ccv_delta_update_args_t) -> int:
    return lib().ccv_delta_update_check(ctypes.byref(args))


def ccv_norm_fwd(args: ccv_norm_fwd_args_t, stream=None) -> int:
    """Enqueue layer norm on `stream`; returns the status code."""
    return lib().ccv_norm_fwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_norm_fwd_check(args: ccv_norm_fwd_args_t) -> int:
    return lib().ccv_norm_fwd_check(ctypes.byref(args))


def ccv_norm_bwd(args: ccv_norm_bwd_args_t, stream=None) -> int:
    """Enqueue layer norm's backward on `stream`; returns the status code."""
    return lib().ccv_norm_bwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_norm_bwd_check(args: ccv_norm_bwd_args_t) -> int:
    return lib().ccv_norm_bwd_check(ctypes.byref(args))


def ccv_norm_bwd_workspace_size(args: ccv_norm_bwd_args_t) -> int:
    """Workspace bytes the backward needs (>= 0), or a negative status."""
    return lib().ccv_norm_bwd_workspace_size(ctypes.byref(args))


def ccv_seq_tables(args: ccv_seq_tables_args_t, stream=None) -> int:
    """Enqueue the tables of a packed row on `stream`; returns the status code."""
    return lib().ccv_seq_tables(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_seq_tables_check(args: ccv_seq_tables_args_t) -> int:
    return lib().ccv_seq_tables_check(ctypes.byref(args))


def ccv_linrec_fwd(args: ccv_linrec_fwd_args_t, stream=None) -> int:
    """Enqueue the gated linear recurrence's forward on `stream`; returns the status code."""
    return lib().ccv_linrec_fwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_linrec_fwd_check(args: ccv_linrec_fwd_args_t) -> int:
    return lib().ccv_linrec_fwd_check(ctypes.byref(args))


def ccv_linrec_fwd_workspace_size(args: ccv_linrec_fwd_args_t) -> int:
    """Workspace bytes the forward needs (>= 0), or a negative status."""
    return lib().ccv_linrec_fwd_workspace_size(ctypes.byref(args))


def ccv_linrec_bwd(args: ccv_linrec_bwd_args_t, stream=None) -> int:
    """Enqueue the gated linear recurrence's backward on `stream`; returns the status code."""
    return lib().ccv_linrec_bwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_linrec_bwd_check(args: ccv_linrec_bwd_args_t) -> int:
    return lib().ccv_linrec_bwd_check(ctypes.byref(args))


def ccv_linrec_bwd_workspace_size(args: ccv_linrec_bwd_args_t) -> int:
    """Workspace bytes the backward needs (>= 0), or a negative status."""
    return lib().ccv_linrec_bwd_workspace_size(ctypes.byref(args))


def ccv_linrec_update(args: ccv_linrec_update_args_t, stream=None) -> int:
    """Enqueue new steps against cached states on `stream`; returns the status code."""
    return lib().ccv_linrec_update(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_linrec_update_check(args: ccv_linrec_update_args_t) -> int:
    return lib().ccv_linrec_update_check(ctypes.byref(args))


def ccv_group_norm_fwd(args: ccv_group_norm_fwd_args_t, stream=None) -> int:
    """Enqueue group norm on `stream`; returns the status code."""
    return lib().ccv_group_norm_fwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_group_norm_fwd_check(args: ccv_group_norm_fwd_args_t) -> int:
    return lib().ccv_group_norm_fwd_check(ctypes.byref(args))


def ccv_group_norm_bwd(args: ccv_group_norm_bwd_args_t, stream=None) -> int:
    """Enqueue group norm's backward on `stream`; returns the status code."""
    return lib().ccv_group_norm_bwd(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_group_norm_bwd_check(args: ccv_group_norm_bwd_args_t) -> int:
    return lib().ccv_group_norm_bwd_check(ctypes.byref(args))


def ccv_group_norm_bwd_workspace_size(args: ccv_group_norm_bwd_args_t) -> int:
    """Workspace bytes the backward needs (>= 0), or a negative status."""
    return lib().ccv_group_norm_bwd_workspace_size(ctypes.byref(args))


def ccv_rotary(args: ccv_rotary_args_t, stream=None) -> int:
    """Enqueue rotary positions on `stream`; returns the status code."""
    return lib().ccv_rotary(ctypes.byref(args), ctypes.c_void_p(_stream_handle(stream)))


def ccv_rotary_check(args: ccv_rotary_args_t) -> int:
    return lib().ccv_rotary_check(ctypes.byref(args))


# ---- tensors -> args -------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _strides3(t: Optional[torch.Tensor]):
    return _I64x3(*(t.stride() if t is not None else (0, 0, 0)))


def _contiguous_ids(seq_idx):
    """The C ABI reads seq_idx as a contiguous [B, L] array: refuse any other layout
    (a view with other strides would be read as different ids)."""
    if seq_idx is not None and not seq_idx.is_contiguous():
        raise ValueError("seq_idx must be contiguous [B, L] for the C ABI; call .contiguous() first")
    return seq_idx


def make_args(x, weight, out, bias=None, seq_idx=None, initial_states=None,
              final_states_out=None, activation=None) -> ccv_fwd_args_t:
    """Fill a ccv_fwd_args_t from tensors (no checks beyond dtype codes and a
    contiguous seq_idx)."""
    _contiguous_ids(seq_idx)
    B, C, L = x.shape
    a = ccv_fwd_args_t()
    a.B, a.C, a.L = B, C, L
    a.K = weight.shape[1]
    a.activation = CCV_ACT_SILU if activation in ("silu", "swish") else CCV_ACT_NONE
    a.x_dtype = DTYPE_CODE[x.dtype]
    a.w_dtype = DTYPE_CODE[weight.dtype]
    a.x, a.x_stride = _ptr(x), _strides3(x)
    a.weight = _ptr(weight)
    a.bias = _ptr(bias)
    a.seq_idx = _ptr(seq_idx)
    a.initial_states, a.init_stride = _ptr(initial_states), _strides3(initial_states)
    a.final_states_out, a.final_stride = _ptr(final_states_out), _strides3(final_states_out)
    a.out, a.out_stride = _ptr(out), _strides3(out)
    return a


def make_update_args(x, weight, state, out, bias=None, activation=None) -> ccv_update_args_t:
    """Fill a ccv_update_args_t from tensors: x and out [B, C, L], state [B, C, K-1]."""
    B, C, L = x.shape
    a = ccv_update_args_t()
    a.B, a.C, a.L = B, C, L
    a.K = weight.shape[1]
    a.activation = CCV_ACT_SILU if activation in ("silu", "swish") else CCV_ACT_NONE
    a.x_dtype = DTYPE_CODE[x.dtype]
    a.w_dtype = DTYPE_CODE[weight.dtype]
    a.x, a.x_stride = _ptr(x), _strides3(x)
    a.weight = _ptr(weight)
    a.bias = _ptr(bias)
    a.state, a.state_stride = _ptr(state), _strides3(state)
    a.out, a.out_stride = _ptr(out), _strides3(out)
    return a


def _raise(status: int, where: str = "ccv_fwd"):
    if status == 0:
        return
    if status == -8:
        raise CcvError(status, where)
    raise CcvArgumentError(status, where)


def empty_like_layout(x: torch.Tensor) -> torch.Tensor:
    """A new [B, C, L] tensor with x's dtype, device and unit-stride dimension."""
    B, C, L = x.shape
    if x.stride(2) == 1 or L <= 1 and x.stride(1) != 1:
        return torch.empty(B, C, L, dtype=x.dtype, device=x.device)
    return torch.empty(B, L, C, dtype=x.dtype, device=x.device).transpose(1, 2)


def causal_conv1d_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                      seq_idx: Optional[torch.Tensor] = None,
                      initial_states: Optional[torch.Tensor] = None,
                      return_final_states: bool = False,
                      final_states_out: Optional[torch.Tensor] = None,
                      activation: Optional[str] = None, out: Optional[torch.Tensor] = None,
                      info: Optional[dict] = None):
    """Causal depthwise conv1d forward on the GPU.

    x [B, C, L] (unit stride in time or in channels; any other strides are copied to
    contiguous first and ``info["x_copied"]`` says so), weight [C, K] (oldest ->
    current), bias [C] (weight dtype), seq_idx int32 [B, L], initial_states
    [B, C, K-1] (x dtype).  Returns out [B, C, L] in x's dtype and layout, or
    (out, final_states) when return_final_states.  final_states is [B, C, K-1] with
    channel stride 1 unless ``final_states_out`` provides the storage.
    """
    if activation not in (None, "silu", "swish"):
        raise ValueError(f"activation must be None, 'silu' or 'swish', not {activation!r}")
    if final_states_out is not None and not return_final_states:
        raise ValueError("final_states_out given but return_final_states is False")
    if x.dim() != 3 or weight.dim() != 2 or weight.shape[0] != x.shape[1]:
        raise ValueError("expected x [B, C, L] and weight [C, K]")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor (there is no CPU path)")
    for name, t in (("weight", weight), ("bias", bias), ("seq_idx", seq_idx),
                    ("initial_states", initial_states), ("final_states_out", final_states_out),
                    ("out", out)):
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} must be on {x.device}")
    B, C, L = x.shape
    K = weight.shape[1]
    copied = False
    if not (x.stride(2) == 1 or x.stride(1) == 1 or L <= 1 or C <= 1):
        x = x.contiguous()          # neither time nor channels unit-stride
        copied = True
    weight = weight.contiguous()
    if bias is not None:
        if bias.dtype != weight.dtype:
            raise ValueError("bias must have the weight's dtype")
        bias = bias.contiguous()
    if seq_idx is not None:
        if seq_idx.dtype != torch.int32 or tuple(seq_idx.shape) != (B, L):
            raise ValueError("seq_idx must be int32 [B, L]")
        seq_idx = seq_idx.contiguous()
    if initial_states is not None:
        if initial_states.dtype != x.dtype or tuple(initial_states.shape) != (B, C, K - 1):
            raise ValueError("initial_states must be [B, C, K-1] in x's dtype")
    fs = None
    if return_final_states:
        if final_states_out is not None:
            if final_states_out.dtype != x.dtype or tuple(final_states_out.shape) != (B, C, K - 1):
                raise ValueError("final_states_out must be [B, C, K-1] in x's dtype")
            fs = final_states_out
        else:
            fs = torch.empty(B, K - 1, C, dtype=x.dtype, device=x.device).transpose(1, 2)
    if out is None:
        out = empty_like_layout(x)
    elif out.dtype != x.dtype or tuple(out.shape) != (B, C, L):
        raise ValueError("out must be [B, C, L] in x's dtype")
    args = make_args(x, weight, out, bias, seq_idx, initial_states, fs, activation)
    with torch.cuda.device(x.device):
        st = ccv_fwd(args)
    _raise(st)
    if info is not None:
        info["x_copied"] = copied
    return (out, fs) if return_final_states else out


def plan_for(x, weight, out=None, **kw) -> dict:
    """The launch causal_conv1d_fwd would make for these tensors (no device work)."""
    if out is None:
        out = empty_like_layout(x)
    st, p = ccv_fwd_plan(make_args(x, weight, out, **kw))
    _raise(st)
    return p.as_dict()


def causal_conv1d_update(x: torch.Tensor, conv_state: torch.Tensor, weight: torch.Tensor,
                         bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One update (decode) call on the GPU: convolve the new steps x against the
    history in ``conv_state`` and advance ``conv_state`` in place.

    x [B, C] (one step) or [B, C, L]; conv_state [B, C, K-1] in x's dtype, time
    ascending (the last K-1 inputs seen so far); weight [C, K] (oldest -> current);
    bias [C] in the weight's dtype.  Any strides are used as they are.  Returns out
    with x's shape and dtype, allocated with x's unit-stride dimension.  Afterwards conv_state holds the last K-1 inputs of
    (old state followed by x), exactly as ``causal_conv1d_fwd`` would return them as
    final states.
    """
    if activation not in (None, "silu", "swish"):
        raise ValueError(f"activation must be None, 'silu' or 'swish', not {activation!r}")
    one_step = x.dim() == 2
    x3 = x.unsqueeze(2) if one_step else x
    if x3.dim() != 3 or weight.dim() != 2 or weight.shape[0] != x3.shape[1]:
        raise ValueError("expected x [B, C] or [B, C, L] and weight [C, K]")
    if not x3.is_cuda:
        raise ValueError("x must be a GPU tensor (there is no CPU path)")
    for name, t in (("conv_state", conv_state), ("weight", weight), ("bias", bias), ("out", out)):
        if t is not None and t.device != x3.device:
            raise ValueError(f"{name} must be on {x3.device}")
    B, C, L = x3.shape
    K = weight.shape[1]
    if conv_state.dtype != x3.dtype or tuple(conv_state.shape) != (B, C, K - 1):
        raise ValueError("conv_state must be [B, C, K-1] in x's dtype")
    weight = weight.contiguous()
    if bias is not None:
        if bias.dtype != weight.dtype:
            raise ValueError("bias must have the weight's dtype")
        bias = bias.contiguous()
    if out is None:
        out3 = empty_like_layout(x3)
    else:
        if out.dtype != x3.dtype or tuple(out.shape) != tuple(x.shape):
            raise ValueError("out must have x's shape and dtype")
        out3 = out.unsqueeze(2) if one_step else out
    args = make_update_args(x3, weight, conv_state, out3, bias, activation)
    with torch.cuda.device(x3.device):
        st = ccv_update(args)
    _raise(st, "ccv_update")
    return out3.squeeze(2) if one_step else out3


def update_plan_for(x, conv_state, weight, bias=None, activation=None) -> dict:
    """The launch causal_conv1d_update would make for these tensors (no device work)."""
    x3 = x.unsqueeze(2) if x.dim() == 2 else x
    out = empty_like_layout(x3)
    st, p = ccv_update_plan(make_update_args(x3, weight.contiguous(), conv_state, out, bias, activation))
    _raise(st, "ccv_update")
    return p.as_dict()


def make_bwd_args(x, weight, bias, dout, dx, dweight, dbias=None, seq_idx=None, initial_states=None,
                  dfinal_states=None, dinitial_states=None, activation=None,
                  workspace=None) -> ccv_bwd_args_t:
    """Fill a ccv_bwd_args_t from tensors (no checks beyond dtype codes and a
    contiguous seq_idx)."""
    _contiguous_ids(seq_idx)
    B, C, L = x.shape
    a = ccv_bwd_args_t()
    a.B, a.C, a.L = B, C, L
    a.K = weight.shape[1]
    a.activation = CCV_ACT_SILU if activation in ("silu", "swish") else CCV_ACT_NONE
    a.x_dtype = DTYPE_CODE[x.dtype]
    a.w_dtype = DTYPE_CODE[weight.dtype]
    a.x, a.x_stride = _ptr(x), _strides3(x)
    a.weight, a.bias, a.seq_idx = _ptr(weight), _ptr(bias), _ptr(seq_idx)
    a.initial_states, a.init_stride = _ptr(initial_states), _strides3(initial_states)
    a.dout, a.dout_stride = _ptr(dout), _strides3(dout)
    a.dfinal_states, a.dfinal_stride = _ptr(dfinal_states), _strides3(dfinal_states)
    a.dx, a.dx_stride = _ptr(dx), _strides3(dx)
    a.dweight, a.dbias = _ptr(dweight), _ptr(dbias)
    a.dinitial_states, a.dinit_stride = _ptr(dinitial_states), _strides3(dinitial_states)
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return a


def causal_conv1d_bwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                      dout: torch.Tensor, seq_idx: Optional[torch.Tensor] = None,
                      initial_states: Optional[torch.Tensor] = None,
                      dfinal_states: Optional[torch.Tensor] = None,
                      activation: Optional[str] = None, dx: Optional[torch.Tensor] = None,
                      return_dinitial_states: bool = False, want_dbias: Optional[bool] = None):
    """Gradients of causal_conv1d_fwd on the GPU: (dx, dweight, dbias, dinitial_states).

    dout [B, C, L] and dfinal_states [B, C, K-1] are in x's dtype; dx is allocated
    in x's layout unless given (any strides); dweight [C, K] and dbias [C] come back
    in the weight's dtype (accumulated in fp32); dbias is None unless a bias was
    given (or want_dbias); dinitial_states [B, C, K-1] only with
    return_dinitial_states (it needs initial_states).  The fp32 workspace for the
    parameter sums is allocated here, through torch.
    """
    if activation not in (None, "silu", "swish"):
        raise ValueError(f"activation must be None, 'silu' or 'swish', not {activation!r}")
    if x.dim() != 3 or weight.dim() != 2 or weight.shape[0] != x.shape[1]:
        raise ValueError("expected x [B, C, L] and weight [C, K]")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor (there is no CPU path)")
    B, C, L = x.shape
    K = weight.shape[1]
    for name, t in (("weight", weight), ("bias", bias), ("dout", dout), ("seq_idx", seq_idx),
                    ("initial_states", initial_states), ("dfinal_states", dfinal_states), ("dx", dx)):
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} must be on {x.device}")
    if dout.dtype != x.dtype or tuple(dout.shape) != (B, C, L):
        raise ValueError("dout must be [B, C, L] in x's dtype")
    if dfinal_states is not None and (dfinal_states.dtype != x.dtype or tuple(dfinal_states.shape) != (B, C, K - 1)):
        raise ValueError("dfinal_states must be [B, C, K-1] in x's dtype")
    if initial_states is not None and (initial_states.dtype != x.dtype
                                       or tuple(initial_states.shape) != (B, C, K - 1)):
        raise ValueError("initial_states must be [B, C, K-1] in x's dtype")
    if return_dinitial_states and initial_states is None:
        raise ValueError("dinitial_states needs initial_states")
    if seq_idx is not None:
        if seq_idx.dtype != torch.int32 or tuple(seq_idx.shape) != (B, L):
            raise ValueError("seq_idx must be int32 [B, L]")
        seq_idx = seq_idx.contiguous()
    weight = weight.contiguous()
    if bias is not None:
        if bias.dtype != weight.dtype:
            raise ValueError("bias must have the weight's dtype")
        bias = bias.contiguous()
    if dx is None:
        dx = empty_like_layout(x)
    elif dx.dtype != x.dtype or tuple(dx.shape) != (B, C, L):
        raise ValueError("dx must be [B, C, L] in x's dtype")
    dweight = torch.empty(C, K, dtype=weight.dtype, device=x.device)
    want_db = (bias is not None) if want_dbias is None else want_dbias
    dbias = torch.empty(C, dtype=weight.dtype, device=x.device) if want_db else None
    dinit = (torch.empty(B, K - 1, C, dtype=x.dtype, device=x.device).transpose(1, 2)
             if return_dinitial_states else None)
    args = make_bwd_args(x, weight, bias, dout, dx, dweight, dbias, seq_idx, initial_states,
                         dfinal_states, dinit, activation)
    ws = ccv_bwd_workspace_size(args)
    _raise(int(ws) if ws < 0 else 0, "ccv_bwd")
    workspace = torch.empty(max(int(ws), 16), dtype=torch.uint8, device=x.device)
    args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel()
    with torch.cuda.device(x.device):
        st = ccv_bwd(args)
    _raise(st, "ccv_bwd")
    return dx, dweight, dbias, dinit


class _CausalConv1dFn(torch.autograd.Function):
    """Forward and backward through the C ABI.  Saves x, weight, bias,
    initial_states and seq_idx (Ch.4 "Dao interface and source map", section "How
    autograd links forward and backward"); z is recomputed in the backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, seq_idx, initial_states, return_final_states, final_states_out,
                activation):
        res = causal_conv1d_fwd(x, weight, bias, seq_idx, initial_states, return_final_states,
                                final_states_out, activation)
        ctx.save_for_backward(x, weight, bias, seq_idx, initial_states)
        ctx.activation = activation
        ctx.return_final_states = return_final_states
        return res

    @staticmethod
    def backward(ctx, dout, *rest):
        x, weight, bias, seq_idx, initial_states = ctx.saved_tensors
        dfs = rest[0] if ctx.return_final_states and rest else None
        if dout is None:
            dout = torch.zeros_like(x)
        dout = dout.to(x.dtype)
        if dfs is not None:
            dfs = dfs.to(x.dtype)
        want_dinit = initial_states is not None and ctx.needs_input_grad[4]
        dx, dw, db, dinit = causal_conv1d_bwd(
            x, weight, bias, dout, seq_idx, initial_states, dfs, ctx.activation,
            return_dinitial_states=want_dinit, want_dbias=bias is not None and ctx.needs_input_grad[2])
        return dx, dw, db, None, dinit, None, None, None


def causal_conv1d_fn(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     seq_idx: Optional[torch.Tensor] = None,
                     initial_states: Optional[torch.Tensor] = None, return_final_states: bool = False,
                     final_states_out: Optional[torch.Tensor] = None, activation: Optional[str] = None):
    """Differentiable causal depthwise conv1d (the full-sequence contract of
    causal_conv1d_fwd, with gradients for x, weight, bias and initial_states through
    causal_conv1d_bwd)."""
    return _CausalConv1dFn.apply(x, weight, bias, seq_idx, initial_states, return_final_states,
                                 final_states_out, activation)


# ---- calls of the layer's operators ------------------------------------------------------------
#
# A small call's cost is the host's, so these fill their args struct in one go: the values, in
# the order of the struct's fields, packed to its layout, which the library takes by address.

CCV_LINREC_CHUNK = 128       # steps between the states that gated_linear_recurrence_fwd leaves for its backward

_FORMAT = {ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_void_p: "P", _I64x2: "2q", _I64x3: "3q"}


_pack_workspace = struct.Struct("@Pq").pack      # the last two fields of every call that takes one


class _Call:
    """One C entry point with its packed args."""

    def __init__(self, name):
        self.name = name
        args_t, self.workspace = _LAYER_CALLS[name]
        self.pack = struct.Struct("@" + "".join(_FORMAT[t] for _, t in args_t._fields_)).pack
        self.size = ctypes.sizeof(args_t)
        self.fn = self.ws_fn = None

    def bind(self):
        L = lib()
        fn = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, ctypes.c_void_p)((self.name, L))
        if self.workspace:
            self.ws_fn = ctypes.CFUNCTYPE(ctypes.c_int64, ctypes.c_char_p)((self.name + "_workspace_size", L))
        self.fn = fn

    def __call__(self, device, *values):
        """Enqueue on the current stream of the device (or of its index); the workspace, which follows the
        values in the struct, is allocated here, through torch."""
        if self.fn is None:
            self.bind()
        if self.workspace:
            args = self.pack(self.size, *values, 0, 0)
            ws = self.ws_fn(args)
            if ws < 0:
                _raise(int(ws), self.name)
            buf = torch.empty(ws or 16, dtype=torch.uint8, device=device)
            args = args[:-16] + _pack_workspace(buf.data_ptr(), ws or 16)
        else:
            args = self.pack(self.size, *values)
        index = device if type(device) is int else device.index
        if index == _current_device():
            st = self.fn(args, _raw_stream(index))
        else:
            with torch.cuda.device(device):
                st = self.fn(args, _raw_stream(index))
        if st:
            _raise(st, self.name)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
# of a process that has tensors on a GPU, and so has initialised it
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_CALLS = {name: _Call(name) for name in _LAYER_CALLS}


def _p(t):
    return 0 if t is None else t.data_ptr()


def _at(t):
    """A tensor's address and its three leading strides, as consecutive values."""
    if t is None:
        return (0, 0, 0, 0)
    s = t.stride()
    return (t.data_ptr(), s[0], s[1], s[2])


_new_version = torch.autograd.graph.increment_version


def _written(*given):
    """Tells autograd that a call wrote the caller's own tensors, which it does by address: a backward
    that has kept one of them then raises, as after torch's in-place operators."""
    for t in given:
        if t is not None:
            _new_version(t)


def _step_at(t):
    """The same of a tensor without the dimension of steps."""
    s = t.stride()
    return (t.data_ptr(), s[0], 0, s[1])


class _FirstOrder(torch.autograd.Function):
    """Gradients made by a C call, passed on as they are: nothing records how they depend on the
    inputs, so differentiating them again has to raise, where they would pass for constants."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tuple(t.view_as(t) for t in tensors[count:])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no second derivative: its gradients cannot be differentiated again")


def _first_order(name, inputs, grads):
    """A backward's gradients (some None) of what `inputs` hold; under create_graph=True marked so
    that they can be used, but not differentiated."""
    given = [t for t in inputs if t is not None and t.requires_grad] if torch.is_grad_enabled() else []
    if not given:
        return grads
    marked = iter(_FirstOrder.apply(name, len(given), *given, *(g for g in grads if g is not None)))
    return tuple(None if g is None else next(marked) for g in grads)


# ---- the gated delta rule ------------------------------------------------------------------

def _same_device(x, **others):
    if not x.is_cuda:
        raise ValueError("tensors must be on a GPU (there is no CPU path)")
    d = x.device
    for name, t in others.items():
        if t is not None and t.device != d:
            raise ValueError(f"{name} must be on {d}")
    return d


def _one_device(x, **others):
    """The index of the GPU that all of the tensors are on."""
    d = x.get_device()
    if d < 0:
        return _same_device(x)
    for t in others.values():
        if t is not None and t.get_device() != d:
            return _same_device(x, **others).index
    return d


def _delta_sizes(q, k, v, g, beta, one=False):
    """(B, L, Hk, Hv, Dk, Dv) of the five inputs, checked against each other; one: a single step
    without its dimension."""
    qs, vs = q.shape, v.shape
    lead = 1 if one else 2
    if len(qs) != lead + 2 or k.shape != qs or len(vs) != lead + 2 or vs[:lead] != qs[:lead]:
        raise ValueError("expected q and k [B, L, Hk, Dk] and v [B, L, Hv, Dv]")
    Hk, Dk = qs[lead:]
    Hv, Dv = vs[lead:]
    B, L = qs[0], 1 if one else qs[1]
    if Hk < 1 or Hv < 1 or Hv % Hk:
        raise ValueError("the value heads must be a multiple of the key heads")
    if not 1 <= Dk <= 128 or Dv < 1:
        raise ValueError("key heads must be 1 to 128 wide, value heads at least 1")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must have one dtype")
    for name, t in (("g", g), ("beta", beta)):
        if t.shape != vs[:-1]:
            raise ValueError(f"{name} must be [B, L, Hv]")
    for name, t in (("q", q), ("g", g), ("beta", beta)):
        if t.dtype not in DTYPE_CODE:
            raise ValueError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    return B, L, Hk, Hv, Dk, Dv


def _unit_heads(t):
    """t as it is when its last dimension has unit stride, else a contiguous copy."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def _delta_states(name, t, shape):
    if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape):
        raise ValueError(f"{name} must be float32 {list(shape)}")
    return t


def _delta_sequences(cu_seqlens, B):
    """(packed sequences, sequences that have states)."""
    if cu_seqlens is None:
        return 0, B
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32 [N + 1]")
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) need B = 1")
    N = cu_seqlens.numel() - 1
    return N, N


def gated_delta_rule_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                         scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                         initial_state: Optional[torch.Tensor] = None, return_final_state: bool = False,
                         final_state_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         info: Optional[dict] = None):
    """The gated delta rule over whole sequences on the GPU.

    With a state S [Dk, Dv] per sequence and value head:
    ``S <- e^g S; u = beta (v - S^T k); S <- S + k u^T; out = scale S^T q``.

    q, k [B, L, Hk, Dk] and v [B, L, Hv, Dv] in one dtype (Hv a multiple of Hk, Dk at most
    128); g (log decay) and beta [B, L, Hv] in any of the three dtypes each.  Strided views
    are used as they are when a head's elements are unit-stride; others are copied
    (``info["copied"]`` lists them).  ``scale`` defaults to Dk^-1/2.  ``cu_seqlens`` (int32
    [N + 1], on the GPU) packs N sequences in one row (B = 1).  States are float32
    [sequences, Hv, Dk, Dv]; ``final_state_out`` may be ``initial_state`` itself.  Returns
    out [B, L, Hv, Dv] in v's dtype, or (out, final_state).
    """
    if final_state_out is not None and not return_final_state:
        raise ValueError("final_state_out given but return_final_state is False")
    B, L, Hk, Hv, Dk, Dv = _delta_sizes(q, k, v, g, beta)
    device = _same_device(q, k=k, v=v, g=g, beta=beta, cu_seqlens=cu_seqlens, initial_state=initial_state,
                          final_state_out=final_state_out, out=out)
    given = (("q", q), ("k", k), ("v", v), ("initial_state", initial_state))
    q, k, v = _unit_heads(q), _unit_heads(k), _unit_heads(v)
    N, seqs = _delta_sequences(cu_seqlens, B)
    shape = (seqs, Hv, Dk, Dv)
    if _delta_states("initial_state", initial_state, shape) is not None:
        initial_state = _unit_heads(initial_state)
    written = (out, final_state_out)
    if out is None:
        out = torch.empty_like(v, memory_format=torch.contiguous_format)
    elif out.dtype != v.dtype or tuple(out.shape) != (B, L, Hv, Dv) or (out.stride(-1) != 1 and Dv > 1):
        raise ValueError("out must be [B, L, Hv, Dv] in v's dtype with unit stride in its last dimension")
    ht = None
    if return_final_state:
        ht = torch.empty(shape, dtype=torch.float32, device=device) if final_state_out is None else final_state_out
        _delta_states("final_state_out", ht, shape)
        if ht.stride(-1) != 1 and Dv > 1:
            raise ValueError("final_state_out must have unit stride in its last dimension")
    _CALLS["ccv_delta_fwd"](device, B, L, N, Hk, Hv, Dk, Dv, DTYPE_CODE[q.dtype], DTYPE_CODE[g.dtype], DTYPE_CODE[beta.dtype],
                            Dk ** -0.5 if scale is None else scale, *_at(q), *_at(k), *_at(v), *_at(g), *_at(beta),
                            _p(cu_seqlens), *_at(initial_state), *_at(ht), *_at(out))
    _written(*written)
    if info is not None:
        now = (q, k, v, initial_state)
        info["copied"] = [name for (name, t), u in zip(given, now) if t is not u]
    return (out, ht) if return_final_state else out


def gated_delta_rule_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                         dout: torch.Tensor, scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                         initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                         return_dinitial_state: bool = False):
    """Gradients of gated_delta_rule_fwd: (dq, dk, dv, dg, dbeta, dinitial_state).

    dout [B, L, Hv, Dv] in v's dtype; dfinal_state float32 like the states, or None (zeros).
    Each gradient has its input's shape and dtype, contiguous; dinitial_state (float32)
    only with return_dinitial_state, which needs initial_state.
    """
    B, L, Hk, Hv, Dk, Dv = _delta_sizes(q, k, v, g, beta)
    device = _same_device(q, k=k, v=v, g=g, beta=beta, dout=dout, cu_seqlens=cu_seqlens, initial_state=initial_state,
                          dfinal_state=dfinal_state)
    if dout.dtype != v.dtype or dout.shape != v.shape:
        raise ValueError("dout must be [B, L, Hv, Dv] in v's dtype")
    if return_dinitial_state and initial_state is None:
        raise ValueError("dinitial_state needs initial_state")
    q, k, v, dout = _unit_heads(q), _unit_heads(k), _unit_heads(v), _unit_heads(dout)
    N, seqs = _delta_sequences(cu_seqlens, B)
    shape = (seqs, Hv, Dk, Dv)
    if _delta_states("initial_state", initial_state, shape) is not None:
        initial_state = _unit_heads(initial_state)
    if _delta_states("dfinal_state", dfinal_state, shape) is not None:
        dfinal_state = _unit_heads(dfinal_state)
    dq, dk, dv, dg, db = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v, g, beta))
    dh = torch.empty(shape, dtype=torch.float32, device=device) if return_dinitial_state else None
    _CALLS["ccv_delta_bwd"](device, B, L, N, Hk, Hv, Dk, Dv, DTYPE_CODE[q.dtype], DTYPE_CODE[g.dtype], DTYPE_CODE[beta.dtype],
                            Dk ** -0.5 if scale is None else scale, *_at(q), *_at(k), *_at(v), *_at(g), *_at(beta),
                            _p(cu_seqlens), *_at(initial_state), *_at(dout), *_at(dfinal_state), *_at(dq), *_at(dk),
                            *_at(dv), *_at(dg), *_at(db), *_at(dh))
    return dq, dk, dv, dg, db, dh


class _GatedDeltaRuleFn(torch.autograd.Function):
    """Forward and backward through the C ABI; saves the inputs, and the backward makes
    everything else again."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale, cu_seqlens, initial_state, return_final_state):
        res = gated_delta_rule_fwd(q, k, v, g, beta, scale, cu_seqlens, initial_state, return_final_state)
        ctx.save_for_backward(q, k, v, g, beta, cu_seqlens, initial_state)
        ctx.scale = scale
        ctx.return_final_state = return_final_state
        ctx.set_materialize_grads(False)
        return res

    @staticmethod
    def backward(ctx, dout, *rest):
        q, k, v, g, beta, cu_seqlens, initial_state = ctx.saved_tensors
        dht = rest[0] if ctx.return_final_state and rest else None
        dout = torch.zeros_like(v) if dout is None else dout.to(v.dtype)
        want_dh = initial_state is not None and ctx.needs_input_grad[7]
        with torch.no_grad():
            grads = gated_delta_rule_bwd(q, k, v, g, beta, dout, ctx.scale, cu_seqlens, initial_state,
                                         None if dht is None else dht.float(), want_dh)
        dq, dk, dv, dg, db, dh = _first_order("gated_delta_rule_fn", (q, k, v, g, beta, initial_state, dout, dht), grads)
        return dq, dk, dv, dg, db, None, None, dh, None


def gated_delta_rule_fn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                        scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                        initial_state: Optional[torch.Tensor] = None, return_final_state: bool = False):
    """Differentiable gated delta rule (gated_delta_rule_fwd, with gradients for q, k, v, g,
    beta and initial_state through gated_delta_rule_bwd).  Differentiable once: a second
    derivative raises."""
    return _GatedDeltaRuleFn.apply(q, k, v, g, beta, scale, cu_seqlens, initial_state, return_final_state)


def gated_delta_rule_update(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                            state: torch.Tensor, scale: Optional[float] = None,
                            state_indices: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """New steps of the gated delta rule against cached states, advanced in place.

    q, k [B, Hk, Dk], v [B, Hv, Dv], g and beta [B, Hv] (one step), or with a dimension of L
    steps after B; state float32 [slots, Hv, Dk, Dv].  Row b uses slot ``state_indices[b]``
    (int32, on the GPU), or slot b without; a row whose index is outside [0, slots) is idle:
    its outputs are zeros.  Two rows may not use one slot.  Returns out with v's shape.
    """
    one = q.dim() == 3
    B, L, Hk, Hv, Dk, Dv = _delta_sizes(q, k, v, g, beta, one)
    device = _same_device(q, k=k, v=v, g=g, beta=beta, state=state, state_indices=state_indices, out=out)
    if state.dtype != torch.float32 or state.dim() != 4 or state.shape[1:] != (Hv, Dk, Dv):
        raise ValueError("state must be float32 [slots, Hv, Dk, Dv]")
    if state.stride(-1) != 1 and Dv > 1:
        raise ValueError("state must have unit stride in its last dimension")
    if state_indices is not None and (state_indices.dtype != torch.int32 or state_indices.shape != (B,)
                                      or not state_indices.is_contiguous()):
        raise ValueError("state_indices must be contiguous int32 [B]")
    if state_indices is None and B > state.shape[0]:
        raise ValueError("more rows than states")
    q, k, v = _unit_heads(q), _unit_heads(k), _unit_heads(v)
    written = (state, out)
    if out is None:
        out = torch.empty_like(v, memory_format=torch.contiguous_format)
    elif out.dtype != v.dtype or out.shape != v.shape or (out.stride(-1) != 1 and Dv > 1):
        raise ValueError("out must have v's shape and dtype with unit stride in its last dimension")
    at = _step_at if one else _at
    _CALLS["ccv_delta_update"](device, B, L, state.shape[0], Hk, Hv, Dk, Dv, DTYPE_CODE[q.dtype], DTYPE_CODE[g.dtype],
                               DTYPE_CODE[beta.dtype], Dk ** -0.5 if scale is None else scale, *at(q), *at(k), *at(v),
                               *at(g), *at(beta), _p(state_indices), *_at(state), *at(out))
    _written(*written)
    return out


# ---- the gated linear recurrence -------------------------------------------------------------

def _linrec_sizes(x, g, one=False):
    """(B, L, C) of the inputs, checked against each other; one: a single step without its dimension."""
    s = x.shape
    if len(s) != (2 if one else 3) or g.shape != s:
        raise ValueError("expected x and g [B, C]" if one else "expected x and g [B, L, C]")
    if x.dtype not in DTYPE_CODE or g.dtype not in DTYPE_CODE:
        raise ValueError(f"x and g must be float32, float16 or bfloat16, not {x.dtype} and {g.dtype}")
    return s[0], 1 if one else s[1], s[-1]


def _rows2(t):
    """A tensor's address and its two leading strides, as consecutive values."""
    if t is None:
        return (0, 0, 0)
    s = t.stride()
    return (t.data_ptr(), s[0], s[1])


def _row1(t):
    """The same of a single step without its dimension."""
    return (t.data_ptr(), t.stride(0), 0)


def _state_at(t):
    """The same of a tensor of states, which has one."""
    return (0, 0) if t is None else (t.data_ptr(), t.stride(0))


def gated_linear_recurrence_fwd(x: torch.Tensor, g: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                                initial_state: Optional[torch.Tensor] = None, return_final_state: bool = False,
                                normalize: bool = False, final_state_out: Optional[torch.Tensor] = None,
                                out: Optional[torch.Tensor] = None, return_carries: bool = False,
                                info: Optional[dict] = None):
    """A gated linear recurrence over whole sequences on the GPU, one state a channel:
    ``h <- e^g h + s x; out = h``, with s = 1, or ``normalize``: s = sqrt(1 - e^2g).

    x [B, L, C] and g (log decay, at most 0) [B, L, C], each in any of the three dtypes.  Strided views
    are used as they are when channels are unit-stride; others are copied (``info["copied"]``
    lists them).  ``cu_seqlens`` (int32 [N + 1], on the GPU) packs N sequences in one row (B = 1).
    States are float32 [sequences, C]; ``final_state_out`` may be ``initial_state`` itself.
    B ceil(L / 128) ceil(C / 64) has to be below 2^23.
    Returns out [B, L, C] in x's dtype, then the final state if wanted, then with
    ``return_carries`` the states that gated_linear_recurrence_bwd can start from (float32
    [B, ceil(L / 128), C]).
    """
    if final_state_out is not None and not return_final_state:
        raise ValueError("final_state_out given but return_final_state is False")
    B, L, C = _linrec_sizes(x, g)
    device = _one_device(x, g=g, cu_seqlens=cu_seqlens, initial_state=initial_state, final_state_out=final_state_out, out=out)
    given = (x, g, initial_state)
    x, g = _unit_heads(x), _unit_heads(g)
    N, seqs = _delta_sequences(cu_seqlens, B)
    if _delta_states("initial_state", initial_state, (seqs, C)) is not None:
        initial_state = _unit_heads(initial_state)
    written = (out, final_state_out)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype != x.dtype or tuple(out.shape) != (B, L, C) or (out.stride(-1) != 1 and C > 1):
        raise ValueError("out must be [B, L, C] in x's dtype with unit stride in its last dimension")
    ht = None
    if return_final_state:
        ht = torch.empty((seqs, C), dtype=torch.float32, device=device) if final_state_out is None else final_state_out
        _delta_states("final_state_out", ht, (seqs, C))
        if ht.stride(-1) != 1 and C > 1:
            raise ValueError("final_state_out must have unit stride in its last dimension")
    carries = None
    if return_carries:
        carries = torch.empty((B, -(-L // CCV_LINREC_CHUNK), C), dtype=torch.float32, device=device)
    _CALLS["ccv_linrec_fwd"](device, B, L, C, N, DTYPE_CODE[x.dtype], DTYPE_CODE[g.dtype], int(normalize), 0, *_rows2(x), *_rows2(g),
                             _p(cu_seqlens), *_state_at(initial_state), *_state_at(ht), *_rows2(out), _p(carries))
    _written(*written)
    if info is not None:
        info["copied"] = [name for name, t, u in zip(("x", "g", "initial_state"), given, (x, g, initial_state)) if t is not u]
    res = (out,) + ((ht,) if return_final_state else ()) + ((carries,) if return_carries else ())
    return res if len(res) > 1 else out


def gated_linear_recurrence_bwd(x: torch.Tensor, g: torch.Tensor, dout: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                                initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                                normalize: bool = False, carries: Optional[torch.Tensor] = None,
                                return_dinitial_state: bool = False):
    """Gradients of gated_linear_recurrence_fwd: (dx, dg, dinitial_state).

    dout [B, L, C] in x's dtype; dfinal_state float32 like the states, or None (zeros); carries:
    what the forward call returned for these inputs, or None (made again, by another pass over x and g).  Each gradient
    has its input's shape and dtype, contiguous; dinitial_state (float32) only with
    return_dinitial_state, which needs initial_state.
    """
    B, L, C = _linrec_sizes(x, g)
    device = _one_device(x, g=g, dout=dout, cu_seqlens=cu_seqlens, initial_state=initial_state, dfinal_state=dfinal_state,
                          carries=carries)
    if dout.dtype != x.dtype or dout.shape != x.shape:
        raise ValueError("dout must be [B, L, C] in x's dtype")
    if return_dinitial_state and initial_state is None:
        raise ValueError("dinitial_state needs initial_state")
    if carries is not None and (carries.dtype != torch.float32 or tuple(carries.shape) != (B, -(-L // CCV_LINREC_CHUNK), C)
                                or not carries.is_contiguous()):
        raise ValueError("carries must be what gated_linear_recurrence_fwd returned for these inputs")
    x, g, dout = _unit_heads(x), _unit_heads(g), _unit_heads(dout)
    N, seqs = _delta_sequences(cu_seqlens, B)
    if _delta_states("initial_state", initial_state, (seqs, C)) is not None:
        initial_state = _unit_heads(initial_state)
    if _delta_states("dfinal_state", dfinal_state, (seqs, C)) is not None:
        dfinal_state = _unit_heads(dfinal_state)
    dx, dg = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (x, g))
    dh = torch.empty((seqs, C), dtype=torch.float32, device=device) if return_dinitial_state else None
    _CALLS["ccv_linrec_bwd"](device, B, L, C, N, DTYPE_CODE[x.dtype], DTYPE_CODE[g.dtype], int(normalize), 0, *_rows2(x), *_rows2(g),
                             _p(cu_seqlens), *_state_at(initial_state), *_rows2(dout), *_state_at(dfinal_state), _p(carries),
                             *_rows2(dx), *_rows2(dg), *_state_at(dh))
    return dx, dg, dh


class _GatedLinearRecurrenceFn(torch.autograd.Function):
    """Forward and backward through the C ABI; saves the inputs and the states between chunks of steps."""

    @staticmethod
    def forward(ctx, x, g, cu_seqlens, initial_state, return_final_state, normalize):
        *res, carries = gated_linear_recurrence_fwd(x, g, cu_seqlens, initial_state, return_final_state, normalize, return_carries=True)
        ctx.save_for_backward(x, g, cu_seqlens, initial_state, carries)
        ctx.normalize = normalize
        ctx.set_materialize_grads(False)
        return tuple(res) if return_final_state else res[0]

    @staticmethod
    def backward(ctx, dout, dht=None):
        x, g, cu_seqlens, initial_state, carries = ctx.saved_tensors
        dout = torch.zeros_like(x) if dout is None else dout.to(x.dtype)
        want_dh = initial_state is not None and ctx.needs_input_grad[3]
        with torch.no_grad():
            grads = gated_linear_recurrence_bwd(x, g, dout, cu_seqlens, initial_state, dht, ctx.normalize, carries, want_dh)
        dx, dg, dh = _first_order("gated_linear_recurrence_fn", (x, g, initial_state, dout, dht), grads)
        return dx, dg, None, dh, None, None


def gated_linear_recurrence_fn(x: torch.Tensor, g: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                               initial_state: Optional[torch.Tensor] = None, return_final_state: bool = False,
                               normalize: bool = False):
    """Differentiable gated linear recurrence (gated_linear_recurrence_fwd, with gradients for x, g and
    initial_state through gated_linear_recurrence_bwd).  Differentiable once: a second derivative raises."""
    return _GatedLinearRecurrenceFn.apply(x, g, cu_seqlens, initial_state, return_final_state, normalize)


def gated_linear_recurrence_update(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                                   state_indices: Optional[torch.Tensor] = None, normalize: bool = False,
                                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """New steps of the gated linear recurrence against cached states, advanced in place.

    x and g [B, C] (one step), or [B, L, C]; state float32 [slots, C].  Row b uses slot
    ``state_indices[b]`` (int32, on the GPU), or slot b without; a row whose index is outside
    [0, slots) is idle: its outputs are zeros.  Two rows may not use one slot.  Returns out
    with x's shape.
    """
    one = x.dim() == 2
    B, L, C = _linrec_sizes(x, g, one)
    device = _one_device(x, g=g, state=state, state_indices=state_indices, out=out)
    if state.dtype != torch.float32 or state.dim() != 2 or state.shape[1] != C:
        raise ValueError("state must be float32 [slots, C]")
    if state.stride(-1) != 1 and C > 1:
        raise ValueError("state must have unit stride in its last dimension")
    if state_indices is not None and (state_indices.dtype != torch.int32 or state_indices.shape != (B,)
                                      or not state_indices.is_contiguous()):
        raise ValueError("state_indices must be contiguous int32 [B]")
    if state_indices is None and B > state.shape[0]:
        raise ValueError("more rows than states")
    x, g = _unit_heads(x), _unit_heads(g)
    written = (state, out)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype != x.dtype or out.shape != x.shape or (out.stride(-1) != 1 and C > 1):
        raise ValueError("out must have x's shape and dtype with unit stride in its last dimension")
    at = _row1 if one else _rows2
    _CALLS["ccv_linrec_update"](device, B, L, C, state.shape[0], DTYPE_CODE[x.dtype], DTYPE_CODE[g.dtype], int(normalize), 0,
                                *at(x), *at(g), _p(state_indices), *_state_at(state), *at(out))
    _written(*written)
    return out


# ---- layer norm ------------------------------------------------------------------------------

def _norm_rows(x):
    """(x, (n0, n1, width), strides of the first two): x as [n0, n1, width] with unit stride along
    the width, copied only where its strides allow no such view."""
    if x.dim() < 1:
        raise ValueError("x needs a last dimension to be normalised")
    if x.shape[-1] > 1 and x.stride(-1) != 1:
        x = x.contiguous()
    dim = x.dim()
    if dim > 3:
        x = x.flatten(0, dim - 3)
    return (x, (1,) * (3 - dim) + tuple(x.shape), (0,) * (3 - dim) + x.stride()[:-1])


def _norm_weights(x, weight, bias):
    width = x.shape[-1:]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (t.shape != width or t.dtype not in DTYPE_CODE):
            raise ValueError(f"{name} must be [width] in float32, float16 or bfloat16")
    if weight is not None and bias is not None and bias.dtype != weight.dtype:
        raise ValueError("bias must have the weight's dtype")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"x must be float32, float16 or bfloat16, not {x.dtype}")
    return (None if weight is None else weight.contiguous(), None if bias is None else bias.contiguous())


def _statistics(x, shape, device):
    """Room for mean and rstd; those of no values, which no call writes, are NaN."""
    new = torch.empty if x.shape[-1] else lambda shape, **kw: torch.full(shape, math.nan, **kw)
    return [new(shape, dtype=torch.float32, device=device) for _ in range(2)]


def _gradient_types(weight_dtype, x, weight, bias=None):
    """(type of dweight and dbias, the call's, weight, bias): a call has one type for the parameters and their gradients, so
    where the caller wants another than the parameters' they go in 32 bits, which hold either's values, and the sums come back so."""
    own = x if weight is None and bias is None else bias if weight is None else weight
    wd = weight_dtype or own.dtype
    if wd not in DTYPE_CODE:
        raise ValueError(f"weight_dtype must be float32, float16 or bfloat16, not {wd}")
    if own is x or own.dtype == wd:
        return wd, wd, weight, bias
    return wd, torch.float32, *(None if t is None else t.float() for t in (weight, bias))


def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, return_stats: bool = False, out: Optional[torch.Tensor] = None):
    """Layer norm over x's last dimension on the GPU: (x - mean) rstd weight + bias.

    x [..., width], any strides (views of up to three dimensions that are unit-stride along
    the width are used as they are); weight and bias [width] or None.  Returns out
    (contiguous, x's dtype), or (out, mean, rstd) with float32 statistics [...] (NaN where width is 0).
    """
    weight, bias = _norm_weights(x, weight, bias)
    device = _same_device(x, weight=weight, bias=bias, out=out)
    rows, shape, s = _norm_rows(x)
    written = out
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype != x.dtype or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous with x's shape and dtype")
    mean = rstd = None
    if return_stats:
        mean, rstd = _statistics(x, x.shape[:-1], device)
    w = weight if weight is not None else bias if bias is not None else x
    _CALLS["ccv_norm_fwd"](device, *shape, DTYPE_CODE[x.dtype], DTYPE_CODE[w.dtype], eps, 0, rows.data_ptr(), s[0], s[1],
                           _p(weight), _p(bias), out.data_ptr(), shape[1] * shape[2], shape[2], _p(mean), _p(rstd))
    _written(written)
    return (out, mean, rstd) if return_stats else out


def layer_norm_bwd(x: torch.Tensor, weight: Optional[torch.Tensor], dout: torch.Tensor, mean: torch.Tensor,
                   rstd: torch.Tensor, want_dx: bool = True, want_dweight: bool = True, want_dbias: bool = True,
                   weight_dtype: Optional[torch.dtype] = None):
    """Gradients of layer_norm_fwd: (dx, dweight, dbias), None where not wanted.

    dout has x's shape and dtype; mean and rstd are the forward's.  dweight and dbias come in
    ``weight_dtype`` (the weight's dtype by default, x's without a weight), summed in float32
    in a fixed order.
    """
    weight, _ = _norm_weights(x, weight, None)
    device = _same_device(x, weight=weight, dout=dout, mean=mean, rstd=rstd)
    if dout.dtype != x.dtype or dout.shape != x.shape:
        raise ValueError("dout must have x's shape and dtype")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.shape != x.shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with x's leading shape")
    wanted, wd, weight, _ = _gradient_types(weight_dtype, x, weight)
    (rows, shape, s), (drows, _, d) = _norm_rows(x), _norm_rows(dout)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if want_dx else None
    dw = torch.empty(x.shape[-1], dtype=wd, device=device) if want_dweight else None
    db = torch.empty(x.shape[-1], dtype=wd, device=device) if want_dbias else None
    _CALLS["ccv_norm_bwd"](device, *shape, DTYPE_CODE[x.dtype], DTYPE_CODE[wd], rows.data_ptr(), s[0], s[1], _p(weight),
                           drows.data_ptr(), d[0], d[1], mean.data_ptr(), rstd.data_ptr(), _p(dx), shape[1] * shape[2], shape[2],
                           _p(dw), _p(db))
    if wd != wanted:
        dw, db = (None if t is None else t.to(wanted) for t in (dw, db))
    return dx, dw, db


class _LayerNormFn(torch.autograd.Function):
    """Forward and backward through the C ABI; saves x, weight and the rows' statistics."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        out, mean, rstd = layer_norm_fwd(x, weight, bias, eps, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return out

    @staticmethod
    def backward(ctx, dout):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        with torch.no_grad():
            grads = layer_norm_bwd(x, weight, dout.to(x.dtype), mean, rstd, need[0], need[1], need[2], ctx.bias_dtype)
        return *_first_order("layer_norm_fn", (x, weight, dout), grads), None


def layer_norm_fn(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm (layer_norm_fwd, with gradients for x, weight and bias
    through layer_norm_bwd).  Differentiable once: a second derivative raises."""
    return _LayerNormFn.apply(x, weight, bias, eps)


# ---- group norm ------------------------------------------------------------------------------

def _flat_rows(t):
    """t [..., C] as [rows, C] with unit stride along the channels, copied only where its strides allow no
    such view."""
    t = _unit_heads(t)
    return t if t.dim() == 2 else t.reshape(math.prod(t.shape[:-1]), t.shape[-1])


def _group_sizes(x, num_groups, activation, weight, bias, gate):
    """(rows, groups, width, activation's code), checked."""
    if x.dim() < 2:
        raise ValueError("expected x [..., C]")
    C = x.shape[-1]
    if num_groups < 1 or C % num_groups:
        raise ValueError("num_groups must divide the channels")
    if activation not in (None, "silu", "swish"):
        raise ValueError(f"activation must be None, 'silu' or 'swish', not {activation!r}")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"x must be float32, float16 or bfloat16, not {x.dtype}")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (t.shape != (C,) or t.dtype not in DTYPE_CODE):
            raise ValueError(f"{name} must be [C] in float32, float16 or bfloat16")
    if weight is not None and bias is not None and bias.dtype != weight.dtype:
        raise ValueError("bias must have the weight's dtype")
    if gate is not None and (gate.shape != x.shape or gate.dtype != x.dtype):
        raise ValueError("gate must have x's shape and dtype")
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    return rows, num_groups, C // num_groups, CCV_ACT_NONE if activation is None else CCV_ACT_SILU


def group_norm_fwd(x: torch.Tensor, num_groups: int, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, activation: Optional[str] = None, eps: float = 1e-5,
                   return_stats: bool = False, out: Optional[torch.Tensor] = None):
    """Group norm of each step's channels on the GPU, with an activation or a gate behind it.

    x [..., C], channels last; every row's C channels are normalised in ``num_groups`` groups of neighbours, each over
    its own C / num_groups values (torch's group_norm of [rows, C]): no step sees another.  With
    y = (x - mean) rstd weight + bias (weight and bias [C] or None) returns act(y), or with
    ``gate`` (x's shape and dtype) y act(gate); activation None or "silu".  Strided rows are used
    as they are when channels are unit-stride and the leading dimensions lie at one stride.
    Returns out (contiguous, x's dtype), or (out, mean, rstd) with float32 statistics [..., num_groups] (NaN without channels).
    """
    rows, groups, width, act = _group_sizes(x, num_groups, activation, weight, bias, gate)
    device = _one_device(x, weight=weight, bias=bias, gate=gate, out=out)
    weight, bias = (None if t is None else t.contiguous() for t in (weight, bias))
    written = out
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif out.dtype != x.dtype or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous with x's shape and dtype")
    C = x.shape[-1]
    mean = rstd = None
    if return_stats:
        mean, rstd = _statistics(x, (*x.shape[:-1], groups), device)
    w = weight if weight is not None else bias if bias is not None else x
    x2, z2 = _flat_rows(x), None if gate is None else _flat_rows(gate)
    _CALLS["ccv_group_norm_fwd"](device, rows, groups, width, DTYPE_CODE[x.dtype], DTYPE_CODE[w.dtype], act, eps, *_state_at(x2),
                                 _p(weight), _p(bias), *_state_at(z2), out.data_ptr(), C, _p(mean), _p(rstd))
    _written(written)
    return (out, mean, rstd) if return_stats else out


def group_norm_bwd(x: torch.Tensor, num_groups: int, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                   dout: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, gate: Optional[torch.Tensor] = None,
                   activation: Optional[str] = None, want_dx: bool = True, want_dweight: bool = True,
                   want_dbias: bool = True, want_dgate: bool = True, weight_dtype: Optional[torch.dtype] = None):
    """Gradients of group_norm_fwd: (dx, dweight, dbias, dgate), None where not wanted (dgate: or without a gate).

    dout has x's shape and dtype; mean and rstd are the forward's.  dweight and dbias come in
    ``weight_dtype`` (the weight's dtype by default, the bias's or x's without one), summed in float32 in
    a fixed order.
    """
    rows, groups, width, act = _group_sizes(x, num_groups, activation, weight, bias, gate)
    device = _one_device(x, weight=weight, bias=bias, dout=dout, mean=mean, rstd=rstd, gate=gate)
    if dout.dtype != x.dtype or dout.shape != x.shape:
        raise ValueError("dout must have x's shape and dtype")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or tuple(t.shape) != (*x.shape[:-1], groups) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 [..., num_groups]")
    weight, bias = (None if t is None else t.contiguous() for t in (weight, bias))
    wanted, wd, weight, bias = _gradient_types(weight_dtype, x, weight, bias)
    C = x.shape[-1]
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if want_dx else None
    dz = torch.empty_like(x, memory_format=torch.contiguous_format) if want_dgate and gate is not None else None
    dw = torch.empty(C, dtype=wd, device=device) if want_dweight else None
    db = torch.empty(C, dtype=wd, device=device) if want_dbias else None
    x2, d2, z2 = _flat_rows(x), _flat_rows(dout), None if gate is None else _flat_rows(gate)
    _CALLS["ccv_group_norm_bwd"](device, rows, groups, width, DTYPE_CODE[x.dtype], DTYPE_CODE[wd], act, 0, *_state_at(x2),
                                 _p(weight), _p(bias), *_state_at(z2), *_state_at(d2), mean.data_ptr(), rstd.data_ptr(),
                                 _p(dx), C, _p(dz), C, _p(dw), _p(db))
    if wd != wanted:
        dw, db = (None if t is None else t.to(wanted) for t in (dw, db))
    return dx, dw, db, dz


class _GroupNormFn(torch.autograd.Function):
    """Forward and backward through the C ABI; saves the inputs and the groups' statistics."""

    @staticmethod
    def forward(ctx, x, num_groups, weight, bias, gate, activation, eps):
        out, mean, rstd = group_norm_fwd(x, num_groups, weight, bias, gate, activation, eps, return_stats=True)
        ctx.save_for_backward(x, weight, bias, gate, mean, rstd)
        ctx.num_groups, ctx.activation = num_groups, activation
        return out

    @staticmethod
    def backward(ctx, dout):
        x, weight, bias, gate, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        with torch.no_grad():
            grads = group_norm_bwd(x, ctx.num_groups, weight, bias, dout.to(x.dtype), mean, rstd, gate, ctx.activation,
                                   need[0], need[2], need[3], need[4])
        dx, dw, db, dz = _first_order("group_norm_fn", (x, weight, bias, gate, dout), grads)
        return dx, None, dw, db, dz, None, None


def group_norm_fn(x: torch.Tensor, num_groups: int, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, activation: Optional[str] = None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable group norm (group_norm_fwd, with gradients for x, weight, bias and gate through
    group_norm_bwd).  Differentiable once: a second derivative raises."""
    return _GroupNormFn.apply(x, num_groups, weight, bias, gate, activation, eps)


# ---- rotary positions ------------------------------------------------------------------------

def rotary_frequencies(turned: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original_length: Optional[int] = None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(frequencies, scale) for rotary_fwd: float64 [turned / 2], base^(-2i / turned) radians a position, and the
    factor of the results.

    ``scaling`` stretches them for contexts ``factor`` times as long as the ones a model was trained on:
      "linear"  every position divided by the factor
      "base"    the base raised by factor^(turned / (turned - 2)), so that the slowest pair is divided by the
                factor and the fastest not at all
      "parts"   pairs that make more than ``fast`` turns over ``original_length`` positions stay, those that make fewer
                than ``slow`` are divided, with a ramp between, which begins at the first pair at the earliest and may
                end behind the last; scale = 0.1 ln(factor) + 1
    """
    if turned < 2 or turned % 2:
        raise ValueError("turned must be a positive even number")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', not {scaling!r}")
    if not base > 1 or not factor >= 1 or not fast > slow > 0:
        raise ValueError("base must be above 1, factor at least 1 and fast above slow above 0")
    if scaling == "base":
        base = base * factor ** (turned / max(turned - 2, 1))
    i = torch.arange(turned // 2, dtype=torch.float64)
    f = base ** (-2 * i / turned)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_length is None or original_length < 1:
            raise ValueError("scaling 'parts' needs original_length")
        pair = lambda turns: turned * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), turned - 1)
        whole = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / factor * (1 - whole) + f * whole
        scale = 0.1 * math.log(factor) + 1
    return f.to(device), scale


def _rotary_sizes(q, k, positions, frequencies):
    """(B, L, Hq, Hk, D), checked; one step without its dimension where q is [B, Hq, D]."""
    one = q.dim() == 3
    lead = q.shape[:-2]
    if q.dim() not in (3, 4):
        raise ValueError("expected q [B, L, Hq, D] or [B, Hq, D]")
    if k is not None and (k.dim() != q.dim() or k.shape[:-2] != lead or k.shape[-1] != q.shape[-1] or k.dtype != q.dtype):
        raise ValueError("k must have q's dtype and sizes, but for its heads")
    if q.dtype not in DTYPE_CODE:
        raise ValueError(f"q must be float32, float16 or bfloat16, not {q.dtype}")
    if positions.dtype != torch.int32 or positions.shape != lead:
        raise ValueError("positions must be int32 [B, L] ([B] for one step)")
    D = q.shape[-1]
    if frequencies.dtype != torch.float64 or frequencies.dim() != 1 or 2 * frequencies.numel() > D:
        raise ValueError("frequencies must be float64 [turned / 2], with turned at most D")
    if not 1 <= D <= 2048:
        raise ValueError("heads must be 1 to 2048 wide")
    return lead[0], 1 if one else lead[1], q.shape[-2], 0 if k is None else k.shape[-2], D


def rotary_fwd(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, frequencies: torch.Tensor,
               interleaved: bool = False, scale: float = 1.0, inverse: bool = False,
               q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Queries and keys turned by their positions on the GPU, in one call.

    q [B, L, Hq, D] and k [B, L, Hk, D] or None, in one dtype; positions int32 [B, L] (those of
    sequence_tables, say; any strides); or one step, without the dimension of L.  frequencies: float64 [turned / 2],
    radians a position (rotary_frequencies).  The first ``turned`` elements of a head make pairs, (i, i + turned / 2)
    or with ``interleaved`` (2i, 2i + 1); a pair (u, v) becomes scale (u cos - v sin, v cos + u sin), the rest of the head
    is copied.  ``inverse`` turns the other way (the scale stays).  q_out and k_out may be q and k
    themselves.  Strided views are used as they are when a head's elements are unit-stride.  Returns (q', k'), k' None
    without k.
    """
    B, L, Hq, Hk, D = _rotary_sizes(q, k, positions, frequencies)
    device = _one_device(q, k=k, positions=positions, frequencies=frequencies, q_out=q_out, k_out=k_out)
    if k is None and k_out is not None:
        raise ValueError("k_out given without k")
    written = (q_out, k_out)
    one = q.dim() == 3
    outs = []
    for name, t, o in (("q_out", q, q_out), ("k_out", k, k_out)):
        if t is None:
            outs.append(None)
        elif o is None:
            outs.append(torch.empty_like(t, memory_format=torch.contiguous_format))
        elif o.dtype != t.dtype or o.shape != t.shape or (o.stride(-1) != 1 and D > 1):
            raise ValueError(f"{name} must have its input's shape and dtype with unit stride in its last dimension")
        else:
            outs.append(o)
    q, k = _unit_heads(q), None if k is None else _unit_heads(k)
    at = _step_at if one else _at
    none = (0, 0, 0, 0)
    ps = positions.stride()
    frequencies = frequencies.contiguous()
    _CALLS["ccv_rotary"](device, B, L, Hq, Hk, D, 2 * frequencies.numel(), DTYPE_CODE[q.dtype], int(interleaved), int(inverse), scale,
                         *at(q), *(none if k is None else at(k)), positions.data_ptr(), ps[0], 0 if one else ps[1],
                         frequencies.data_ptr(), *at(outs[0]), *(none if k is None else at(outs[1])))
    _written(*written)
    return outs[0], outs[1]


class _RotaryFn(torch.autograd.Function):
    """Forward and backward through the C ABI; the backward turns the gradients the other way."""

    @staticmethod
    def forward(ctx, q, k, positions, frequencies, interleaved, scale):
        ctx.save_for_backward(positions, frequencies)
        ctx.how = interleaved, scale
        ctx.set_materialize_grads(False)
        return rotary_fwd(q, k, positions, frequencies, interleaved, scale)

    @staticmethod
    def backward(ctx, dq, dk):
        given = [t for t in (dq, dk) if t is not None]
        if not given:
            return (None,) * 6
        with torch.no_grad():
            turned = rotary_fwd(given[0], given[1] if len(given) > 1 else None, *ctx.saved_tensors, *ctx.how, inverse=True)
        turned = iter(_first_order("rotary_fn", given, turned))
        return next(turned) if dq is not None else None, next(turned) if dk is not None else None, None, None, None, None


def rotary_fn(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, frequencies: torch.Tensor,
              interleaved: bool = False, scale: float = 1.0):
    """Differentiable rotary positions (rotary_fwd, with gradients for q and k by the inverse turn).
    Differentiable once: a second derivative raises.  The frequencies get no gradient, and may not want one."""
    if frequencies.requires_grad and torch.is_grad_enabled():
        raise ValueError("frequencies get no gradient: detach them")
    return _RotaryFn.apply(q, k, positions, frequencies, interleaved, scale)


# ---- sequence tables -------------------------------------------------------------------------

def sequence_tables(lengths: torch.Tensor, total: int):
    """The tables of a row of ``total`` steps that packs sequences of the given lengths
    (int32 [N], on the GPU): (cu_seqlens [N + 1], seq_idx [1, total], positions [1, total]),
    all int32, made on the GPU without a look by the host.

    seq_idx is what causal_conv1d_fwd takes, cu_seqlens what gated_delta_rule_fwd and
    gated_linear_recurrence_fwd take, positions what rotary_fwd takes.
    Steps past the last sequence have seq_idx -1 and position 0; lengths that do not fit
    are cut at ``total``, negative ones count as 0.
    """
    if lengths.dtype != torch.int32 or lengths.dim() != 1 or not lengths.is_contiguous():
        raise ValueError("lengths must be contiguous int32 [N]")
    if total < 0:
        raise ValueError("total must not be negative")
    device = _same_device(lengths)
    n = lengths.numel()
    cu, seq, pos = lengths.new_empty(n + 1), lengths.new_empty((1, total)), lengths.new_empty((1, total))
    _CALLS["ccv_seq_tables"](device, n, total, lengths.data_ptr(), cu.data_ptr(), seq.data_ptr(), pos.data_ptr())
    return cu, seq, pos

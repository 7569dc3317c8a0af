"""GB300-native second-order Higher-order Linear Attention (HLA): masked, unmasked and
the asymmetric variant AHLA, the backward pass of the masked forward, and masked
third-order HLA (forward and decode); beside them two more layers whose serving state
has a constant size: a gated linear recurrence (``gated_*``) and softmax attention over a
sliding window with first tokens that stay visible (``window_*``); and the operators of a
selective state space layer: its short causal convolution (``conv_*``), its scan
(``ssm_*``) and the norm over groups of channels with an activated gate (``norm_*``).

Thin ctypes binding over the C ABI in ``include/hla.h`` (library
``_lib/libhla_gb300.so``, built for sm_103a by ``_build.build()``).  Functions named
like the C entry points take device pointers (ints) or torch CUDA tensors and only
marshal arguments; every step of the computation runs in the library's kernels.
PyTorch is used for device memory and streams only.

If the library has not been built, every call raises ``RuntimeError``: there is no
fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from collections import namedtuple
from dataclasses import dataclass

from ._build import LIB_PATH

HLA_OK, HLA_ERR_ARG, HLA_ERR_UNSUPPORTED, HLA_ERR_CUDA, HLA_ERR_TIMEOUT = 0, 1, 2, 3, 4
HLA_F32, HLA_BF16 = 0, 1
HLA_NORMALIZE, HLA_DECAY, HLA_UNMASKED, HLA_ASYMMETRIC = 1, 2, 4, 8
HLA_GATE_GIVEN, HLA_GATE_SIGMOID, HLA_GATE_RATE = 0, 1, 2
HLA_ACT_NONE, HLA_ACT_SILU = 0, 1

__all__ = [
    "HLA_OK", "HLA_ERR_ARG", "HLA_ERR_UNSUPPORTED", "HLA_ERR_CUDA", "HLA_ERR_TIMEOUT",
    "HLA_F32", "HLA_BF16", "HLA_NORMALIZE", "HLA_DECAY", "HLA_UNMASKED", "HLA_ASYMMETRIC",
    "HlaError", "hla_params", "hla_state", "library", "EXPORTS",
    "hla_forward_workspace_size", "hla_forward_kernel", "hla_forward_chunked", "hla_state_combine",
    "hla_decode_step", "hla_sync_status", "hla_status_string", "hla_last_error", "hla_forward_chunked_noalloc",
    "hla_backward_workspace_size", "hla_backward_chunked", "hla_backward_chunked_traced",
    "hla_backward_chunked_state", "hla_state3", "hla_state3_combine", "state3_combine", "hla_forward3_workspace_size", "hla_forward3_chunked", "hla_forward3_chunked_traced",
    "hla_decode3_step", "State3", "forward3", "decode3_step", "hla_selftest_expired_wait",
    "State", "new_workspace", "forward", "state_combine", "decode_step", "backward",
    "HLA_GATE_GIVEN", "HLA_GATE_SIGMOID", "HLA_GATE_RATE", "hla_tensor", "hla_gated_params", "hla_window_params",
    "hla_gated_workspace_size", "hla_gated_forward", "hla_gated_backward", "hla_gated_step",
    "hla_window_forward", "hla_window_backward_workspace_size", "hla_window_backward", "hla_window_step",
    "hla_window_cache_fill",
    "gated_workspace", "gated_forward", "gated_backward", "gated_step", "GatedGradients",
    "window_forward", "window_workspace", "window_backward", "window_cache", "window_cache_fill", "window_step",
    "HLA_ACT_NONE", "HLA_ACT_SILU", "hla_conv_params", "hla_ssm_params", "hla_norm_params", "hla_ssm_gradients",
    "hla_conv_forward", "hla_conv_backward_workspace_size", "hla_conv_backward", "hla_conv_step",
    "hla_ssm_workspace_size", "hla_ssm_forward", "hla_ssm_backward", "hla_ssm_step",
    "hla_norm_forward", "hla_norm_backward_workspace_size", "hla_norm_backward",
    "conv_forward", "conv_workspace", "conv_backward", "conv_step", "ConvGradients",
    "ssm_workspace", "ssm_forward", "ssm_backward", "ssm_step", "SsmGradients",
    "norm_forward", "norm_workspace", "norm_backward", "NormGradients",
]

# Every symbol include/hla.h declares.
EXPORTS = ("hla_forward_workspace_size", "hla_forward_chunked", "hla_state_combine", "hla_decode_step",
           "hla_sync_status", "hla_status_string", "hla_last_error", "hla_forward_chunked_noalloc",
           "hla_backward_workspace_size", "hla_backward_chunked", "hla_backward_chunked_traced",
           "hla_forward3_workspace_size", "hla_forward3_chunked", "hla_forward3_chunked_traced", "hla_decode3_step",
           "hla_selftest_expired_wait", "hla_forward_kernel", "hla_backward_chunked_state", "hla_state3_combine",
           "hla_gated_workspace_size", "hla_gated_forward", "hla_gated_backward", "hla_gated_step",
           "hla_window_forward", "hla_window_backward_workspace_size", "hla_window_backward", "hla_window_step",
           "hla_window_cache_fill", "hla_conv_forward", "hla_conv_backward_workspace_size", "hla_conv_backward",
           "hla_conv_step", "hla_ssm_workspace_size", "hla_ssm_forward", "hla_ssm_backward", "hla_ssm_step",
           "hla_norm_forward", "hla_norm_backward_workspace_size", "hla_norm_backward")


class HlaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class hla_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("n", ctypes.c_int), ("d", ctypes.c_int),
                ("dv", ctypes.c_int), ("chunk", ctypes.c_int), ("in_dtype", ctypes.c_int),
                ("flags", ctypes.c_uint), ("eps", ctypes.c_float), ("gamma", ctypes.c_void_p),
                ("Hkv", ctypes.c_int)]


class hla_state(ctypes.Structure):
    _fields_ = [("S", ctypes.c_void_p), ("C", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("G", ctypes.c_void_p), ("h", ctypes.c_void_p)]


class hla_state3(ctypes.Structure):
    _fields_ = [("S", ctypes.c_void_p), ("P", ctypes.c_void_p), ("T", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("SQ", ctypes.c_void_p), ("MQP", ctypes.c_void_p), ("MKQ", ctypes.c_void_p), ("mqm", ctypes.c_void_p)]


class hla_tensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong), ("st", ctypes.c_longlong)]


class hla_gated_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n", ctypes.c_int), ("d", ctypes.c_int), ("in_dtype", ctypes.c_int),
                ("gate", ctypes.c_int), ("rate", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


class hla_window_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("Hkv", ctypes.c_int), ("n", ctypes.c_int),
                ("nk", ctypes.c_int), ("d", ctypes.c_int), ("dv", ctypes.c_int), ("in_dtype", ctypes.c_int),
                ("window", ctypes.c_int), ("sinks", ctypes.c_int), ("scale", ctypes.c_float),
                ("lengths", ctypes.c_void_p)]


class hla_conv_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n", ctypes.c_int), ("d", ctypes.c_int), ("width", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("activation", ctypes.c_int), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


class hla_ssm_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("G", ctypes.c_int), ("n", ctypes.c_int),
                ("P", ctypes.c_int), ("N", ctypes.c_int), ("in_dtype", ctypes.c_int), ("dt_softplus", ctypes.c_int),
                ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p)]


class hla_ssm_gradients(ctypes.Structure):
    _fields_ = [("dx", hla_tensor), ("d_dt", hla_tensor), ("db", hla_tensor), ("dc", hla_tensor),
                ("dA", ctypes.c_void_p), ("dD", ctypes.c_void_p), ("d_dt_bias", ctypes.c_void_p),
                ("d_state_in", ctypes.c_void_p)]


class hla_norm_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n", ctypes.c_int), ("d", ctypes.c_int), ("groups", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("center", ctypes.c_int), ("activation", ctypes.c_int),
                ("gate_first", ctypes.c_int), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


_lib = None


def library(path: str | None = None):
    """Load libhla_gb300.so (raises RuntimeError if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, S, vp, sz = ctypes.POINTER(hla_params), ctypes.POINTER(hla_state), ctypes.c_void_p, ctypes.c_size_t
    i, u, f = ctypes.c_int, ctypes.c_uint, ctypes.c_float
    lib.hla_forward_workspace_size.argtypes = [P]
    lib.hla_forward_workspace_size.restype = sz
    lib.hla_forward_kernel.argtypes = [P]
    lib.hla_forward_kernel.restype = ctypes.c_char_p
    lib.hla_forward_chunked.argtypes = [P, vp, vp, vp, vp, S, S, vp, sz, vp]
    lib.hla_forward_chunked_noalloc.argtypes = [P, vp, vp, vp, vp, S, S, vp]
    lib.hla_forward_chunked_noalloc.restype = ctypes.c_int
    lib.hla_state_combine.argtypes = [i, i, i, u, S, S, S, vp, vp]
    lib.hla_decode_step.argtypes = [i, i, i, i, i, i, u, f, vp, S, vp, vp, vp, vp, vp]
    lib.hla_backward_workspace_size.argtypes = [P]
    lib.hla_backward_workspace_size.restype = sz
    lib.hla_backward_chunked.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hla_backward_chunked_traced.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                                ctypes.POINTER(ctypes.c_void_p)]
    lib.hla_backward_chunked_state.argtypes = [P, vp, vp, vp, vp, ctypes.POINTER(hla_state), vp, vp, vp,
                                               ctypes.POINTER(hla_state), vp, sz, vp]
    S3 = ctypes.POINTER(hla_state3)
    lib.hla_forward3_workspace_size.argtypes = [P]
    lib.hla_forward3_workspace_size.restype = sz
    lib.hla_forward3_chunked.argtypes = [P, vp, vp, vp, vp, S3, S3, vp, sz, vp]
    lib.hla_forward3_chunked_traced.argtypes = [P, vp, vp, vp, vp, S3, S3, vp, sz, vp,
                                                ctypes.POINTER(ctypes.c_void_p)]
    lib.hla_decode3_step.argtypes = [i, i, i, i, i, u, f, vp, S3, vp, vp, vp, vp, vp]
    lib.hla_state3_combine.argtypes = [i, i, i, u, S3, S3, S3, vp, vp]
    lib.hla_sync_status.argtypes = [vp]
    lib.hla_selftest_expired_wait.argtypes = [vp]
    for fn in (lib.hla_forward_chunked, lib.hla_state_combine, lib.hla_decode_step, lib.hla_sync_status,
               lib.hla_backward_chunked, lib.hla_backward_chunked_traced, lib.hla_forward3_chunked,
               lib.hla_forward3_chunked_traced, lib.hla_decode3_step, lib.hla_selftest_expired_wait,
               lib.hla_state3_combine):
        fn.restype = ctypes.c_int
    GP, WP, T = ctypes.POINTER(hla_gated_params), ctypes.POINTER(hla_window_params), ctypes.POINTER(hla_tensor)
    lib.hla_gated_workspace_size.argtypes = [GP]
    lib.hla_gated_workspace_size.restype = sz
    lib.hla_gated_forward.argtypes = [GP, T, T, T, vp, vp, vp, sz, vp]
    lib.hla_gated_backward.argtypes = [GP, T, T, T, T, vp, vp, T, T, vp, vp, vp, sz, vp]
    lib.hla_gated_step.argtypes = [GP, T, T, T, vp, vp, vp]
    lib.hla_window_forward.argtypes = [WP, T, T, T, T, vp, vp]
    lib.hla_window_backward_workspace_size.argtypes = [WP]
    lib.hla_window_backward_workspace_size.restype = sz
    lib.hla_window_backward.argtypes = [WP, T, T, T, T, vp, T, T, T, T, vp, sz, vp]
    lib.hla_window_step.argtypes = [WP, T, T, T, T, T, vp, T, vp]
    lib.hla_window_cache_fill.argtypes = [WP, T, T, T, T, vp]
    for fn in (lib.hla_gated_forward, lib.hla_gated_backward, lib.hla_gated_step, lib.hla_window_forward,
               lib.hla_window_backward, lib.hla_window_step, lib.hla_window_cache_fill):
        fn.restype = ctypes.c_int
    CP, SP, NP = (ctypes.POINTER(t) for t in (hla_conv_params, hla_ssm_params, hla_norm_params))
    lib.hla_conv_forward.argtypes = [CP, T, T, vp, vp, vp]
    lib.hla_conv_backward_workspace_size.argtypes = [CP]
    lib.hla_conv_backward.argtypes = [CP, T, T, T, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hla_conv_step.argtypes = [CP, T, T, vp, vp]
    lib.hla_ssm_workspace_size.argtypes = [SP, i]
    lib.hla_ssm_forward.argtypes = [SP, T, T, T, T, T, vp, vp, vp, sz, vp]
    lib.hla_ssm_backward.argtypes = [SP, T, T, T, T, T, vp, vp, ctypes.POINTER(hla_ssm_gradients), vp, sz, vp]
    lib.hla_ssm_step.argtypes = [SP, T, T, T, T, T, vp, vp]
    lib.hla_norm_forward.argtypes = [NP, T, T, T, vp]
    lib.hla_norm_backward_workspace_size.argtypes = [NP]
    lib.hla_norm_backward.argtypes = [NP, T, T, T, T, T, vp, vp, vp, sz, vp]
    for fn in (lib.hla_conv_backward_workspace_size, lib.hla_ssm_workspace_size, lib.hla_norm_backward_workspace_size):
        fn.restype = sz
    for fn in (lib.hla_conv_forward, lib.hla_conv_backward, lib.hla_conv_step, lib.hla_ssm_forward,
               lib.hla_ssm_backward, lib.hla_ssm_step, lib.hla_norm_forward, lib.hla_norm_backward):
        fn.restype = ctypes.c_int
    lib.hla_status_string.argtypes = [ctypes.c_int]
    lib.hla_status_string.restype = ctypes.c_char_p
    lib.hla_last_error.argtypes = []
    lib.hla_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same handle without the object around it
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != HLA_OK:
        lib = library()
        raise HlaError(status, lib.hla_last_error().decode() or lib.hla_status_string(status).decode())


def _state_struct(st):
    if st is None:
        return None
    if isinstance(st, hla_state):
        return ctypes.pointer(st)
    return ctypes.pointer(hla_state(_ptr(st.S), _ptr(st.C), _ptr(st.m), _ptr(st.G), _ptr(st.h)))


# --------------------------------------------------------------------- raw ABI
def hla_status_string(status: int) -> str:
    return library().hla_status_string(status).decode()


def hla_last_error() -> str:
    return library().hla_last_error().decode()


def hla_forward_workspace_size(params: hla_params) -> int:
    return library().hla_forward_workspace_size(ctypes.byref(params))


def hla_forward_kernel(params: hla_params):
    """Name of the kernel the forward launches for these parameters (None: no launch)."""
    r = library().hla_forward_kernel(ctypes.byref(params))
    return r.decode() if r else None


def hla_forward_chunked(params: hla_params, q, k, v, o, state_in=None, state_out=None, workspace=None,
                        workspace_bytes: int = 0, stream=None) -> None:
    _check(library().hla_forward_chunked(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                         _state_struct(state_in), _state_struct(state_out), _ptr(workspace),
                                         workspace_bytes, _stream(stream)))


def hla_forward_chunked_noalloc(params: hla_params, q, k, v, o, state_in=None, state_out=None,
                                stream=None) -> None:
    """The forward without a caller workspace, for callers that cannot allocate
    device memory (the scratch is a fixed array inside the library; see hla.h)."""
    _check(library().hla_forward_chunked_noalloc(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                                 _state_struct(state_in), _state_struct(state_out),
                                                 _stream(stream)))


def hla_state_combine(count: int, d: int, dv: int, flags: int, A, B, out, decay_pow=None, stream=None) -> None:
    _check(library().hla_state_combine(count, d, dv, flags, _state_struct(A), _state_struct(B), _state_struct(out),
                                       _ptr(decay_pow), _stream(stream)))


def hla_decode_step(N: int, H: int, Hkv: int, d: int, dv: int, dtype: int, flags: int, eps: float, gamma,
                    state, q, k, v, o, stream=None) -> None:
    _check(library().hla_decode_step(N, H, Hkv, d, dv, dtype, flags, eps, _ptr(gamma), _state_struct(state),
                                     _ptr(q), _ptr(k), _ptr(v), _ptr(o), _stream(stream)))


def hla_backward_workspace_size(params: hla_params) -> int:
    return library().hla_backward_workspace_size(ctypes.byref(params))


def hla_backward_chunked(params: hla_params, q, k, v, dout, dq, dk, dv, workspace, workspace_bytes: int,
                         stream=None) -> None:
    _check(library().hla_backward_chunked(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq),
                                          _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes, _stream(stream)))


def hla_backward_chunked_state(params: hla_params, q, k, v, dout, state_in, dq, dk, dv, d_state_in, workspace,
                               workspace_bytes: int, stream=None) -> None:
    _check(library().hla_backward_chunked_state(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                                                _state_struct(state_in), _ptr(dq), _ptr(dk), _ptr(dv),
                                                _state_struct(d_state_in), _ptr(workspace), workspace_bytes,
                                                _stream(stream)))


def hla_backward_chunked_traced(params: hla_params, q, k, v, dout, dq, dk, dv, workspace, workspace_bytes: int,
                                stream=None, events=None) -> None:
    """hla_backward_chunked recording four events (torch.cuda.Event that have been
    recorded once, or raw cudaEvent_t ints) at its phase boundaries."""
    arr = None
    if events is not None:
        hs = [e if isinstance(e, int) else e.cuda_event for e in events]
        assert len(hs) == 4 and all(hs), "four created events are needed"
        arr = (ctypes.c_void_p * 4)(*hs)
    _check(library().hla_backward_chunked_traced(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                                                 _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace_bytes,
                                                 _stream(stream), arr))


def _state3_struct(st):
    if st is None:
        return None
    return ctypes.byref(hla_state3(*(_ptr(x) for x in (st.S, st.P, st.T, st.m, st.h, st.SQ, st.MQP, st.MKQ,
                                                         st.mqm))))


def _events(events):
    if events is None:
        return None
    hs = [e if isinstance(e, int) else e.cuda_event for e in events]
    assert len(hs) == 4 and all(hs), "four created events are needed"
    return (ctypes.c_void_p * 4)(*hs)


def hla_forward3_workspace_size(params: hla_params) -> int:
    return library().hla_forward3_workspace_size(ctypes.byref(params))


def hla_forward3_chunked(params: hla_params, q, k, v, o, state_in=None, state_out=None, workspace=None,
                         workspace_bytes: int = 0, stream=None) -> None:
    _check(library().hla_forward3_chunked(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                          _state3_struct(state_in), _state3_struct(state_out), _ptr(workspace),
                                          workspace_bytes, _stream(stream)))


def hla_forward3_chunked_traced(params: hla_params, q, k, v, o, state_in=None, state_out=None, workspace=None,
                                workspace_bytes: int = 0, stream=None, events=None) -> None:
    _check(library().hla_forward3_chunked_traced(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                                 _state3_struct(state_in), _state3_struct(state_out),
                                                 _ptr(workspace), workspace_bytes, _stream(stream),
                                                 _events(events)))


def hla_decode3_step(N: int, H: int, d: int, dv: int, dtype: int, flags: int, eps: float, gamma, state, q, k, v, o,
                     stream=None) -> None:
    _check(library().hla_decode3_step(N, H, d, dv, dtype, flags, eps, _ptr(gamma), _state3_struct(state), _ptr(q),
                                      _ptr(k), _ptr(v), _ptr(o), _stream(stream)))


def hla_state3_combine(count: int, d: int, dv: int, flags: int, A, B, out, decay_pow=None, stream=None) -> None:
    _check(library().hla_state3_combine(count, d, dv, flags, _state3_struct(A), _state3_struct(B),
                                        _state3_struct(out), _ptr(decay_pow), _stream(stream)))


def hla_selftest_expired_wait(stream=None) -> None:
    """Launch the failure-path self-test (a bounded wait that expires); the next
    hla_sync_status reports HLA_ERR_TIMEOUT."""
    _check(library().hla_selftest_expired_wait(_stream(stream)))


def hla_sync_status(stream=None) -> None:
    _check(library().hla_sync_status(_stream(stream)))


def hla_gated_workspace_size(params: hla_gated_params) -> int:
    return library().hla_gated_workspace_size(ctypes.byref(params))


def hla_gated_forward(params: hla_gated_params, x, g, y, state_in=None, state_out=None, workspace=None,
                      workspace_bytes: int = 0, stream=None) -> None:
    _check(library().hla_gated_forward(ctypes.byref(params), x, g, y, _ptr(state_in), _ptr(state_out),
                                       _ptr(workspace), workspace_bytes, _stream(stream)))


def hla_gated_backward(params: hla_gated_params, x, g, y, dy, state_in, d_state_out, dx, dg, d_rate, d_state_in,
                       workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(library().hla_gated_backward(ctypes.byref(params), x, g, y, dy, _ptr(state_in), _ptr(d_state_out), dx, dg,
                                        _ptr(d_rate), _ptr(d_state_in), _ptr(workspace), workspace_bytes,
                                        _stream(stream)))


def hla_gated_step(params: hla_gated_params, x, g, y, state, state_out, stream=None) -> None:
    _check(library().hla_gated_step(ctypes.byref(params), x, g, y, _ptr(state), _ptr(state_out), _stream(stream)))


def hla_window_forward(params: hla_window_params, q, k, v, o, lse=None, stream=None) -> None:
    _check(library().hla_window_forward(ctypes.byref(params), q, k, v, o, _ptr(lse), _stream(stream)))


def hla_window_backward_workspace_size(params: hla_window_params) -> int:
    return library().hla_window_backward_workspace_size(ctypes.byref(params))


def hla_window_backward(params: hla_window_params, q, k, v, o, lse, dout, dq, dk, dv, workspace,
                        workspace_bytes: int, stream=None) -> None:
    _check(library().hla_window_backward(ctypes.byref(params), q, k, v, o, _ptr(lse), dout, dq, dk, dv,
                                         _ptr(workspace), workspace_bytes, _stream(stream)))


def hla_window_step(params: hla_window_params, q, k, v, kc, vc, pos, o, stream=None) -> None:
    _check(library().hla_window_step(ctypes.byref(params), q, k, v, kc, vc, _ptr(pos), o, _stream(stream)))


def hla_window_cache_fill(params: hla_window_params, k, v, kc, vc, stream=None) -> None:
    _check(library().hla_window_cache_fill(ctypes.byref(params), k, v, kc, vc, _stream(stream)))


def hla_conv_forward(params: hla_conv_params, x, y, state_in=None, state_out=None, stream=None) -> None:
    _check(library().hla_conv_forward(ctypes.byref(params), x, y, _ptr(state_in), _ptr(state_out), _stream(stream)))


def hla_conv_backward_workspace_size(params: hla_conv_params) -> int:
    return library().hla_conv_backward_workspace_size(ctypes.byref(params))


def hla_conv_backward(params: hla_conv_params, x, dy, dx, state_in, d_state_out, d_weight, d_bias, d_state_in,
                      workspace, workspace_bytes: int, stream=None) -> None:
    _check(library().hla_conv_backward(ctypes.byref(params), x, dy, dx, _ptr(state_in), _ptr(d_state_out),
                                       _ptr(d_weight), _ptr(d_bias), _ptr(d_state_in), _ptr(workspace),
                                       workspace_bytes, _stream(stream)))


def hla_conv_step(params: hla_conv_params, x, y, state, stream=None) -> None:
    _check(library().hla_conv_step(ctypes.byref(params), x, y, _ptr(state), _stream(stream)))


def hla_ssm_workspace_size(params: hla_ssm_params, backward: bool) -> int:
    return library().hla_ssm_workspace_size(ctypes.byref(params), 1 if backward else 0)


def hla_ssm_forward(params: hla_ssm_params, x, dt, b, c, y, state_in, state_out, workspace, workspace_bytes: int,
                    stream=None) -> None:
    _check(library().hla_ssm_forward(ctypes.byref(params), x, dt, b, c, y, _ptr(state_in), _ptr(state_out),
                                     _ptr(workspace), workspace_bytes, _stream(stream)))


def hla_ssm_backward(params: hla_ssm_params, x, dt, b, c, dy, state_in, d_state_out, grads: hla_ssm_gradients,
                     workspace, workspace_bytes: int, stream=None) -> None:
    _check(library().hla_ssm_backward(ctypes.byref(params), x, dt, b, c, dy, _ptr(state_in), _ptr(d_state_out),
                                      ctypes.byref(grads), _ptr(workspace), workspace_bytes, _stream(stream)))


def hla_ssm_step(params: hla_ssm_params, x, dt, b, c, y, state, stream=None) -> None:
    _check(library().hla_ssm_step(ctypes.byref(params), x, dt, b, c, y, _ptr(state), _stream(stream)))


def hla_norm_forward(params: hla_norm_params, x, gate, y, stream=None) -> None:
    _check(library().hla_norm_forward(ctypes.byref(params), x, gate, y, _stream(stream)))


def hla_norm_backward_workspace_size(params: hla_norm_params) -> int:
    return library().hla_norm_backward_workspace_size(ctypes.byref(params))


def hla_norm_backward(params: hla_norm_params, x, gate, dy, dx, d_gate, d_weight, d_bias, workspace,
                      workspace_bytes: int, stream=None) -> None:
    _check(library().hla_norm_backward(ctypes.byref(params), x, gate, dy, dx, d_gate, _ptr(d_weight), _ptr(d_bias),
                                       _ptr(workspace), workspace_bytes, _stream(stream)))


# ------------------------------------------------------- tensor-level helpers
@dataclass
class State:
    """Five fp32 summaries of `units` pairs: S [U,d,d], C [U,d,dv], m [U,d], G [U,d,dv], h [U,d]."""
    S: object
    C: object
    m: object
    G: object
    h: object

    @staticmethod
    def empty(units: int, d: int, dv: int, device="cuda") -> "State":
        import torch
        z = lambda *s: torch.empty(*s, dtype=torch.float32, device=device)
        return State(z(units, d, d), z(units, d, dv), z(units, d), z(units, d, dv), z(units, d))

    @staticmethod
    def zeros(units: int, d: int, dv: int, device="cuda") -> "State":
        import torch
        z = lambda *s: torch.zeros(*s, dtype=torch.float32, device=device)
        return State(z(units, d, d), z(units, d, dv), z(units, d), z(units, d, dv), z(units, d))

    def astuple(self):
        return (self.S, self.C, self.m, self.G, self.h)


@dataclass
class State3:
    """Third-order streaming state of `units` pairs, fp32: S [U,d,d] (key moment S^K),
    P [U,d,dv] (key-value moment), T [U,d,dv] (masked third-order accumulator); with
    ratio normalisation also m [U,d] (key mass) and h [U,d] (T of a unit value); with
    the segment maps (for state3_combine) SQ [U,d,d], MQP [U,d,dv], MKQ [U,d,d] and,
    normalised, mqm [U,d]."""
    S: object
    P: object
    T: object
    m: object = None
    h: object = None
    SQ: object = None
    MQP: object = None
    MKQ: object = None
    mqm: object = None

    @staticmethod
    def _make(z, units, d, dv, normalize, maps):
        mh = (z(units, d), z(units, d)) if normalize else (None, None)
        mp = (z(units, d, d), z(units, d, dv), z(units, d, d), z(units, d) if normalize else None) if maps else \
            (None,) * 4
        return State3(z(units, d, d), z(units, d, dv), z(units, d, dv), *mh, *mp)

    @staticmethod
    def empty(units: int, d: int, dv: int, device="cuda", normalize: bool = False, maps: bool = False) -> "State3":
        import torch
        return State3._make(lambda *s: torch.empty(*s, dtype=torch.float32, device=device), units, d, dv, normalize,
                            maps)

    @staticmethod
    def zeros(units: int, d: int, dv: int, device="cuda", normalize: bool = False, maps: bool = False) -> "State3":
        import torch
        return State3._make(lambda *s: torch.zeros(*s, dtype=torch.float32, device=device), units, d, dv, normalize,
                            maps)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return HLA_F32
    if t.dtype == torch.bfloat16:
        return HLA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _variant_flags(unmasked: bool, asymmetric: bool) -> int:
    return (HLA_UNMASKED if unmasked else 0) | (HLA_ASYMMETRIC if asymmetric else 0)


def make_params(q, v, chunk: int, gamma=None, normalize: bool = False, eps: float = 0.0,
                unmasked: bool = False, asymmetric: bool = False) -> hla_params:
    """Parameters for q [B,H,n,d] and v [B,Hkv,n,dv] (Hkv = H, or a divisor of H when
    key/value heads are shared)."""
    B, H, n, d = q.shape
    flags = (HLA_NORMALIZE if normalize else 0) | (HLA_DECAY if gamma is not None else 0) | \
        _variant_flags(unmasked, asymmetric)
    return hla_params(B, H, n, d, v.shape[-1], chunk, _dtype_code(q), flags, float(eps), _ptr(gamma),
                      v.shape[1])


def new_workspace(nbytes: int, device="cuda"):
    """A zeroed device workspace of `nbytes` (each forward call leaves it ready for the next)."""
    import torch
    return torch.zeros(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def forward(q, k, v, chunk: int, gamma=None, normalize: bool = False, eps: float = 0.0, state_in=None,
            return_state: bool = False, out=None, workspace=None, stream=None, unmasked: bool = False,
            asymmetric: bool = False):
    """2nd-order HLA forward (masked; unmasked with ``unmasked=True``; the asymmetric
    variant AHLA with ``asymmetric=True``, state R, P, m^K, E, n).  q [B,H,n,d],
    k [B,Hkv,n,d], v [B,Hkv,n,dv] contiguous CUDA tensors (bf16 or fp32; Hkv divides H);
    gamma [H] fp32 or None.  Returns o (and the final State)."""
    import torch
    p = make_params(q, v, chunk, gamma, normalize, eps, unmasked, asymmetric)
    o = out if out is not None else torch.empty(q.shape[:3] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    need = hla_forward_workspace_size(p)
    if workspace is None and need:
        workspace = new_workspace(need, q.device)
    st = State.empty(p.B * p.H, p.d, p.dv, device=q.device) if return_state else None
    hla_forward_chunked(p, q, k, v, o, state_in, st, workspace, need if workspace is not None else 0, stream)
    return (o, st) if return_state else o


def state_combine(A: State, B: State, decay_pow=None, out: State | None = None, stream=None,
                  unmasked: bool = False, asymmetric: bool = False) -> State:
    count, d, dv = A.C.shape
    out = out if out is not None else State.empty(count, d, dv, device=A.S.device)
    hla_state_combine(count, d, dv, _variant_flags(unmasked, asymmetric), A, B, out, decay_pow, stream)
    return out


def decode_step(state: State, q, k, v, H: int, gamma=None, normalize: bool = False, eps: float = 0.0,
                out=None, stream=None, unmasked: bool = False, asymmetric: bool = False):
    """One decode step for N pairs (q [N,d]; k [N/H*Hkv,d], v [N/H*Hkv,dv]); state
    updated in place."""
    import torch
    N, d = q.shape
    dv = v.shape[-1]
    Hkv = k.shape[0] * H // N if N else H
    o = out if out is not None else torch.empty((N, dv), dtype=q.dtype, device=q.device)
    flags = (HLA_NORMALIZE if normalize else 0) | (HLA_DECAY if gamma is not None else 0) | \
        _variant_flags(unmasked, asymmetric)
    hla_decode_step(N, H, Hkv, d, dv, _dtype_code(q), flags, float(eps), gamma, state, q, k, v, o, stream)
    return o


def backward(q, k, v, dout, chunk: int, gamma=None, workspace=None, out=None, stream=None,
             normalize: bool = False, eps: float = 0.0, state_in: State | None = None, want_dstate: bool = False):
    """Gradients (dq, dk, dv) of sum(dout * o) for the masked forward o of q, k, v from a
    zero state, or from ``state_in`` (with ``normalize=True`` the ratio-normalised o).  q [B,H,n,d], k [B,Hkv,n,d], v [B,Hkv,n,dv], dout [B,H,n,dv]
    contiguous CUDA tensors of one dtype (bf16 or fp32); gamma [H] fp32 or None.
    ``out`` may hold three preallocated result tensors.  ``want_dstate``: also return the
    gradient with respect to the initial state (a State)."""
    import torch
    p = make_params(q, v, chunk, gamma, normalize, eps)
    need = hla_backward_workspace_size(p)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dq, dk, dv = out if out is not None else (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    if state_in is None and not want_dstate:
        hla_backward_chunked(p, q, k, v, dout, dq, dk, dv, workspace, need if workspace is not None else 0, stream)
        return dq, dk, dv
    dst = State.empty(p.B * p.H, p.d, p.dv, device=q.device) if want_dstate else None
    hla_backward_chunked_state(p, q, k, v, dout, state_in, dq, dk, dv, dst, workspace,
                               need if workspace is not None else 0, stream)
    return (dq, dk, dv, dst) if want_dstate else (dq, dk, dv)


def forward3(q, k, v, chunk: int, state_in: State3 | None = None, return_state: bool = False, out=None,
             workspace=None, stream=None, gamma=None, normalize: bool = False, eps: float = 0.0, maps: bool = False):
    """Masked third-order HLA forward.  q, k [B,H,n,d], v [B,H,n,dv] contiguous CUDA
    tensors (bf16 or fp32); gamma: [H] fp32 CUDA tensor of decay rates or None;
    normalize: o = num / (den + eps).  Returns o (and the final State3)."""
    import torch
    p = make_params(q, v, chunk, gamma, normalize, eps)
    o = out if out is not None else torch.empty(q.shape[:3] + (v.shape[-1],), dtype=q.dtype, device=q.device)
    need = hla_forward3_workspace_size(p)
    if workspace is None and need:
        workspace = new_workspace(need, device=q.device)
    st = State3.empty(p.B * p.H, p.d, p.dv, device=q.device, normalize=normalize, maps=maps) if return_state else None
    hla_forward3_chunked(p, q, k, v, o, state_in, st, workspace, need if workspace is not None else 0, stream)
    return (o, st) if return_state else o


def state3_combine(A: State3, B: State3, decay_pow=None, normalize: bool = False, out: State3 | None = None,
                   stream=None) -> State3:
    """Concatenation (A before B) of third-order states with their segment maps, item by
    item; decay_pow [U] fp32 = gamma^(tokens of B) or None."""
    units, d, dv = A.P.shape
    if out is None:
        out = State3.empty(units, d, dv, device=A.P.device, normalize=normalize, maps=True)
    hla_state3_combine(units, d, dv, HLA_NORMALIZE if normalize else 0, A, B, out, decay_pow, stream)
    return out


def decode3_step(state: State3, q, k, v, out=None, stream=None, H: int = 1, gamma=None, normalize: bool = False,
                 eps: float = 0.0):
    """One third-order decode step for N pairs (q, k [N,d], v [N,dv]); state updated in
    place.  gamma: [H] decay rates (pair i uses gamma[i % H]) or None."""
    import torch
    N, d = q.shape
    dv = v.shape[-1]
    o = out if out is not None else torch.empty((N, dv), dtype=q.dtype, device=q.device)
    flags = (HLA_DECAY if gamma is not None else 0) | (HLA_NORMALIZE if normalize else 0)
    hla_decode3_step(N, H, d, dv, _dtype_code(q), flags, float(eps), gamma, state, q, k, v, o, stream)
    return o


# ------------------------------------------------- gated recurrence, windowed attention
_GATES = {"given": HLA_GATE_GIVEN, "sigmoid": HLA_GATE_SIGMOID, "rate": HLA_GATE_RATE}
GatedGradients = namedtuple("GatedGradients", "dx dg d_rate d_state_in")


def _expect(t, name, shape, dtype, device, contiguous=False):
    """Shape, type and device of one argument; its channels have to be adjacent."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.is_contiguous():
        return
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of the last dimension must be adjacent")


def _current(t):
    """The kernels run on the current device: refuse tensors of another one."""
    import torch
    if not t.is_cuda:
        raise ValueError("CUDA tensors are needed")
    dev = t.device
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


_NO_CONTEXT = contextlib.nullcontext()


def _on(stream, device):
    """What a call allocates belongs to the stream the call runs on, one of its tensors' device
    (entering another device's stream would make that device the current one)."""
    if stream is None:
        return _NO_CONTEXT
    import torch
    if isinstance(stream, int):  # (0 given to ExternalStream makes a stream of its own)
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _t2(t):
    """[B, d] rows, or [B, n, d]."""
    s = t.stride()
    return hla_tensor(t.data_ptr(), s[0], 0, s[1] if len(s) == 3 else 0)


def _t4(t):
    """[B, H, w] rows, or [B, H, n, w]."""
    s = t.stride()
    return hla_tensor(t.data_ptr(), s[0], s[1], s[2] if len(s) == 4 else 0)


def _zeroed(like, shapes):
    """Zeroed tensors of these shapes, by one launch."""
    import torch
    out = tuple(torch.empty(s, dtype=like.dtype, device=like.device) for s in shapes)
    torch._foreach_zero_(out)
    return out


def _int32(x, name):
    """ctypes would cut a larger number to its low bits."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _fits(*tensors):
    """The same of sizes (strides are 64 bits wide)."""
    for t in tensors:
        if not 0 < t.numel() < 2 ** 31 and max(t.shape) >= 2 ** 31:  # (the largest of a shape takes longer to find)
            raise ValueError(f"a size of {max(t.shape)} does not fit 32 bits")


def _gated_params(x, g, gate, rate, lengths, device):
    if gate not in _GATES:
        raise ValueError(f"gate must be one of {sorted(_GATES)}")
    import torch
    code = _dtype_code(x)
    shape, dtype = x.shape, x.dtype
    B, d = shape[0], shape[-1]
    n = shape[1] if len(shape) == 3 else 1
    _expect(x, "x", shape, dtype, device)
    _expect(g, "g", shape, dtype, device)
    if (rate is not None) != (gate == "rate"):
        raise ValueError("rate belongs to gate='rate', which needs it")
    if rate is not None:
        _expect(rate, "rate", (d,), torch.float32, device, True)
    if lengths is not None:
        _expect(lengths, "lengths", (B,), torch.int32, device, True)
    return hla_gated_params(B, n, d, code, _GATES[gate], _ptr(rate), _ptr(lengths))


def _optional(t, name, shape, dtype, device):
    if t is not None:
        _expect(t, name, shape, dtype, device, True)


def _space(need, workspace, device, zeroed):
    """(workspace, bytes) of a call that needs `need` bytes."""
    import torch
    if workspace is None:
        if not need:
            return None, 0
        workspace = new_workspace(need, device) if zeroed else torch.empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("the workspace must be a contiguous tensor on the same device")
    return workspace, workspace.numel() * workspace.element_size()


def gated_workspace(x, stream=None):
    """A zeroed workspace for gated_forward and gated_backward of x [B,n,d], about half of B n d
    bytes; each call leaves it ready for the next.  Calls that may overlap in time need one each.
    A call of more than 64 tokens without one allocates and zeroes it anew."""
    B, n, d = x.shape
    with _on(stream, x.device):
        return new_workspace(hla_gated_workspace_size(hla_gated_params(B, n, d, _dtype_code(x), 0, None, None)), x.device)


def gated_forward(x, g, gate: str = "given", rate=None, state_in=None, return_state: bool = False, lengths=None,
                  out=None, workspace=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + b_t over x, g [B,n,d] (bf16 or fp32, any
    strides with adjacent channels): gate "given" a = g, b = x; "sigmoid" a = sigma(g),
    b = (1 - a) x; "rate" a = exp(-rate sigma(g)), b = sqrt(1 - a^2) x with rate [d] fp32,
    positive.  state_in [B,d] fp32 or None (zeros); lengths [B] int32: tokens of each
    sequence (rows behind them: zero in a new y, left as they were in ``out``).  Returns
    y [B,n,d] (and the final state [B,d] fp32)."""
    import torch
    dev = _current(x)
    if x.dim() != 3:
        raise ValueError("x must be [B, n, d]")
    p = _gated_params(x, g, gate, rate, lengths, dev)
    _optional(state_in, "state_in", (p.B, p.d), torch.float32, dev)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        st = torch.empty((p.B, p.d), dtype=torch.float32, device=dev) if return_state else None
        ws, nbytes = _space(hla_gated_workspace_size(p) if p.n > 64 or workspace is not None else 0, workspace, dev, True)
        hla_gated_forward(p, _t2(x), _t2(g), _t2(out), state_in, st, ws, nbytes, stream)
    return (out, st) if return_state else out


def gated_backward(x, g, y, dy, gate: str = "given", rate=None, state_in=None, d_state_out=None,
                   want_dstate: bool = False, lengths=None, out=None, workspace=None, stream=None):
    """Gradients of gated_forward from its y and the gradients dy of y and d_state_out [B,d]
    fp32 of the final state (None: zero).  Returns GatedGradients(dx, dg, d_rate, d_state_in):
    d_rate [d] fp32 with gate "rate" (else None), d_state_in [B,d] fp32 with want_dstate
    (else None).  ``out`` may hold two tensors for dx and dg."""
    import torch
    dev = _current(x)
    if x.dim() != 3:
        raise ValueError("x must be [B, n, d]")
    p = _gated_params(x, g, gate, rate, lengths, dev)
    _expect(y, "y", x.shape, x.dtype, dev)
    _expect(dy, "dy", x.shape, x.dtype, dev)
    _optional(state_in, "state_in", (p.B, p.d), torch.float32, dev)
    _optional(d_state_out, "d_state_out", (p.B, p.d), torch.float32, dev)
    with _on(stream, dev):
        new = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)  # noqa: E731
        if out is None:
            out = _zeroed(x, (x.shape, x.shape)) if lengths is not None else \
                (torch.empty(x.shape, dtype=x.dtype, device=dev), torch.empty(x.shape, dtype=x.dtype, device=dev))
        dx, dg = out
        _expect(dx, "dx", x.shape, x.dtype, dev)
        _expect(dg, "dg", x.shape, x.dtype, dev)
        dr = new(p.d) if gate == "rate" else None
        ds = new(p.B, p.d) if want_dstate else None
        ws, nbytes = _space(hla_gated_workspace_size(p) if p.n > 64 or dr is not None or workspace is not None else 0,
                            workspace, dev, True)
        hla_gated_backward(p, _t2(x), _t2(g), _t2(y), _t2(dy), state_in, d_state_out, _t2(dx), _t2(dg), dr, ds, ws,
                           nbytes, stream)
    return GatedGradients(dx, dg, dr, ds)


def gated_step(state, x, g, gate: str = "given", rate=None, lengths=None, state_out=None, out=None, stream=None):
    """One token of every sequence: x, g [B,d], state [B,d] fp32 updated in place, or read and
    the new one written to ``state_out``.  lengths [B] int32: 0 marks an idle sequence, whose
    rows of y (zero in a new one) and of the state are left as they were.  Returns (y, state)."""
    import torch
    dev = _current(x)
    if x.dim() != 2:
        raise ValueError("x must be [B, d]")
    p = _gated_params(x, g, gate, rate, lengths, dev)
    _expect(state, "state", x.shape, torch.float32, dev, True)
    if state_out is None:
        state_out = state
    else:
        _expect(state_out, "state_out", x.shape, torch.float32, dev, True)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        hla_gated_step(p, _t2(x), _t2(g), _t2(out), state, state_out, stream)
    return out, state_out


def _window_params(q, k, v, window, sinks, scale, lengths, device):
    import torch
    code = _dtype_code(q)
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B, heads, tokens, width]")
    B, H, n, d = q.shape
    Hkv, nk, dv = k.shape[1], k.shape[2], v.shape[3]
    _expect(q, "q", q.shape, q.dtype, device)
    _expect(k, "k", (B, Hkv, nk, d), q.dtype, device)
    _expect(v, "v", (B, Hkv, nk, dv), q.dtype, device)
    if lengths is not None:
        _expect(lengths, "lengths", (B,), torch.int32, device, True)
    return hla_window_params(B, H, Hkv, n, nk, d, dv, code, _int32(window, "window"), _int32(sinks, "sinks"),
                             d ** -0.5 if scale is None else scale, _ptr(lengths))


def window_forward(q, k, v, window: int, sinks: int = 0, scale: float | None = None, lengths=None,
                   return_lse: bool = False, out=None, stream=None):
    """Softmax attention of q [B,H,n,d] over k [B,Hkv,nk,d], v [B,Hkv,nk,dv] (bf16 or fp32,
    widths up to 128, any strides with adjacent channels): the query at position
    p = nk - n + i sees the keys j <= p with j > p - window or j < sinks.  scale: 1/sqrt(d)
    unless given.  lengths [B] int32: tokens of each sequence; rows behind them are zero in a
    new o, left as they were in ``out``.  Returns o [B,H,n,dv] (and lse [B,H,n] fp32)."""
    import torch
    dev = _current(q)
    p = _window_params(q, k, v, window, sinks, scale, lengths, dev)
    with _on(stream, dev):
        make = torch.zeros if lengths is not None else torch.empty
        if out is None:
            out = make((p.B, p.H, p.n, p.dv), dtype=q.dtype, device=dev)
        else:
            _expect(out, "out", (p.B, p.H, p.n, p.dv), q.dtype, dev)
        lse = make((p.B, p.H, p.n), dtype=torch.float32, device=dev) if return_lse else None
        hla_window_forward(p, _t4(q), _t4(k), _t4(v), _t4(out), lse, stream)
    return (out, lse) if return_lse else out


def window_workspace(q, k, v, window: int, sinks: int = 0, stream=None):
    """A workspace for window_backward of these shapes: B H n floats, and with first tokens up to
    a few fp32 copies of their dk and dv."""
    import torch
    p = _window_params(q, k, v, window, sinks, None, None, q.device)
    with _on(stream, q.device):
        return torch.empty(max(hla_window_backward_workspace_size(p), 1), dtype=torch.uint8, device=q.device)


def window_backward(q, k, v, o, lse, dout, window: int, sinks: int = 0, scale: float | None = None, lengths=None,
                    out=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * o) for window_forward, from its o and lse.  ``out``
    may hold the three result tensors; rows behind the lengths are zero in new ones, left as
    they were in those."""
    import torch
    dev = _current(q)
    p = _window_params(q, k, v, window, sinks, scale, lengths, dev)
    _expect(o, "o", (p.B, p.H, p.n, p.dv), q.dtype, dev)
    _expect(dout, "dout", (p.B, p.H, p.n, p.dv), q.dtype, dev)
    _expect(lse, "lse", (p.B, p.H, p.n), torch.float32, dev, True)
    with _on(stream, dev):
        if out is None:
            shapes = (q.shape, k.shape, v.shape)
            out = _zeroed(q, shapes) if lengths is not None else \
                tuple(torch.empty(x, dtype=q.dtype, device=dev) for x in shapes)
        dq, dk, dv = out
        for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
            _expect(t, name, like.shape, q.dtype, dev)
        ws, nbytes = _space(hla_window_backward_workspace_size(p) if workspace is None else 0, workspace, dev, False)
        hla_window_backward(p, _t4(q), _t4(k), _t4(v), _t4(o), lse, _t4(dout), _t4(dq), _t4(dk), _t4(dv), ws, nbytes,
                            stream)
    return dq, dk, dv


def window_cache(B: int, Hkv: int, window: int, sinks: int, d: int, dv: int | None = None, dtype=None, device="cuda"):
    """Ring cache (kc [B,Hkv,sinks+window,d], vc [B,Hkv,sinks+window,dv]) for window_step,
    bf16 unless given; slots are written before they are read, so it is not cleared."""
    import torch
    new = lambda w: torch.empty((B, Hkv, sinks + window, w), dtype=dtype or torch.bfloat16, device=device)  # noqa: E731
    return new(d), new(d if dv is None else dv)


def _cache_params(kc, vc, q_heads, window, sinks, scale, lengths, nk, device):
    import torch
    if kc.dim() != 4 or vc.dim() != 4:
        raise ValueError("kc and vc must be [B, Hkv, sinks + window, width]")
    B, Hkv, d, dv = kc.shape[0], kc.shape[1], kc.shape[3], vc.shape[3]
    _expect(kc, "kc", (B, Hkv, sinks + window, d), kc.dtype, device)
    _expect(vc, "vc", (B, Hkv, sinks + window, dv), kc.dtype, device)
    if lengths is not None:
        _expect(lengths, "lengths", (B,), torch.int32, device, True)
    return hla_window_params(B, q_heads, Hkv, 1, nk, d, dv, _dtype_code(kc), _int32(window, "window"),
                             _int32(sinks, "sinks"), d ** -0.5 if scale is None else scale, _ptr(lengths))


def window_cache_fill(kc, vc, k, v, window: int, sinks: int = 0, lengths=None, stream=None) -> None:
    """The cache after a prompt k [B,Hkv,n,d], v [B,Hkv,n,dv]: the first ``sinks`` and the last
    ``window`` tokens of every sequence (lengths [B] int32, None: n).  Decoding goes on at
    pos = the lengths."""
    dev = _current(kc)
    p = _cache_params(kc, vc, kc.shape[1], window, sinks, None, lengths, k.shape[2], dev)
    _expect(k, "k", (p.B, p.Hkv, p.nk, p.d), kc.dtype, dev)
    _expect(v, "v", (p.B, p.Hkv, p.nk, p.dv), kc.dtype, dev)
    with _on(stream, dev):
        hla_window_cache_fill(p, _t4(k), _t4(v), _t4(kc), _t4(vc), stream)


def window_step(kc, vc, pos, q, k, v, window: int, sinks: int = 0, scale: float | None = None, out=None, stream=None):
    """One token of every sequence: writes k [B,Hkv,d], v [B,Hkv,dv] into the ring cache at the
    token's slot and attends q [B,H,d] over the visible slots.  pos [B] int64: the tokens
    before this one (advanced by the caller), or negative for an idle sequence, whose row of o
    (zero in a new one) and cache are left as they were.  Returns o [B,H,dv]."""
    import torch
    dev = _current(q)
    if q.dim() != 3:
        raise ValueError("q must be [B, H, d]")
    p = _cache_params(kc, vc, q.shape[1], window, sinks, scale, None, 1, dev)
    _expect(q, "q", (p.B, p.H, p.d), kc.dtype, dev)
    _expect(k, "k", (p.B, p.Hkv, p.d), kc.dtype, dev)
    _expect(v, "v", (p.B, p.Hkv, p.dv), kc.dtype, dev)
    _expect(pos, "pos", (p.B,), torch.int64, dev, True)
    with _on(stream, dev):
        if out is None:
            out = torch.zeros((p.B, p.H, p.dv), dtype=q.dtype, device=dev)
        else:
            _expect(out, "out", (p.B, p.H, p.dv), q.dtype, dev)
        hla_window_step(p, _t4(q), _t4(k), _t4(v), _t4(kc), _t4(vc), pos, _t4(out), stream)
    return out


# ------------------------------------------------------- selective state space layer
_ACTIVATIONS = {"none": HLA_ACT_NONE, "silu": HLA_ACT_SILU}
ConvGradients = namedtuple("ConvGradients", "dx d_weight d_bias d_state_in")
SsmGradients = namedtuple("SsmGradients", "dx d_dt dA dB dC dD d_dt_bias d_state_in")
NormGradients = namedtuple("NormGradients", "dx d_gate d_weight d_bias")


def _activation(name):
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
    return _ACTIVATIONS[name]


def _conv_params(x, weight, bias, activation, lengths, device):
    import torch
    code = _dtype_code(x)
    B, d = x.shape[0], x.shape[-1]
    _expect(x, "x", x.shape, x.dtype, device)
    if weight.dim() != 2:
        raise ValueError("weight must be [d, width]")
    _fits(x, weight)
    _expect(weight, "weight", (d, weight.shape[1]), torch.float32, device, True)
    _optional(bias, "bias", (d,), torch.float32, device)
    _optional(lengths, "lengths", (B,), torch.int32, device)
    return hla_conv_params(B, x.shape[1] if x.dim() == 3 else 1, d, weight.shape[1], code, _activation(activation),
                           _ptr(weight), _ptr(bias), _ptr(lengths))


def conv_forward(x, weight, bias=None, activation: str = "none", state_in=None, return_state: bool = False,
                 lengths=None, out=None, stream=None):
    """Short causal convolution per channel: y_t = act(bias + sum_i weight[:, i] x_{t-(w-1)+i}) over
    x [B,n,d] (bf16 or fp32, any strides with adjacent channels), weight [d,w] fp32 with w of 2 to
    4, bias [d] fp32 or None, activation "none" or "silu".  state_in [B,w-1,d] (x's type): the
    inputs before the first token, or None (zeros).  lengths [B] int32: tokens of each sequence
    (rows behind them: zero in a new y, left as they were in ``out``).  Returns y (and the last
    w - 1 inputs of each sequence)."""
    import torch
    dev = _current(x)
    if x.dim() != 3:
        raise ValueError("x must be [B, n, d]")
    p = _conv_params(x, weight, bias, activation, lengths, dev)
    held = (p.B, p.width - 1, p.d)
    _optional(state_in, "state_in", held, x.dtype, dev)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        st = torch.empty(held, dtype=x.dtype, device=dev) if return_state else None
        hla_conv_forward(p, _t2(x), _t2(out), state_in, st, stream)
    return (out, st) if return_state else out


def conv_workspace(x, weight, stream=None):
    """A workspace for conv_backward of these shapes: partial sums of the filters' gradients.
    Calls that may overlap in time need one each."""
    import torch
    p = _conv_params(x, weight, None, "none", None, x.device)
    with _on(stream, x.device):
        return torch.empty(max(hla_conv_backward_workspace_size(p), 1), dtype=torch.uint8, device=x.device)


def conv_backward(x, dy, weight, bias=None, activation: str = "none", state_in=None, d_state_out=None,
                  want_dstate: bool = False, lengths=None, out=None, workspace=None, stream=None):
    """Gradients of conv_forward from dy and d_state_out [B,w-1,d] (None: zero).  Returns
    ConvGradients(dx, d_weight, d_bias, d_state_in): d_weight [d,w] and d_bias [d] fp32 (None
    without a bias), d_state_in with want_dstate (else None).  ``out`` may hold dx."""
    import torch
    dev = _current(x)
    if x.dim() != 3:
        raise ValueError("x must be [B, n, d]")
    p = _conv_params(x, weight, bias, activation, lengths, dev)
    held = (p.B, p.width - 1, p.d)
    _expect(dy, "dy", x.shape, x.dtype, dev)
    _optional(state_in, "state_in", held, x.dtype, dev)
    _optional(d_state_out, "d_state_out", held, x.dtype, dev)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "dx", x.shape, x.dtype, dev)
        dw = torch.empty((p.d, p.width), dtype=torch.float32, device=dev)
        db = torch.empty((p.d,), dtype=torch.float32, device=dev) if bias is not None else None
        ds = torch.empty(held, dtype=x.dtype, device=dev) if want_dstate else None
        ws, nbytes = _space(hla_conv_backward_workspace_size(p) if workspace is None else 0, workspace, dev, False)
        hla_conv_backward(p, _t2(x), _t2(dy), _t2(out), state_in, d_state_out, dw, db, ds, ws, nbytes, stream)
    return ConvGradients(out, dw, db, ds)


def conv_step(state, x, weight, bias=None, activation: str = "none", lengths=None, out=None, stream=None):
    """One token of every sequence: x [B,d], state [B,w-1,d] shifted by one in place.  lengths [B]
    int32: 0 marks an idle sequence, whose rows of y (zero in a new one) and of the state are left
    as they were.  Returns y [B,d]."""
    import torch
    dev = _current(x)
    if x.dim() != 2:
        raise ValueError("x must be [B, d]")
    p = _conv_params(x, weight, bias, activation, lengths, dev)
    _expect(state, "state", (p.B, p.width - 1, p.d), x.dtype, dev, True)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        hla_conv_step(p, _t2(x), _t2(out), state, stream)
    return out


def _t_steps(t):
    """dt [B, H] or [B, H, n]: single elements, so any strides."""
    s = t.stride()
    return hla_tensor(t.data_ptr(), s[0], s[1], s[2] if len(s) == 3 else 0)


def _like(x, zero):
    """A new tensor of x's shape with tokens outside heads where x has them so."""
    import torch
    make = torch.zeros if zero else torch.empty
    if x.stride(1) < x.stride(2):
        shape = (x.shape[0], x.shape[2], x.shape[1]) + x.shape[3:]
        return make(shape, dtype=x.dtype, device=x.device).transpose(1, 2)
    return make(x.shape, dtype=x.dtype, device=x.device)


def _expect_steps(t, name, shape, dtype, device):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ssm_params(x, dt, A, B, C, D, dt_bias, dt_softplus, lengths, device):
    import torch
    code = _dtype_code(x)
    tail = x.shape[2:-1]  # (n,), or nothing for a step
    batch, H, P = x.shape[0], x.shape[1], x.shape[-1]
    if B.dim() != x.dim():
        raise ValueError("B and C must be [B, G, n, N] (a step's [B, G, N])")
    _fits(x, B)
    G, N = B.shape[1], B.shape[-1]
    _expect(x, "x", x.shape, x.dtype, device)
    _expect_steps(dt, "dt", (batch, H) + tail, x.dtype, device)
    _expect(B, "B", (batch, G) + tail + (N,), x.dtype, device)
    _expect(C, "C", (batch, G) + tail + (N,), x.dtype, device)
    _expect(A, "A", (H,), torch.float32, device, True)
    _optional(D, "D", (H,), torch.float32, device)
    _optional(dt_bias, "dt_bias", (H,), torch.float32, device)
    _optional(lengths, "lengths", (batch,), torch.int32, device)
    return hla_ssm_params(batch, H, G, tail[0] if tail else 1, P, N, code, 1 if dt_softplus else 0, _ptr(A), _ptr(D),
                          _ptr(dt_bias), _ptr(lengths))


def ssm_workspace(x, B, backward: bool = False, stream=None):
    """A workspace for ssm_forward (or ssm_backward) of x [B,H,n,P] and B [B,G,n,N], whatever their
    strides: the states between chunks of tokens (forward: less than x's own bytes where prompts are
    long); no initial contents.  Calls that may overlap in time need one each."""
    import torch
    _fits(x, B)
    p = hla_ssm_params(x.shape[0], x.shape[1], B.shape[1], x.shape[2], x.shape[3], B.shape[3], _dtype_code(x), 0, None,
                       None, None, None)
    with _on(stream, x.device):
        return torch.empty(max(hla_ssm_workspace_size(p, backward), 1), dtype=torch.uint8, device=x.device)


def ssm_forward(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus: bool = False, state_in=None,
                return_state: bool = False, lengths=None, out=None, workspace=None, stream=None):
    """Selective state space scan over x [B,H,n,P], dt [B,H,n], B, C [B,G,n,N] (bf16 or fp32, any
    strides with adjacent channels, widths up to 128; head h reads group h // (H // G)):
    h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t^T, y_t = C_t h_t + D x_t per head, with A [H] and D [H]
    (or None) fp32 and dt as given, or softplus(dt + dt_bias) with dt_softplus (dt_bias [H] fp32 or
    None).  state_in [B,H,N,P] fp32 or None (zeros); lengths [B] int32: tokens of each sequence
    (rows behind them: zero in a new y, left as they were in ``out``).  A new y lies in memory as
    x does (tokens outside heads, or heads outside tokens).  Rows below the lengths must be finite.  bf16 on
    16-byte rows takes weights and states rounded to bf16 on the way to y (never in the state).
    Returns y (and the final state)."""
    import torch
    dev = _current(x)
    if x.dim() != 4:
        raise ValueError("x must be [B, H, n, P]")
    p = _ssm_params(x, dt, A, B, C, D, dt_bias, dt_softplus, lengths, dev)
    held = (p.B, p.H, p.N, p.P)
    _optional(state_in, "state_in", held, torch.float32, dev)
    with _on(stream, dev):
        if out is None:
            out = _like(x, lengths is not None)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        st = torch.empty(held, dtype=torch.float32, device=dev) if return_state else None
        ws, nbytes = _space(hla_ssm_workspace_size(p, False) if workspace is None else 0, workspace, dev, False)
        hla_ssm_forward(p, _t4(x), _t_steps(dt), _t4(B), _t4(C), _t4(out), state_in, st, ws, nbytes, stream)
    return (out, st) if return_state else out


def ssm_backward(x, dt, A, B, C, dy, D=None, dt_bias=None, dt_softplus: bool = False, state_in=None,
                 d_state_out=None, want_dstate: bool = False, lengths=None, out=None, workspace=None, stream=None):
    """Gradients of ssm_forward from dy and d_state_out [B,H,N,P] fp32 (None: zero).  Returns
    SsmGradients(dx, d_dt, dA, dB, dC, dD, d_dt_bias, d_state_in): dA, dD, d_dt_bias [H] fp32 (the
    latter two None without D, dt_bias), d_state_in fp32 with want_dstate (else None).  ``out`` may
    hold four tensors for dx, d_dt, dB and dC."""
    import torch
    dev = _current(x)
    if x.dim() != 4:
        raise ValueError("x must be [B, H, n, P]")
    p = _ssm_params(x, dt, A, B, C, D, dt_bias, dt_softplus, lengths, dev)
    held = (p.B, p.H, p.N, p.P)
    _expect(dy, "dy", x.shape, x.dtype, dev)
    _optional(state_in, "state_in", held, torch.float32, dev)
    _optional(d_state_out, "d_state_out", held, torch.float32, dev)
    with _on(stream, dev):
        new = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)  # noqa: E731
        dx, ddt, dB, dC = out if out is not None else tuple(_like(t, lengths is not None) for t in (x, dt, B, C))
        for t, name, like in ((dx, "dx", x), (dB, "dB", B), (dC, "dC", C)):
            _expect(t, name, like.shape, x.dtype, dev)
        _expect_steps(ddt, "d_dt", dt.shape, x.dtype, dev)
        dA = new(p.H)
        dD = new(p.H) if D is not None else None
        db = new(p.H) if dt_bias is not None else None
        ds = new(*held) if want_dstate else None
        ws, nbytes = _space(hla_ssm_workspace_size(p, True) if workspace is None else 0, workspace, dev, False)
        g = hla_ssm_gradients(_t4(dx), _t_steps(ddt), _t4(dB), _t4(dC), _ptr(dA), _ptr(dD), _ptr(db), _ptr(ds))
        hla_ssm_backward(p, _t4(x), _t_steps(dt), _t4(B), _t4(C), _t4(dy), state_in, d_state_out, g, ws, nbytes, stream)
    return SsmGradients(dx, ddt, dA, dB, dC, dD, db, ds)


def ssm_step(state, x, dt, A, B, C, D=None, dt_bias=None, dt_softplus: bool = False, lengths=None, out=None,
             stream=None):
    """One token of every sequence: x [B,H,P], dt [B,H], B, C [B,G,N]; state [B,H,N,P] fp32 is
    updated in place.  lengths [B] int32: 0 marks an idle sequence, whose rows of y (zero in a new
    one) and state are left as they were.  Returns y [B,H,P]."""
    import torch
    dev = _current(x)
    if x.dim() != 3:
        raise ValueError("x must be [B, H, P]")
    p = _ssm_params(x, dt, A, B, C, D, dt_bias, dt_softplus, lengths, dev)
    _expect(state, "state", (p.B, p.H, p.N, p.P), torch.float32, dev, True)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        hla_ssm_step(p, _t4(x), _t_steps(dt), _t4(B), _t4(C), _t4(out), state, stream)
    return out


def _norm_params(x, weight, bias, groups, eps, center, gate, gate_first, activation, lengths, device):
    import torch
    code = _dtype_code(x)
    if x.dim() != 3:
        raise ValueError("x must be [B, n, d]")
    _fits(x)
    B, n, d = x.shape
    _expect(x, "x", x.shape, x.dtype, device)
    if gate is not None:
        _expect(gate, "gate", x.shape, x.dtype, device)
    _optional(weight, "weight", (d,), torch.float32, device)
    _optional(bias, "bias", (d,), torch.float32, device)
    _optional(lengths, "lengths", (B,), torch.int32, device)
    return hla_norm_params(B, n, d, _int32(groups, "groups"), code, 1 if center else 0, _activation(activation),
                           1 if gate_first else 0, float(eps), _ptr(weight), _ptr(bias), _ptr(lengths))


def norm_forward(x, weight=None, bias=None, groups: int = 1, eps: float = 1e-5, center: bool = True, gate=None,
                 gate_first: bool = False, activation: str = "none", lengths=None, out=None, stream=None):
    """Norm over groups of d / groups adjacent channels of each token of x [B,n,d] (bf16 or fp32,
    any strides with adjacent channels): u = x, or x silu(gate) with gate_first; z = (u - mean) /
    sqrt(var + eps), with center=False u / sqrt(mean(u^2) + eps); v = z weight + bias (fp32 [d] or
    None).  y = v silu(gate) with a gate [B,n,d] that is not first, silu(v) with activation "silu"
    and no gate, else v.  A gate needs activation "silu".  lengths [B] int32: rows behind them are
    zero in a new y, left as they were in ``out``.  Returns y."""
    import torch
    dev = _current(x)
    p = _norm_params(x, weight, bias, groups, eps, center, gate, gate_first, activation, lengths, dev)
    with _on(stream, dev):
        if out is None:
            out = (torch.zeros if lengths is not None else torch.empty)(x.shape, dtype=x.dtype, device=dev)
        else:
            _expect(out, "out", x.shape, x.dtype, dev)
        hla_norm_forward(p, _t2(x), None if gate is None else _t2(gate), _t2(out), stream)
    return out


def norm_workspace(x, stream=None):
    """A workspace for norm_backward of x [B,n,d], whatever its groups: partial sums for the scale's
    and the shift's gradients.  Calls that may overlap in time need one each."""
    import torch
    _fits(x)
    p = hla_norm_params(*x.shape, 1, _dtype_code(x), 0, 0, 0, 0.0, None, None, None)
    with _on(stream, x.device):
        return torch.empty(max(hla_norm_backward_workspace_size(p), 1), dtype=torch.uint8, device=x.device)


def norm_backward(x, dy, weight=None, bias=None, groups: int = 1, eps: float = 1e-5, center: bool = True, gate=None,
                  gate_first: bool = False, activation: str = "none", lengths=None, out=None, workspace=None,
                  stream=None):
    """Gradients of norm_forward from x, gate and dy.  Returns NormGradients(dx, d_gate, d_weight,
    d_bias): d_weight and d_bias [d] fp32 (None without weight, bias), d_gate None without a gate.
    ``out`` may hold dx, or dx and d_gate with a gate."""
    import torch
    dev = _current(x)
    p = _norm_params(x, weight, bias, groups, eps, center, gate, gate_first, activation, lengths, dev)
    _expect(dy, "dy", x.shape, x.dtype, dev)
    with _on(stream, dev):
        if out is None:
            make = torch.zeros if lengths is not None else torch.empty
            out = tuple(make(x.shape, dtype=x.dtype, device=dev) for _ in range(1 if gate is None else 2))
        elif gate is None:
            out = (out,) if torch.is_tensor(out) else tuple(out)
        dx, dg = out[0], out[1] if gate is not None else None
        for t, name in ((dx, "dx"), (dg, "d_gate")):
            if t is not None:
                _expect(t, name, x.shape, x.dtype, dev)
        dw = torch.empty((p.d,), dtype=torch.float32, device=dev) if weight is not None else None
        db = torch.empty((p.d,), dtype=torch.float32, device=dev) if bias is not None else None
        ws, nbytes = _space(hla_norm_backward_workspace_size(p) if workspace is None else 0, workspace, dev, False)
        hla_norm_backward(p, _t2(x), None if gate is None else _t2(gate), _t2(dy), _t2(dx),
                          None if dg is None else _t2(dg), dw, db, ws, nbytes, stream)
    return NormGradients(dx, dg, dw, db)

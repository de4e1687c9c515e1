"""ctypes binding of liblinattn.so (C ABI: include/linattn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C entry points.  Tensors must be contiguous CUDA tensors
(``norm_rotate`` and its gradients take strided ones);
outputs and workspaces are allocated here with torch (the library allocates
nothing).  There is no CPU fallback: a missing or unbuildable library raises.

Names follow the C ABI:

* ``forward_causal``    -> ``la_forward_causal``
* ``forward_noncausal`` -> ``la_forward_noncausal``
* ``decode_step``       -> ``la_decode_step``
* ``forward_causal_gated``, ``decode_step_gated``, ``forward_noncausal_phi``,
  ``random_features`` -> the gated and feature-map entry points
* ``forward_delta``, ``backward_delta``, ``decode_step_delta`` -> the gated delta rule
* ``layer_norm``, ``layer_norm_backward`` -> the norm that follows it
* ``forward_retention``, ``backward_retention``, ``decode_step_retention`` -> retention: a decay for
  each head, no feature map, no denominator
* ``norm_rotate``, ``norm_rotate_backward`` -> queries and keys normed and rotated by position
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from . import _build

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA, LA_ERR_TIMEOUT, LA_ERR_WORKSPACE = range(6)
LA_DTYPE_F32, LA_DTYPE_BF16 = 0, 1
PHI = {"elu1": 0, "identity": 1}   # la_phi
LAYOUT = {"bhnd": 0, "bnhd": 1}    # la_layout
NORM = {None: 0, "rms": 1, "l2": 2}       # la_norm
PAIRS = {"halves": 0, "adjacent": 1}      # la_pairs

_lock = threading.Lock()
_lib = None


class LinAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def library_path() -> str:
    return _build.LIB


def lib():
    """Load (building first if the sources are newer) and return the ctypes library."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if _build.is_stale():
                _build.build()
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"liblinattn.so missing at {_build.LIB}")
            L = ctypes.CDLL(_build.LIB)
            vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            L.la_status_string.argtypes = [i]
            L.la_status_string.restype = ctypes.c_char_p
            L.la_version.argtypes = []
            L.la_version.restype = ctypes.c_char_p
            L.la_causal_workspace_bytes.argtypes = [i, i, i, i, i, i]
            L.la_causal_workspace_bytes.restype = sz
            L.la_noncausal_workspace_bytes.argtypes = [i, i, i, i, i, i]
            L.la_noncausal_workspace_bytes.restype = sz
            L.la_forward_causal.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, vp, vp, vp,
                                            vp, sz, vp]
            L.la_forward_causal.restype = i
            L.la_forward_noncausal.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, vp, vp,
                                               sz, vp]
            L.la_forward_noncausal.restype = i
            L.la_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
            L.la_decode_step.restype = i
            L.la_causal_host_buffer_bytes.argtypes = [i, i, i, i, i, i]
            L.la_causal_host_buffer_bytes.restype = sz
            L.la_forward_causal_host.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, vp, vp,
                                                 sz, vp]
            L.la_forward_causal_host.restype = i
            L.la_forward_causal_decay.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp, vp, vp,
                                                  vp, vp, vp, sz, vp]
            L.la_forward_causal_decay.restype = i
            L.la_decode_step_decay.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, vp]
            L.la_decode_step_decay.restype = i
            L.la_causal_backward_workspace_bytes.argtypes = [i, i, i, i, i, i]
            L.la_causal_backward_workspace_bytes.restype = sz
            L.la_backward_causal.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f,
                                             vp, vp, vp, vp, vp, sz, vp]
            L.la_backward_causal.restype = i
            L.la_backward_causal_decay.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                                   f, vp, vp, vp, vp, vp, vp, sz, vp]
            L.la_backward_causal_decay.restype = i
            L.la_workspace_status.argtypes = [vp, sz, vp]
            L.la_workspace_status.restype = i
            L.la_debug_set_fault.argtypes = [i, ctypes.c_longlong]
            L.la_debug_set_fault.restype = None
            L.la_debug_set_stall.argtypes = [ctypes.c_longlong]
            L.la_debug_set_stall.restype = None
            L.la_debug_feature_bf16.argtypes = [vp, vp, ctypes.c_longlong, f, vp]
            L.la_debug_feature_bf16.restype = i
            L.la_forward_noncausal_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, vp,
                                                       vp, vp]
            L.la_forward_noncausal_noalloc.restype = i
            L.la_noalloc_status.argtypes = [vp]
            L.la_noalloc_status.restype = i
            L.la_forward_causal_gated.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, i,
                                                  vp, vp, vp, vp, vp, sz, vp]
            L.la_forward_causal_gated.restype = i
            L.la_causal_gated_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
            L.la_causal_gated_workspace_bytes.restype = sz
            L.la_decode_step_gated.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i,
                                               vp]
            L.la_decode_step_gated.restype = i
            L.la_noncausal_phi_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.la_noncausal_phi_workspace_bytes.restype = sz
            L.la_forward_noncausal_phi.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp,
                                                   vp, sz, vp]
            L.la_forward_noncausal_phi.restype = i
            L.la_random_features.argtypes = [vp, vp, ctypes.c_longlong, i, i, i, vp, vp]
            L.la_random_features.restype = i
            L.la_delta_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.la_delta_workspace_bytes.restype = sz
            L.la_forward_delta.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, vp,
                                           vp, sz, vp]
            L.la_forward_delta.restype = i
            L.la_delta_backward_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.la_delta_backward_workspace_bytes.restype = sz
            L.la_backward_delta.argtypes = [vp] * 11 + [i] * 8 + [vp, vp, vp, vp, sz, vp]
            L.la_backward_delta.restype = i
            L.la_decode_step_delta.argtypes = [vp] * 8 + [i] * 6 + [vp]
            L.la_decode_step_delta.restype = i
            L.la_layer_norm.argtypes = [vp] * 6 + [ctypes.c_longlong, i, i, f, vp]
            L.la_layer_norm.restype = i
            L.la_layer_norm_backward_workspace_bytes.argtypes = [ctypes.c_longlong, i, i]
            L.la_layer_norm_backward_workspace_bytes.restype = sz
            L.la_layer_norm_backward.argtypes = [vp] * 8 + [ctypes.c_longlong, i, i, vp, sz, vp]
            L.la_layer_norm_backward.restype = i
            ll = ctypes.c_longlong
            rotate = [i] * 8 + [f, vp, vp, vp, i, i, vp, ll]   # B .. norm, eps, weights, freq .. positions_stride
            L.la_norm_rotate.argtypes = [vp] * 5 + rotate + [vp]
            L.la_norm_rotate.restype = i
            L.la_norm_rotate_backward_workspace_bytes.argtypes = [i] * 6
            L.la_norm_rotate_backward_workspace_bytes.restype = sz
            L.la_norm_rotate_backward.argtypes = [vp] * 7 + rotate + [vp, vp, vp, sz, vp]
            L.la_norm_rotate_backward.restype = i
            L.la_retention_workspace_bytes.argtypes = [i] * 6
            L.la_retention_workspace_bytes.restype = sz
            L.la_forward_retention.argtypes = [vp] * 5 + [i] * 7 + [vp, vp, vp, sz, vp]
            L.la_forward_retention.restype = i
            L.la_retention_backward_workspace_bytes.argtypes = [i] * 6
            L.la_retention_backward_workspace_bytes.restype = sz
            L.la_backward_retention.argtypes = [vp] * 8 + [i] * 7 + [vp, vp, vp, vp, sz, vp]
            L.la_backward_retention.restype = i
            L.la_decode_step_retention.argtypes = [vp] * 7 + [i] * 5 + [vp]
            L.la_decode_step_retention.restype = i
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().la_status_string(int(status)).decode()


def version() -> str:
    return lib().la_version().decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LA_DTYPE_BF16
    if t.dtype == torch.float32:
        return LA_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors (no CPU fallback)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _raise(st: int, where: str):
    if st != LA_OK:
        raise LinAttnError(st, where)


def causal_workspace_bytes(B, H, N, d, dv, dtype=torch.bfloat16) -> int:
    code = LA_DTYPE_BF16 if dtype == torch.bfloat16 else LA_DTYPE_F32
    return int(lib().la_causal_workspace_bytes(B, H, N, d, dv, code))


def noncausal_workspace_bytes(B, H, N, d, dv, dtype=torch.bfloat16) -> int:
    code = LA_DTYPE_BF16 if dtype == torch.bfloat16 else LA_DTYPE_F32
    return int(lib().la_noncausal_workspace_bytes(B, H, N, d, dv, code))


def alloc_workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    # torch's caching allocator returns blocks aligned to at least 512 bytes
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def forward_causal(q, k, v, eps: float = 1e-6, S_in=None, z_in=None, return_state=False,
                   out=None, S_out=None, z_out=None, workspace=None, stream=None,
                   check_status=False):
    """Causal elu+1 linear attention.  q, k: [B,H,N,d]; v: [B,H,N,dv] (bf16 or fp32).

    Returns y [B,H,N,dv] float32 (and the final (S, z) when ``return_state``).
    With ``check_status`` the call synchronises and raises if a kernel recorded
    a run-time error (a bounded wait that ran out) in the workspace.
    """
    _check_cuda(q, k, v, S_in, z_in, out, S_out, z_out, workspace)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes / dtypes disagree")
    y = out if out is not None else torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    if return_state and S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=q.device)
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    need = int(lib().la_causal_workspace_bytes(B, H, N, d, dv, dt))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().la_forward_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(y), B, H, N, d, dv, dt,
                                 float(eps), _ptr(S_in), _ptr(z_in), _ptr(S_out), _ptr(z_out),
                                 _ptr(workspace), wbytes, _stream_handle(stream, q.device))
    _raise(st, "la_forward_causal")
    if check_status and need and workspace is not None:   # without need nothing is recorded there
        err, where = workspace_header(workspace)
        if err != LA_OK:
            raise LinAttnError(err, f"la_forward_causal (run time, wait site {where})")
    return (y, S_out, z_out) if return_state else y


def forward_causal_decay(q, k, v, gamma, eps: float = 1e-6, S_in=None, z_in=None,
                         return_state=False, out=None, S_out=None, z_out=None, workspace=None,
                         stream=None, check_status=False):
    """Causal attention with a per-head decay ``gamma`` (float32 CUDA tensor [H]).

    q, k: [B,H,N,d]; v: [B,H,N,dv].  Returns y [B,H,N,dv] float32 (and the
    final (S, z) when ``return_state``).  The workspace and ``check_status``
    are as in ``forward_causal``.
    """
    _check_cuda(q, k, v, gamma, S_in, z_in, out, S_out, z_out, workspace)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes / dtypes disagree")
    if gamma.shape != (H,) or gamma.dtype != torch.float32:
        raise ValueError("gamma must be a float32 tensor of shape [H]")
    y = out if out is not None else torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    if return_state and S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=q.device)
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    need = int(lib().la_causal_workspace_bytes(B, H, N, d, dv, dt))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().la_forward_causal_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(y), B, H, N, d, dv, dt,
                                       float(eps), _ptr(gamma), _ptr(S_in), _ptr(z_in),
                                       _ptr(S_out), _ptr(z_out), _ptr(workspace), wbytes,
                                       _stream_handle(stream, q.device))
    _raise(st, "la_forward_causal_decay")
    if check_status and need and workspace is not None:   # without need nothing is recorded there
        err, where = workspace_header(workspace)
        if err != LA_OK:
            raise LinAttnError(err, f"la_forward_causal_decay (run time, wait site {where})")
    return (y, S_out, z_out) if return_state else y


def decode_step_decay(q, k, v, S, z, gamma, eps: float = 1e-6, out=None, stream=None):
    """One decode step with decay; S and z are updated in place.  Returns y."""
    _check_cuda(q, k, v, S, z, gamma, out)
    B, H, d = q.shape
    dv = v.shape[-1]
    if gamma.shape != (H,) or gamma.dtype != torch.float32:
        raise ValueError("gamma must be a float32 tensor of shape [H]")
    y = out if out is not None else torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    st = lib().la_decode_step_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(y), _ptr(S), _ptr(z), B, H,
                                    d, dv, _dtype_code(q), float(eps), _ptr(gamma),
                                    _stream_handle(stream, q.device))
    _raise(st, "la_decode_step_decay")
    return y


def causal_backward_workspace_bytes(B, H, N, d, dv, dtype=torch.bfloat16) -> int:
    code = LA_DTYPE_BF16 if dtype == torch.bfloat16 else LA_DTYPE_F32
    return int(lib().la_causal_backward_workspace_bytes(B, H, N, d, dv, code))


def backward_causal(q, k, v, dy, eps: float = 1e-6, S_in=None, z_in=None,
                    return_state_grad=False, out=None, workspace=None, stream=None, gamma=None):
    """Gradients of the causal forward for the upstream gradient ``dy``.

    q, k: [B,H,N,d]; v: [B,H,N,dv] (bf16 or fp32); dy: [B,H,N,dv] float32.
    With ``gamma`` (float32 CUDA tensor [H]) the gradients are those of the
    decayed forward (``forward_causal_decay``).
    Returns (dq, dk, dv) float32, plus (dS_in, dz_in) when ``return_state_grad``.
    ``out`` may be a preallocated (dq, dk, dv) triple.
    """
    _check_cuda(q, k, v, dy, S_in, z_in, workspace, gamma)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes / dtypes disagree")
    if dy.shape != v.shape or dy.dtype != torch.float32:
        raise ValueError("dy must be float32 with the shape of v")
    if out is None:
        out = (torch.empty((B, H, N, d), dtype=torch.float32, device=q.device),
               torch.empty((B, H, N, d), dtype=torch.float32, device=q.device),
               torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device))
    gq, gk, gv = out
    _check_cuda(gq, gk, gv)
    gS = gz = None
    if return_state_grad:
        gS = torch.empty((B, H, d, dv), dtype=torch.float32, device=q.device)
        gz = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    need = int(lib().la_causal_backward_workspace_bytes(B, H, N, d, dv, dt))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if gamma is None:
        st = lib().la_backward_causal(_ptr(q), _ptr(k), _ptr(v), _ptr(dy), _ptr(gq), _ptr(gk),
                                      _ptr(gv), B, H, N, d, dv, dt, float(eps), _ptr(S_in),
                                      _ptr(z_in), _ptr(gS), _ptr(gz), _ptr(workspace), wbytes,
                                      _stream_handle(stream, q.device))
        _raise(st, "la_backward_causal")
    else:
        if gamma.shape != (H,) or gamma.dtype != torch.float32:
            raise ValueError("gamma must be a float32 tensor of shape [H]")
        st = lib().la_backward_causal_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(dy), _ptr(gq),
                                            _ptr(gk), _ptr(gv), B, H, N, d, dv, dt, float(eps),
                                            _ptr(gamma), _ptr(S_in), _ptr(z_in), _ptr(gS),
                                            _ptr(gz), _ptr(workspace), wbytes,
                                            _stream_handle(stream, q.device))
        _raise(st, "la_backward_causal_decay")
    return (gq, gk, gv, gS, gz) if return_state_grad else (gq, gk, gv)


def causal_host_buffer_bytes(B, H, N, d, dv, dtype=torch.bfloat16) -> int:
    code = LA_DTYPE_BF16 if dtype == torch.bfloat16 else LA_DTYPE_F32
    return int(lib().la_causal_host_buffer_bytes(B, H, N, d, dv, code))


def forward_causal_host(q, k, v, eps: float = 1e-6, return_state=False, out=None, S_out=None,
                        z_out=None, dev_buf=None, device=None, stream=None):
    """Causal forward on host (CPU) tensors through la_forward_causal_host.

    q, k: [B,H,N,d]; v: [B,H,N,dv] CPU tensors (bf16 or fp32; page-locked
    memory makes the copies overlap).  Returns y [B,H,N,dv] float32 on the CPU
    (and the final (S, z) when ``return_state``).  ``dev_buf`` is the device
    staging memory (allocated on ``device`` when not given).
    """
    for t in (q, k, v, out, S_out, z_out):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("forward_causal_host takes contiguous CPU tensors")
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes / dtypes disagree")
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    y = out if out is not None else torch.empty((B, H, N, dv), dtype=torch.float32)
    if return_state and S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32)
        z_out = torch.empty((B, H, d), dtype=torch.float32)
    if dev_buf is None:
        dev_buf = alloc_workspace(int(lib().la_causal_host_buffer_bytes(B, H, N, d, dv, dt)), dev)
    nbytes = 0 if dev_buf is None else dev_buf.numel() * dev_buf.element_size()
    st = lib().la_forward_causal_host(_ptr(q), _ptr(k), _ptr(v), _ptr(y), B, H, N, d, dv, dt,
                                      float(eps), _ptr(S_out), _ptr(z_out), _ptr(dev_buf), nbytes,
                                      _stream_handle(stream, dev))
    _raise(st, "la_forward_causal_host")
    return (y, S_out, z_out) if return_state else y


def forward_noncausal(q, k, v, eps: float = 1e-6, return_state=False, out=None, S_out=None,
                      z_out=None, workspace=None, stream=None, check_status=False):
    """Non-causal elu+1 linear attention.  Returns y [B,H,N,dv] float32 (+ S, z).

    ``check_status`` as for :func:`forward_causal`.
    """
    _check_cuda(q, k, v, out, S_out, z_out, workspace)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes / dtypes disagree")
    y = out if out is not None else torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    if return_state and S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=q.device)
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    need = int(lib().la_noncausal_workspace_bytes(B, H, N, d, dv, dt))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().la_forward_noncausal(_ptr(q), _ptr(k), _ptr(v), _ptr(y), B, H, N, d, dv, dt,
                                    float(eps), _ptr(S_out), _ptr(z_out), _ptr(workspace), wbytes,
                                    _stream_handle(stream, q.device))
    _raise(st, "la_forward_noncausal")
    if check_status and workspace is not None:
        err, where = workspace_header(workspace)
        if err != LA_OK:
            raise LinAttnError(err, f"la_forward_noncausal (run time, wait site {where})")
    return (y, S_out, z_out) if return_state else y


def decode_step(q, k, v, S, z, eps: float = 1e-6, out=None, stream=None):
    """One decode step in place on (S, z).  q, k: [B,H,d]; v: [B,H,dv]; returns y [B,H,dv] fp32."""
    _check_cuda(q, k, v, S, z, out)
    B, H, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if S.dtype != torch.float32 or z.dtype != torch.float32:
        raise TypeError("state must be float32")
    if S.shape != (B, H, d, dv) or z.shape != (B, H, d):
        raise ValueError("state shape mismatch")
    y = out if out is not None else torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    st = lib().la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(y), _ptr(S), _ptr(z), B, H, d, dv,
                              dt, float(eps), _stream_handle(stream, q.device))
    _raise(st, "la_decode_step")
    return y


def workspace_status(workspace, stream=None) -> int:
    """Synchronise and return the run-time status recorded in ``workspace``."""
    if workspace is None:
        return LA_OK
    return int(lib().la_workspace_status(_ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream_handle(stream, workspace.device)))


def workspace_header(workspace) -> tuple[int, int]:
    """(error word, diagnostic word) recorded in a workspace header (synchronises)."""
    torch.cuda.synchronize(workspace.device)
    h = workspace[:8].cpu().view(torch.int32)
    return int(h[0]), int(h[1])


def set_fault(drop_load_item: int = -1, wait_limit_ns: int = 0) -> None:
    """Test hook: see la_debug_set_fault in include/linattn.h."""
    lib().la_debug_set_fault(int(drop_load_item), int(wait_limit_ns))


def set_stall(ns: int = 0) -> None:
    """Test hook: see la_debug_set_stall in include/linattn.h."""
    lib().la_debug_set_stall(int(ns))


def _gate_dim(gate, lead, d):
    """gate_dim of a gate tensor whose leading shape is ``lead`` (1 or d)."""
    if gate is None:
        return 1
    if gate.dtype != torch.float32:
        raise TypeError("gate must be float32")
    if tuple(gate.shape) == tuple(lead):
        return 1
    if tuple(gate.shape) == tuple(lead) + (d,):
        return d
    raise ValueError(f"gate shape {tuple(gate.shape)} must be {tuple(lead)} or {tuple(lead) + (d,)}")


def causal_gated_workspace_bytes(B, H, N, d, dv, dtype=torch.bfloat16, phi="elu1",
                                 gate_dim=1) -> int:
    code = LA_DTYPE_BF16 if dtype == torch.bfloat16 else LA_DTYPE_F32
    return int(lib().la_causal_gated_workspace_bytes(B, H, N, d, dv, code, PHI[phi], gate_dim))


def forward_causal_gated(q, k, v, gate=None, phi="elu1", eps: float = 1e-6, S_in=None,
                         z_in=None, return_state=False, out=None, S_out=None, z_out=None,
                         workspace=None, stream=None, check_status=False):
    """Gated causal attention.  gate: None, [B,H,N] or [B,H,N,d] float32; phi:
    "elu1" or "identity".  bf16 inputs with d, dv in {64, 128}, one gate per
    token and elu + 1 run on the tensor cores (heads whose gates all lie in
    [2^-1/2, 1]); everything else in fp32 on the CUDA cores.  Returns y (and the
    final (S, z)); ``check_status`` as for :func:`forward_causal`."""
    _check_cuda(q, k, v, gate, S_in, z_in, out, S_out, z_out, workspace)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes / dtypes disagree")
    gd = _gate_dim(gate, (B, H, N), d)
    y = out if out is not None else torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    if return_state and S_out is None:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=q.device)
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    need = (causal_gated_workspace_bytes(B, H, N, d, dv, q.dtype, phi, gd) if gate is not None
            else 256)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    st = lib().la_forward_causal_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(y), B, H, N, d, dv, dt,
                                       float(eps), PHI[phi], _ptr(gate), gd, _ptr(S_in),
                                       _ptr(z_in), _ptr(S_out), _ptr(z_out), _ptr(workspace),
                                       workspace.numel() if workspace is not None else 0,
                                       _stream_handle(stream, q.device))
    _raise(st, "la_forward_causal_gated")
    if check_status and workspace is not None:
        err, where = workspace_header(workspace)
        if err != LA_OK:
            raise LinAttnError(err, f"la_forward_causal_gated (run time, wait site {where})")
    return (y, S_out, z_out) if return_state else y


def decode_step_gated(q, k, v, S, z, gate=None, phi="elu1", eps: float = 1e-6, out=None,
                      stream=None):
    """One gated decode step in place on (S, z); gate None, [B,H] or [B,H,d]."""
    _check_cuda(q, k, v, S, z, gate, out)
    B, H, d = q.shape
    dv = v.shape[-1]
    gd = _gate_dim(gate, (B, H), d)
    y = out if out is not None else torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    st = lib().la_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(y), _ptr(S), _ptr(z), B, H,
                                    d, dv, _dtype_code(q), float(eps), PHI[phi], _ptr(gate), gd,
                                    _stream_handle(stream, q.device))
    _raise(st, "la_decode_step_gated")
    return y


def forward_noncausal_phi(q, k, v, phi="identity", eps: float = 1e-6, return_state=False,
                          out=None, workspace=None, stream=None):
    """Non-causal attention with the feature map ``phi`` ("elu1" or "identity")."""
    _check_cuda(q, k, v, out, workspace)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    y = out if out is not None else torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    S_out = z_out = None
    if return_state:
        S_out = torch.empty((B, H, d, dv), dtype=torch.float32, device=q.device)
        z_out = torch.empty((B, H, d), dtype=torch.float32, device=q.device)
    need = int(lib().la_noncausal_phi_workspace_bytes(B, H, N, d, dv, dt, PHI[phi]))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().la_forward_noncausal_phi(_ptr(q), _ptr(k), _ptr(v), _ptr(y), B, H, N, d, dv, dt,
                                        float(eps), PHI[phi], _ptr(S_out), _ptr(z_out),
                                        _ptr(workspace), wbytes, _stream_handle(stream, q.device))
    _raise(st, "la_forward_noncausal_phi")
    return (y, S_out, z_out) if return_state else y


def random_features(x, W, out=None, stream=None):
    """exp(W x - ||x||^2 / 2) / sqrt(m) for every row of x ([..., d], bf16 or fp32);
    W: float32 [m, d] CUDA tensor.  Returns float32 [..., m]."""
    _check_cuda(x, W, out)
    d = x.shape[-1]
    if W.dtype != torch.float32 or W.dim() != 2 or W.shape[1] != d:
        raise ValueError("W must be float32 [m, d]")
    m = W.shape[0]
    rows = x.numel() // d
    y = out if out is not None else torch.empty(tuple(x.shape[:-1]) + (m,), dtype=torch.float32,
                                                device=x.device)
    st = lib().la_random_features(_ptr(x), _ptr(y), rows, d, m, _dtype_code(x), _ptr(W),
                                  _stream_handle(stream, x.device))
    _raise(st, "la_random_features")
    return y


# ---- gated delta rule, layer norm -------------------------------------------
# Small calls cost mostly this module's own time, so the calls below read each property once, and take
# the device's index and the stream's handle without the objects around them where torch offers that.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device_index: torch.cuda.current_stream(device_index).cuda_stream)


def _elsewhere(fn, stream, t, *args, **kw):
    """``fn`` with ``t``'s device and, if given, ``stream`` current, so that what it allocates belongs
    to the device and stream that use it."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors (no CPU fallback)")
    if stream is not None and stream.device != t.device:
        raise ValueError("the stream is of another device than the tensors")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        return fn(t, *args, **kw)


def _addr(t):
    return None if t is None else t.data_ptr()


def _expect(name, t, shape, dtype, device_index):
    """Address of ``t``, which is None or a contiguous tensor of this shape and dtype on this device."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, not {t.dtype} of {tuple(t.shape)}")
    if t.get_device() != device_index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device_index}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _workspace(workspace, need, like):
    """(tensor, address, bytes) of the workspace; one is allocated when none is given."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the tensors' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=1024)
def _delta_bytes(device_index, *sizes):   # the split depends on the current device
    return int(lib().la_delta_workspace_bytes(*sizes))


@functools.lru_cache(maxsize=1024)
def _delta_backward_bytes(device_index, *sizes):
    return int(lib().la_delta_backward_workspace_bytes(*sizes))


def _check_run_time(workspace, need, where):
    if need:   # a call that needs no workspace records nothing in one it is given
        err, site = workspace_header(workspace)
        if err != LA_OK:
            raise LinAttnError(err, f"{where} (run time, wait site {site})")


def _delta_inputs(q, k, v, beta, log_gate, layout):
    """Checks the inputs of a delta-rule call: its sizes (B, H, Hk, N, d, dv, dtype code), the
    device's index and the inputs' addresses."""
    if layout not in LAYOUT:
        raise ValueError(f"layout must be one of {sorted(LAYOUT)}")
    shape, vs = q.shape, v.shape
    if len(shape) != 4 or len(vs) != 4:
        raise ValueError("q, k and v must have four dimensions")
    if layout == "bhnd":
        B, Hk, N, d = shape
        H, dv = vs[1], vs[3]
        vshape = (B, H, N, dv)
    else:
        B, N, Hk, d = shape
        H, dv = vs[2], vs[3]
        vshape = (B, N, H, dv)
    dev, dt = q.get_device(), q.dtype
    at = (_expect("q", q, shape, dt, dev), _expect("k", k, shape, dt, dev), _expect("v", v, vshape, dt, dev),
          _expect("beta", beta, vshape[:3], torch.float32, dev),
          _expect("log_gate", log_gate, vshape[:3], torch.float32, dev))
    return (B, H, Hk, N, d, dv, _dtype_code(q)), dev, at


def forward_delta(q, k, v, beta, log_gate=None, S_in=None, return_state=False, out=None,
                  S_out=None, layout="bhnd", workspace=None, check_status=False, stream=None):
    """The gated delta rule, causal:
    S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T, y_t = S_t^T q_t, a_t = exp(log_gate_t).

    q, k: [B,Hk,N,d]; v: [B,H,N,dv], H a multiple of Hk (bf16 or fp32); beta, log_gate: float32
    [B,H,N] (log_gate None: no gate); with ``layout="bnhd"`` heads and tokens swap places in all of
    them.  Returns y in v's shape and dtype (and the final state [B,H,d,dv], float32, when
    ``return_state``).  S_in: the initial state; S_out may be S_in.
    """
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(forward_delta, stream, q, k, v, beta, log_gate, S_in, return_state, out, S_out, layout,
                          workspace, check_status)
    sizes, dev, (qa, ka, va, ba, la) = _delta_inputs(q, k, v, beta, log_gate, layout)
    B, H, Hk, N, d, dv, dt = sizes
    state = (B, H, d, dv)
    if out is None:
        out = torch.empty_like(v)
    if return_state and S_out is None:
        S_out = torch.empty(state, dtype=torch.float32, device=q.device)
    need = _delta_bytes(dev, *sizes)
    workspace, wa, wbytes = _workspace(workspace, need, q)
    st = lib().la_forward_delta(qa, ka, va, _expect("out", out, v.shape, v.dtype, dev), ba, la, B, H, Hk,
                                N, d, dv, dt, LAYOUT[layout],
                                _expect("S_in", S_in, state, torch.float32, dev),
                                _expect("S_out", S_out, state, torch.float32, dev), wa, wbytes,
                                _current_stream(dev))
    _raise(st, "la_forward_delta")
    if check_status:
        _check_run_time(workspace, need, "la_forward_delta")
    return (out, S_out) if return_state else out


def backward_delta(q, k, v, beta, dy, log_gate=None, S_in=None, grad_S_out=None, layout="bhnd",
                   workspace=None, check_status=False, stream=None):
    """Gradients of ``forward_delta`` for dy = dL/dy (dtype and shape of v) and grad_S_out = dL/dS
    of the final state (None: zero).  Returns (grad_q, grad_k, grad_v, grad_beta, grad_log_gate,
    grad_S_in): the first three in the inputs' dtype, the others float32; grad_log_gate is None
    without log_gate, grad_S_in is None unless S_in or grad_S_out is given.
    """
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(backward_delta, stream, q, k, v, beta, dy, log_gate, S_in, grad_S_out, layout, workspace,
                          check_status)
    sizes, dev, (qa, ka, va, ba, la) = _delta_inputs(q, k, v, beta, log_gate, layout)
    B, H, Hk, N, d, dv, dt = sizes
    state = (B, H, d, dv)
    gq, gk, gv, gb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(beta)
    gl = None if log_gate is None else torch.empty_like(log_gate)
    gS = None
    if S_in is not None or grad_S_out is not None:
        gS = torch.empty(state, dtype=torch.float32, device=q.device)
    need = _delta_backward_bytes(dev, *sizes)
    workspace, wa, wbytes = _workspace(workspace, need, q)
    st = lib().la_backward_delta(qa, ka, va, _expect("dy", dy, v.shape, v.dtype, dev), ba, la, gq.data_ptr(),
                                 gk.data_ptr(), gv.data_ptr(), gb.data_ptr(), _addr(gl), B, H, Hk, N, d, dv,
                                 dt, LAYOUT[layout], _expect("S_in", S_in, state, torch.float32, dev),
                                 _expect("grad_S_out", grad_S_out, state, torch.float32, dev), _addr(gS),
                                 wa, wbytes, _current_stream(dev))
    _raise(st, "la_backward_delta")
    if check_status:
        _check_run_time(workspace, need, "la_backward_delta")
    return gq, gk, gv, gb, gl, gS


def decode_step_delta(q, k, v, beta, S, log_gate=None, S_out=None, out=None, stream=None):
    """One token of ``forward_delta``: q, k [B,Hk,d]; v [B,H,dv]; beta, log_gate [B,H] float32;
    S [B,H,d,dv] float32, updated in place unless ``S_out`` is given.  Returns y [B,H,dv] in v's dtype.
    """
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(decode_step_delta, stream, q, k, v, beta, S, log_gate, S_out, out)
    shape, vs = q.shape, v.shape
    if len(shape) != 3 or len(vs) != 3:
        raise ValueError("q, k and v must have three dimensions")
    B, Hk, d = shape
    H, dv = vs[1], vs[2]
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    if out is None:
        out = torch.empty_like(v)
    sa = _expect("S", S, (B, H, d, dv), f32, dev)
    st = lib().la_decode_step_delta(_expect("q", q, shape, dt, dev), _expect("k", k, shape, dt, dev),
                                    _expect("v", v, (B, H, dv), dt, dev), _expect("out", out, vs, dt, dev),
                                    _expect("beta", beta, (B, H), f32, dev),
                                    _expect("log_gate", log_gate, (B, H), f32, dev), sa,
                                    sa if S_out is None else _expect("S_out", S_out, (B, H, d, dv), f32, dev),
                                    B, H, Hk, d, dv, _dtype_code(q), _current_stream(dev))
    _raise(st, "la_decode_step_delta")
    return out


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, return_stats=False, out=None, stream=None):
    """(x - mean) * rstd * weight + bias over the last dimension (at most 16384 values, bf16 or
    fp32); weight, bias: float32 [D] or None.  Returns y in x's dtype (and mean, rstd, float32 in
    x's shape without its last dimension, when ``return_stats``).  ``out`` may be x."""
    if stream is not None or not x.is_cuda or x.get_device() != _current_device():
        return _elsewhere(layer_norm, stream, x, weight, bias, eps, return_stats, out)
    shape, dev, f32 = x.shape, x.get_device(), torch.float32
    if not shape:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    if out is None:
        out = torch.empty_like(x)
    mean = rstd = None
    if return_stats:
        mean = x.new_empty(shape[:-1], dtype=f32)
        rstd = torch.empty_like(mean)
    st = lib().la_layer_norm(_expect("x", x, shape, x.dtype, dev), _expect("out", out, shape, x.dtype, dev),
                             _expect("weight", weight, (D,), f32, dev), _expect("bias", bias, (D,), f32, dev),
                             _addr(mean), _addr(rstd), x.numel() // D if D else 0, D, _dtype_code(x),
                             eps, _current_stream(dev))
    _raise(st, "la_layer_norm")
    return (out, mean, rstd) if return_stats else out


@functools.lru_cache(maxsize=1024)
def _norm_backward_bytes(device_index, rows, D, dt):   # as many sums as the device has CTAs
    return int(lib().la_layer_norm_backward_workspace_bytes(rows, D, dt))


def layer_norm_backward(dy, x, mean, rstd, weight=None, sums=None, workspace=None, stream=None):
    """Gradients of ``layer_norm`` from its mean and rstd: (grad_x, grad_weight, grad_bias), the
    first in x's dtype, the sums float32 [D].  ``sums`` says whether to compute the latter two
    (default: when weight is given); they are None otherwise."""
    if stream is not None or not dy.is_cuda or dy.get_device() != _current_device():
        return _elsewhere(layer_norm_backward, stream, dy, x, mean, rstd, weight, sums, workspace)
    shape, dev, f32 = x.shape, x.get_device(), torch.float32
    if not shape:
        raise ValueError("x must have at least one dimension")
    D, dt = shape[-1], _dtype_code(x)
    gx = torch.empty_like(x)
    rows = x.numel() // D if D else 0
    gw = gb = wa = None
    wbytes = 0
    if weight is not None if sums is None else sums:
        gw = x.new_empty(D, dtype=f32)
        gb = torch.empty_like(gw)
        workspace, wa, wbytes = _workspace(workspace, _norm_backward_bytes(dev, rows, D, dt), x)
    st = lib().la_layer_norm_backward(_expect("dy", dy, shape, x.dtype, dev), _expect("x", x, shape, x.dtype, dev),
                                      _expect("mean", mean, shape[:-1], f32, dev),
                                      _expect("rstd", rstd, shape[:-1], f32, dev),
                                      _expect("weight", weight, (D,), f32, dev), gx.data_ptr(), _addr(gw),
                                      _addr(gb), rows, D, dt, wa, wbytes, _current_stream(dev))
    _raise(st, "la_layer_norm_backward")
    return gx, gw, gb


# ---- norm and rotation of queries and keys ------------------------------------
# What follows from shapes and types alone is worked out once for each combination of them.
def _dense(name, t, dtype, device_index):
    """Address of ``t``, which is None or a contiguous tensor of this dtype on this device; its shape is known."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != device_index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device_index}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _shape(t):
    return None if t is None else t.shape


def _code_of(dtype):
    if dtype is torch.bfloat16:
        return LA_DTYPE_BF16
    if dtype is torch.float32:
        return LA_DTYPE_F32
    raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")


@functools.lru_cache(maxsize=1024)
def _rotate_plan(qs, ks, dtype, strides, freq, positions, norm, wq, wk, pairs, layout):
    """From the shapes, and the strides of tensors of q's shape and of k's in turn (None: contiguous, in the shape's order):
    (B, Hq, Hk, N, d, dtype code, layout, norm), rotated, pairs, the positions' stride from one sequence to the
    next, the strides of batch, head and token for the C call."""
    if layout not in LAYOUT or norm not in NORM or pairs not in PAIRS:
        raise ValueError(f"layout must be one of {sorted(LAYOUT)}, norm of {list(NORM)}, pairs of {sorted(PAIRS)}")
    if len(qs) not in (3, 4) or len(ks) != len(qs):
        raise ValueError("q and k must have four dimensions, or three for single tokens")
    h, t = (1, None) if len(qs) == 3 else (1, 2) if layout == "bhnd" else (2, 1)
    B, d, N = qs[0], qs[-1], 1 if t is None else qs[t]
    if ks[0] != B or ks[-1] != d or (t is not None and ks[t] != N):
        raise ValueError("q and k must differ in their number of heads only")
    rotated = 0
    if freq is not None:
        if len(freq) != 1:
            raise ValueError("freq must be of one dimension")
        rotated = freq[0]
    for name, w in (("q_weight", wq), ("k_weight", wk)):
        if w is not None and tuple(w) != (d,):
            raise ValueError(f"{name} must be of shape {(d,)}, not {tuple(w)}")
    step = 0
    if positions is not None:
        own = (B,) if t is None else (B, N)
        if tuple(positions) == own:
            step = 1 if t is None else N
        elif t is None or tuple(positions) != (N,):
            raise ValueError(f"positions must be of shape {own}" + ("" if t is None else f" or {(N,)}"))
    elif t is None and rotated:
        raise ValueError("single tokens need positions")
    flat = []
    for i, st in enumerate(strides):
        shape = ks if i % 2 else qs
        if st is not None and len(st) != len(shape):
            raise ValueError("all tensors must have as many dimensions as q")
        if st is None:
            st = [1] * len(shape)
            for x in reversed(range(len(shape) - 1)):
                st[x] = st[x + 1] * shape[x + 1]
        elif st[-1] != 1 and d > 1:
            raise ValueError("the last dimension must be contiguous")
        flat += st[0], st[h], 0 if t is None else st[t]
    return ((B, qs[h], ks[h], N, d, _code_of(dtype), LAYOUT[layout], NORM[norm]), rotated, PAIRS[pairs], step,
            (ctypes.c_longlong * len(flat))(*flat))


def _rows(name, t, like, device_index):
    """Address of ``t``, of ``like``'s shape and dtype."""
    if t.shape != like.shape or t.dtype is not like.dtype:
        raise ValueError(f"{name} must be {like.dtype} of shape {tuple(like.shape)}, not {t.dtype} of {tuple(t.shape)}")
    if t.get_device() != device_index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device_index}")
    return t.data_ptr()


_contiguous = torch.contiguous_format


def norm_rotate(q, k, freq=None, positions=None, norm="rms", q_weight=None, k_weight=None, eps: float = 1e-6,
                pairs="halves", layout="bhnd", out=None, stream=None):
    """Queries and keys normed over each head's d values, weighted and rotated by position, in one pass.

    q: [B,Hq,N,d], k: [B,Hk,N,d] (``layout="bnhd"``: [B,N,H,d]; single tokens: [B,H,d]), bf16 or fp32; the last
    dimension contiguous, any strides else, so that both may be parts of one projection's output.  norm: "rms"
    (x / sqrt(mean(x^2) + eps)), "l2" (unit length, x / sqrt(sum(x^2) + eps)) or None; weights: float32 [d] or None.
    freq: float64 [r], radians a position of the first 2 r values' pairs (e, e + r) ("halves") or
    (2 e, 2 e + 1) ("adjacent"); None: no rotation.  positions: int64 [B,N] or [N] ([B] for single tokens);
    None: 0, 1, ... .  Returns (q', k') in the inputs' shape and dtype; ``out`` may be (q, k).
    """
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(norm_rotate, stream, q, k, freq, positions, norm, q_weight, k_weight, eps, pairs, layout, out)
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    if k.dtype is not dt:
        raise ValueError("q and k must have the same dtype")
    strides = (q.stride(), k.stride(), *((None, None) if out is None else (t.stride() for t in out)))
    sizes, rotated, pair_code, step, st = _rotate_plan(q.shape, k.shape, dt, strides, _shape(freq), _shape(positions),
                                                       norm, _shape(q_weight), _shape(k_weight), pairs, layout)
    ka = _rows("k", k, k, dev)
    if out is None:
        yq, yk = torch.empty_like(q, memory_format=_contiguous), torch.empty_like(k, memory_format=_contiguous)
        at = yq.data_ptr(), yk.data_ptr()
    else:
        yq, yk = out
        at = _rows("out[0]", yq, q, dev), _rows("out[1]", yk, k, dev)
    status = lib().la_norm_rotate(q.data_ptr(), ka, *at, st, *sizes, eps, _dense("q_weight", q_weight, f32, dev),
                                  _dense("k_weight", k_weight, f32, dev), _dense("freq", freq, torch.float64, dev),
                                  rotated, pair_code, _dense("positions", positions, torch.int64, dev), step,
                                  _current_stream(dev))
    if status:
        _raise(status, "la_norm_rotate")
    return yq, yk


@functools.lru_cache(maxsize=1024)
def _rotate_backward_bytes(device_index, *sizes):   # as many sums as the device has CTAs
    return int(lib().la_norm_rotate_backward_workspace_bytes(*sizes))


def norm_rotate_backward(grad_q_out, grad_k_out, q, k, freq=None, positions=None, norm="rms", q_weight=None,
                         k_weight=None, eps: float = 1e-6, pairs="halves", layout="bhnd", sums=None, out=None,
                         workspace=None, stream=None):
    """Gradients of ``norm_rotate`` for those of its outputs (their shape and dtype, strides as q and k):
    (grad_q, grad_k, grad_q_weight, grad_k_weight), the first two in q's dtype, the sums float32 [d].
    ``sums`` says whether to compute those (default: each where its weight is given); they are None otherwise.
    ``out``: where grad_q and grad_k go; they may be q and k, or the outputs' gradients."""
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(_norm_rotate_backward_of_q, stream, q, k, grad_q_out, grad_k_out, freq, positions, norm,
                          q_weight, k_weight, eps, pairs, layout, sums, out, workspace)
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    if k.dtype is not dt:
        raise ValueError("q and k must have the same dtype")
    strides = (q.stride(), k.stride(), grad_q_out.stride(), grad_k_out.stride(),
               *((None, None) if out is None else (t.stride() for t in out)))
    sizes, rotated, pair_code, step, st = _rotate_plan(q.shape, k.shape, dt, strides, _shape(freq), _shape(positions),
                                                       norm, _shape(q_weight), _shape(k_weight), pairs, layout)
    at = [q.data_ptr(), _rows("k", k, k, dev), _rows("grad_q_out", grad_q_out, q, dev),
          _rows("grad_k_out", grad_k_out, k, dev)]
    if out is None:
        yq, yk = torch.empty_like(q, memory_format=_contiguous), torch.empty_like(k, memory_format=_contiguous)
        at += yq.data_ptr(), yk.data_ptr()
    else:
        yq, yk = out
        at += _rows("out[0]", yq, q, dev), _rows("out[1]", yk, k, dev)
    d = sizes[4]
    gwq = torch.empty(d, dtype=f32, device=q.device) if (q_weight is not None if sums is None else sums) else None
    gwk = torch.empty(d, dtype=f32, device=q.device) if (k_weight is not None if sums is None else sums) else None
    wa, wbytes = None, 0
    if gwq is not None or gwk is not None:
        workspace, wa, wbytes = _workspace(workspace, _rotate_backward_bytes(dev, *sizes[:6]), q)
    status = lib().la_norm_rotate_backward(*at, st, *sizes, eps,
                                           _dense("q_weight", q_weight, f32, dev),
                                           _dense("k_weight", k_weight, f32, dev),
                                           _dense("freq", freq, torch.float64, dev), rotated, pair_code,
                                           _dense("positions", positions, torch.int64, dev), step, _addr(gwq),
                                           _addr(gwk), wa, wbytes, _current_stream(dev))
    if status:
        _raise(status, "la_norm_rotate_backward")
    return yq, yk, gwq, gwk


def _norm_rotate_backward_of_q(q, k, grad_q_out, grad_k_out, *args):
    return norm_rotate_backward(grad_q_out, grad_k_out, q, k, *args)


# ---- retention -----------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def _retention_bytes(device_index, *sizes):   # the split depends on the current device
    return int(lib().la_retention_workspace_bytes(*sizes))


@functools.lru_cache(maxsize=1024)
def _retention_backward_bytes(device_index, *sizes):
    return int(lib().la_retention_backward_workspace_bytes(*sizes))


@functools.lru_cache(maxsize=1024)
def _retention_plan(qs, ks, vs, gs, dtype, layout):
    """From the shapes: (B, H, N, d, dv, dtype code), the layout's code, the state's shape."""
    if layout not in LAYOUT:
        raise ValueError(f"layout must be one of {sorted(LAYOUT)}")
    if len(qs) != 4 or len(vs) != 4:
        raise ValueError("q, k and v must have four dimensions")
    B, H, N, d = qs if layout == "bhnd" else (qs[0], qs[2], qs[1], qs[3])
    if tuple(ks) != tuple(qs) or tuple(vs[:3]) != tuple(qs[:3]):
        raise ValueError(f"k must be of q's shape {tuple(qs)} and v of shape {(*qs[:3], 'dv')}, not {tuple(ks)} and {tuple(vs)}")
    if tuple(gs) != (H,):
        raise ValueError(f"gamma must be of shape {(H,)}, not {tuple(gs)}")
    return (B, H, N, d, vs[3], _code_of(dtype)), LAYOUT[layout], (B, H, d, vs[3])


def forward_retention(q, k, v, gamma, S_in=None, return_state=False, out=None, S_out=None, layout="bhnd",
                      workspace=None, check_status=False, stream=None):
    """Retention, causal: S_t = gamma_h S_{t-1} + k_t v_t^T, y_t = S_t^T q_t.

    q, k: [B,H,N,d]; v: [B,H,N,dv] (bf16 or fp32; ``layout="bnhd"``: [B,N,H,...]); gamma: float32 [H],
    in [0, 1].  Returns y in v's shape and dtype (and the final state [B,H,d,dv], float32, when
    ``return_state``).  S_in: the initial state; S_out may be S_in.  Unlike ``forward_causal_decay`` there is
    no feature map and no denominator.
    """
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(forward_retention, stream, q, k, v, gamma, S_in, return_state, out, S_out, layout, workspace,
                          check_status)
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    sizes, code, state = _retention_plan(q.shape, k.shape, v.shape, gamma.shape, dt, layout)
    at = (_dense("q", q, dt, dev), _dense("k", k, dt, dev), _dense("v", v, dt, dev))
    if out is None:
        out = torch.empty_like(v)
        ya = out.data_ptr()
    else:
        ya = _expect("out", out, v.shape, dt, dev)
    if return_state and S_out is None:
        S_out = torch.empty(state, dtype=torch.float32, device=q.device)
    need = _retention_bytes(dev, *sizes)
    workspace, wa, wbytes = _workspace(workspace, need, q)
    st = lib().la_forward_retention(*at, ya, _dense("gamma", gamma, f32, dev), *sizes, code,
                                    _expect("S_in", S_in, state, f32, dev), _expect("S_out", S_out, state, f32, dev),
                                    wa, wbytes, _current_stream(dev))
    if st:
        _raise(st, "la_forward_retention")
    if check_status:
        _check_run_time(workspace, need, "la_forward_retention")
    return (out, S_out) if return_state else out


def backward_retention(q, k, v, gamma, dy, S_in=None, grad_S_out=None, layout="bhnd", workspace=None,
                       check_status=False, stream=None):
    """Gradients of ``forward_retention`` for dy = dL/dy (dtype and shape of v) and grad_S_out = dL/dS of the final
    state (None: zero): (grad_q, grad_k, grad_v, grad_S_in), the first three in the inputs' dtype, the last
    float32, None unless S_in or grad_S_out is given."""
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(backward_retention, stream, q, k, v, gamma, dy, S_in, grad_S_out, layout, workspace,
                          check_status)
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    sizes, code, state = _retention_plan(q.shape, k.shape, v.shape, gamma.shape, dt, layout)
    at = (_dense("q", q, dt, dev), _dense("k", k, dt, dev), _dense("v", v, dt, dev))
    gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    gS = None
    if S_in is not None or grad_S_out is not None:
        gS = torch.empty(state, dtype=torch.float32, device=q.device)
    need = _retention_backward_bytes(dev, *sizes)
    workspace, wa, wbytes = _workspace(workspace, need, q)
    st = lib().la_backward_retention(*at, _expect("dy", dy, v.shape, dt, dev), _dense("gamma", gamma, f32, dev),
                                     gq.data_ptr(), gk.data_ptr(), gv.data_ptr(), *sizes, code,
                                     _expect("S_in", S_in, state, f32, dev),
                                     _expect("grad_S_out", grad_S_out, state, f32, dev), _addr(gS), wa, wbytes,
                                     _current_stream(dev))
    if st:
        _raise(st, "la_backward_retention")
    if check_status:
        _check_run_time(workspace, need, "la_backward_retention")
    return gq, gk, gv, gS


@functools.lru_cache(maxsize=1024)
def _retention_step_plan(qs, ks, vs, gs, dtype):
    """From the shapes: (B, H, d, dv, dtype code), the state's shape."""
    if len(qs) != 3 or len(vs) != 3:
        raise ValueError("q, k and v must have three dimensions")
    B, H, d = qs
    if tuple(ks) != tuple(qs) or tuple(vs[:2]) != (B, H) or tuple(gs) != (H,):
        raise ValueError("q and k must be [B, H, d], v [B, H, dv] and gamma [H]")
    return (B, H, d, vs[2], _code_of(dtype)), (B, H, d, vs[2])


def decode_step_retention(q, k, v, gamma, S, S_out=None, out=None, stream=None):
    """One token of ``forward_retention``: q, k [B,H,d]; v [B,H,dv]; gamma [H] float32; S [B,H,d,dv] float32,
    updated in place unless ``S_out`` is given.  Returns y [B,H,dv] in v's dtype."""
    if stream is not None or not q.is_cuda or q.get_device() != _current_device():
        return _elsewhere(decode_step_retention, stream, q, k, v, gamma, S, S_out, out)
    dev, dt, f32 = q.get_device(), q.dtype, torch.float32
    sizes, state = _retention_step_plan(q.shape, k.shape, v.shape, gamma.shape, dt)
    at = (_dense("q", q, dt, dev), _dense("k", k, dt, dev), _dense("v", v, dt, dev))
    if out is None:
        out = torch.empty_like(v)
        ya = out.data_ptr()
    else:
        ya = _expect("out", out, v.shape, dt, dev)
    sa = _expect("S", S, state, f32, dev)
    st = lib().la_decode_step_retention(*at, ya, _dense("gamma", gamma, f32, dev), sa,
                                        sa if S_out is None else _expect("S_out", S_out, state, f32, dev), *sizes,
                                        _current_stream(dev))
    if st:
        _raise(st, "la_decode_step_retention")
    return out

"""Python binding of liblinattn.so (kernelized linear attention, phi = elu + 1).

Argument marshalling only: every function here checks shapes and dtypes,
passes raw device pointers and the current CUDA stream to the C ABI declared
in include/linattn.h, and raises on a non-OK status. All arithmetic runs in
the library's CUDA kernels; there is no other code path. PyTorch supplies
device memory and streams.

Importing the package loads the library and fails loudly if it has not been
built (``python linear_attention_elu_gb300/build.py``).
"""
import contextlib
import ctypes
import os

import torch

from . import build as _build

__all__ = [
    "LA_F32", "LA_BF16", "LA_OP_NONCAUSAL", "LA_OP_CAUSAL", "LA_OP_DECODE", "LinAttnError",
    "la_status_string", "la_version", "la_workspace_size", "la_launch_count", "la_workspace_init",
    "la_noncausal_fwd", "la_causal_fwd", "la_decode_step", "la_query_status", "workspace",
    "la_host_staging_size", "host_staging", "la_causal_fwd_host", "la_causal_fwd_state",
    "la_causal_bwd", "LA_OP_CAUSAL_BWD", "la_noncausal_bwd", "LA_OP_NONCAUSAL_BWD",
    "LA_PHI_ELU1", "LA_PHI_IDENTITY", "la_positive_random_features", "LA_OP_LAYER_DECODE",
    "la_layer_decode_step", "la_causal_fwd_noalloc", "la_noalloc_query_status",
    "la_noalloc_set_wait_limit", "library_path", "LA_ROPE_MAX_AXES", "la_rope_table",
    "la_qk_norm_rope_fwd", "la_qk_norm_rope_bwd", "la_qk_norm_rope_bwd_workspace_size",
    "qk_norm_rope_workspace", "la_short_conv_fwd", "la_short_conv_step",
    "LA_OP_SELECTIVE_SCAN", "la_selective_scan_fwd", "la_selective_scan_step",
    "LA_OP_DECAY_ATTN", "LA_OP_DECAY_ATTN_BWD", "la_decay_attn_fwd", "la_decay_attn_bwd",
    "la_decay_attn_step", "la_group_norm_fwd", "la_group_norm_bwd", "la_group_norm_workspace_size",
    "group_norm_workspace",
]

LA_F32, LA_BF16 = 0, 1
LA_OP_NONCAUSAL, LA_OP_CAUSAL, LA_OP_DECODE, LA_OP_CAUSAL_BWD, LA_OP_NONCAUSAL_BWD = 0, 1, 2, 3, 4
LA_OP_LAYER_DECODE, LA_OP_SELECTIVE_SCAN = 5, 6
LA_OP_DECAY_ATTN, LA_OP_DECAY_ATTN_BWD = 8, 9
LA_PHI_ELU1, LA_PHI_IDENTITY = 0, 1
LA_ROPE_HALVES, LA_ROPE_INTERLEAVED, LA_ROPE_MAX_AXES = 0, 1, 4
LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_WORKSPACE, LA_ERR_CUDA, LA_ERR_TIMEOUT = 0, 1, 2, 3, 4, 5

_DTYPES = {torch.float32: LA_F32, torch.bfloat16: LA_BF16}


class LinAttnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {la_status_string(status)}")


def library_path():
    return _build.LIB


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(
            f"liblinattn.so is not built ({path}); run `python linear_attention_elu_gb300/build.py`"
            " or __graft_entry__.build(). There is no fallback implementation.")
    lib = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.la_status_string.argtypes = [I]
    lib.la_status_string.restype = ctypes.c_char_p
    lib.la_version.argtypes = []
    lib.la_version.restype = ctypes.c_uint32
    lib.la_workspace_size.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(Z)]
    lib.la_workspace_size.restype = I
    lib.la_launch_count.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(I)]
    lib.la_launch_count.restype = I
    lib.la_workspace_init.argtypes = [P, Z, P]
    lib.la_workspace_init.restype = I
    lib.la_noncausal_fwd.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, Z, P]
    lib.la_noncausal_fwd.restype = I
    lib.la_causal_fwd.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P, Z, P]
    lib.la_causal_fwd.restype = I
    lib.la_causal_bwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, Z, P]
    lib.la_causal_bwd.restype = I
    lib.la_noncausal_bwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, Z, P]
    lib.la_noncausal_bwd.restype = I
    lib.la_causal_fwd_state.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, P, Z, P]
    lib.la_causal_fwd_state.restype = I
    lib.la_host_staging_size.argtypes = [I, I, I, I, I, I, ctypes.POINTER(Z)]
    lib.la_host_staging_size.restype = I
    lib.la_causal_fwd_host.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P, Z, P, Z, P]
    lib.la_causal_fwd_host.restype = I
    lib.la_decode_step.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P]
    lib.la_decode_step.restype = I
    L = ctypes.c_int64
    lib.la_noncausal_fwd_phi.argtypes = [P, P, P, P, I, I, I, I, I, I, I, F, P, Z, P]
    lib.la_noncausal_fwd_phi.restype = I
    lib.la_causal_fwd_phi.argtypes = [P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P, P, Z, P]
    lib.la_causal_fwd_phi.restype = I
    lib.la_decode_step_phi.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, P]
    lib.la_decode_step_phi.restype = I
    lib.la_causal_bwd_phi.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, Z, P]
    lib.la_causal_bwd_phi.restype = I
    lib.la_noncausal_bwd_phi.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, Z, P]
    lib.la_noncausal_bwd_phi.restype = I
    lib.la_positive_random_features.argtypes = [P, P, P, L, I, I, I, F, P]
    lib.la_positive_random_features.restype = I
    lib.la_causal_fwd_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P]
    lib.la_causal_fwd_noalloc.restype = I
    lib.la_noalloc_query_status.argtypes = [P]
    lib.la_noalloc_query_status.restype = I
    lib.la_noalloc_set_wait_limit.argtypes = [ctypes.c_uint, I, P]
    lib.la_noalloc_set_wait_limit.restype = I
    lib.la_layer_decode_step.argtypes = [P, P, P, P, P, P, I, I, I, I, F, P, Z, P]
    lib.la_layer_decode_step.restype = I
    lib.la_rope_table.argtypes = [P, P, I, I, P]
    lib.la_rope_table.restype = I
    lib.la_qk_norm_rope_fwd.argtypes = [P, L, L, P, L, L, P, P, P, I, P, I, P, P, I, I, I, I, I, I,
                                        I, F, I, P]
    lib.la_qk_norm_rope_fwd.restype = I
    lib.la_qk_norm_rope_bwd_workspace_size.argtypes = [I, I, I, I, I, ctypes.POINTER(Z)]
    lib.la_qk_norm_rope_bwd_workspace_size.restype = I
    lib.la_qk_norm_rope_bwd.argtypes = [P, L, L, P, L, L, P, P, P, I, P, I, P, P, P, L, L, P, L, L,
                                        P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
    lib.la_qk_norm_rope_bwd.restype = I
    lib.la_short_conv_fwd.argtypes = [P, L, L, P, P, I, P, P, P, P, L, L, I, I, I, I, I, P]
    lib.la_short_conv_fwd.restype = I
    lib.la_short_conv_step.argtypes = [P, L, P, P, I, P, P, L, I, I, I, I, P]
    lib.la_short_conv_step.restype = I
    lib.la_selective_scan_fwd.argtypes = [P, L, L, P, L, L, P, P, L, L, P, L, L, P, P, L, L, P, I, P,
                                          P, P, P, L, L, I, I, I, I, I, I, I, P, Z, P]
    lib.la_selective_scan_fwd.restype = I
    lib.la_selective_scan_step.argtypes = [P, L, P, L, P, P, L, P, L, P, P, L, P, I, P, P, L, I, I, I,
                                           I, I, I, P]
    lib.la_selective_scan_step.restype = I
    lib.la_decay_attn_fwd.argtypes = [P, P, P, P, F, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]
    lib.la_decay_attn_fwd.restype = I
    lib.la_decay_attn_bwd.argtypes = [P, P, P, P, P, F, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]
    lib.la_decay_attn_bwd.restype = I
    lib.la_decay_attn_step.argtypes = [P, P, P, P, F, P, P, P, I, I, I, I, I, P]
    lib.la_decay_attn_step.restype = I
    lib.la_group_norm_workspace_size.argtypes = [I, I, I, I, ctypes.POINTER(Z)]
    lib.la_group_norm_workspace_size.restype = I
    lib.la_group_norm_fwd.argtypes = [P, L, L, P, P, P, L, L, P, L, L, P, I, I, I, I, I, I, F, P, Z, P]
    lib.la_group_norm_fwd.restype = I
    lib.la_group_norm_bwd.argtypes = [P, L, L, P, P, P, L, L, P, L, L, P, P, L, L, P, L, L, P, P, I, I, I, I, I,
                                      I, P, Z, P]
    lib.la_group_norm_bwd.restype = I
    lib.la_query_status.argtypes = [P, P]
    lib.la_query_status.restype = I
    return lib


_lib = _load()


def _check(status, where):
    if status != LA_OK:
        raise LinAttnError(status, where)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _dt(t):
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")
    return _DTYPES[t.dtype]


def _need_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous ([B, H, N, D], D innermost)")


def la_status_string(status):
    return _lib.la_status_string(int(status)).decode()


def la_version():
    return int(_lib.la_version())


def la_workspace_size(op, B, H, N, Dk, Dv, dtype):
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    n = ctypes.c_size_t(0)
    _check(_lib.la_workspace_size(int(op), B, H, N, Dk, Dv, dt, ctypes.byref(n)),
           "la_workspace_size")
    return int(n.value)


def la_launch_count(op, B, H, N, Dk, Dv, dtype):
    """Kernel launches one call of `op` makes at this shape (host-only query)."""
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    n = ctypes.c_int(0)
    _check(_lib.la_launch_count(int(op), B, H, N, Dk, Dv, dt, ctypes.byref(n)), "la_launch_count")
    return int(n.value)


def la_workspace_init(ws, stream=None):
    _need_cuda(ws)
    _check(_lib.la_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "la_workspace_init")
    return ws


def workspace(op, B, H, N, Dk, Dv, dtype, device=None, stream=None):
    """Allocates (through PyTorch) and initialises a workspace for `op` at this shape."""
    n = la_workspace_size(op, B, H, N, Dk, Dv, dtype)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")
    return la_workspace_init(ws, stream)


def _shape4(q, k, v):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError(f"expected q, k [B,H,N,Dk] and v [B,H,N,Dv]; got {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)}")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    B, H, N, Dk = q.shape
    return B, H, N, Dk, v.shape[3]


def la_noncausal_fwd(q, k, v, o=None, eps=1e-6, ws=None, stream=None, phi=LA_PHI_ELU1):
    """o_i = phi(q_i)^T S / (phi(q_i)^T z + eps), S = sum_j phi(k_j) v_j^T, z = sum_j phi(k_j).

    `phi`: LA_PHI_ELU1 (elu + 1) or LA_PHI_IDENTITY (q, k are features already)."""
    B, H, N, Dk, Dv = _shape4(q, k, v)
    if o is None:
        o = torch.empty_like(v)
    _need_cuda(q, k, v, o, ws)
    if ws is None:
        ws = workspace(LA_OP_NONCAUSAL, B, H, N, Dk, Dv, q.dtype, q.device, stream)
    if phi == LA_PHI_ELU1:
        _check(_lib.la_noncausal_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv, _dt(q),
                                     float(eps), _ptr(ws), ws.numel(), _stream(stream)),
               "la_noncausal_fwd")
    else:
        _check(_lib.la_noncausal_fwd_phi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv,
                                         _dt(q), int(phi), float(eps), _ptr(ws), ws.numel(),
                                         _stream(stream)),
               "la_noncausal_fwd_phi")
    return o


def la_causal_fwd(q, k, v, o=None, eps=1e-6, S_out=None, z_out=None, ws=None, stream=None,
                  phi=LA_PHI_ELU1):
    """Causal o_i = phi(q_i)^T S_i / (phi(q_i)^T z_i + eps); optional final state out (fp32)."""
    if phi != LA_PHI_ELU1:
        return _causal_phi(q, k, v, None, None, o, eps, S_out, z_out, ws, stream, phi)
    B, H, N, Dk, Dv = _shape4(q, k, v)
    if o is None:
        o = torch.empty_like(v)
    _need_cuda(q, k, v, o, ws, S_out, z_out)
    for t, shp in ((S_out, (B, H, Dk, Dv)), (z_out, (B, H, Dk))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shp):
            raise ValueError(f"state outputs must be float32 with shape {shp}")
    if ws is None:
        ws = workspace(LA_OP_CAUSAL, B, H, N, Dk, Dv, q.dtype, q.device, stream)
    _check(_lib.la_causal_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv, _dt(q),
                              float(eps), _ptr(S_out), _ptr(z_out), _ptr(ws), ws.numel(),
                              _stream(stream)),
           "la_causal_fwd")
    return o


def _causal_phi(q, k, v, S0, z0, o, eps, S_out, z_out, ws, stream, phi):
    B, H, N, Dk, Dv = _shape4(q, k, v)
    if o is None:
        o = torch.empty_like(v)
    _need_cuda(q, k, v, o, ws, S0, z0, S_out, z_out)
    for t, shp in ((S0, (B, H, Dk, Dv)), (z0, (B, H, Dk)), (S_out, (B, H, Dk, Dv)),
                   (z_out, (B, H, Dk))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shp):
            raise ValueError(f"states must be float32 with shape {shp}")
    if ws is None:
        ws = workspace(LA_OP_CAUSAL, B, H, N, Dk, Dv, q.dtype, q.device, stream)
    _check(_lib.la_causal_fwd_phi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv, _dt(q),
                                  int(phi), float(eps), _ptr(S0), _ptr(z0), _ptr(S_out),
                                  _ptr(z_out), _ptr(ws), ws.numel(), _stream(stream)),
           "la_causal_fwd_phi")
    return o


def la_causal_fwd_noalloc(q, k, v, o=None, eps=1e-6, S_out=None, z_out=None, stream=None):
    """la_causal_fwd without a workspace (scratch is a fixed array inside the library).

    The library uses the array of the current device, so the call runs with
    q's device current."""
    B, H, N, Dk, Dv = _shape4(q, k, v)
    if o is None:
        o = torch.empty_like(v)
    _need_cuda(q, k, v, o, S_out, z_out)
    for t, shp in ((S_out, (B, H, Dk, Dv)), (z_out, (B, H, Dk))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shp):
            raise ValueError(f"state outputs must be float32 with shape {shp}")
    with torch.cuda.device(q.device):
        _check(_lib.la_causal_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv,
                                          _dt(q), float(eps), _ptr(S_out), _ptr(z_out),
                                          _stream(stream)),
               "la_causal_fwd_noalloc")
    return o


def la_noalloc_query_status(device=None, stream=None):
    """Reads and clears the device-side status of the no-allocation calls on `device`."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return _lib.la_noalloc_query_status(_stream(stream))


def la_noalloc_set_wait_limit(max_spin_us=0, hold_loads=False, device=None, stream=None):
    """Wait limit (microseconds, 0 = default) and load-withholding test hook of the
    no-allocation calls on `device`."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(_lib.la_noalloc_set_wait_limit(int(max_spin_us), 1 if hold_loads else 0,
                                              _stream(stream)),
               "la_noalloc_set_wait_limit")


def la_causal_fwd_state(q, k, v, S0, z0, o=None, eps=1e-6, S_out=None, z_out=None, ws=None,
                        stream=None, phi=LA_PHI_ELU1):
    """Causal forward continuing from the state (S0 [B,H,Dk,Dv], z0 [B,H,Dk], float32)."""
    if phi != LA_PHI_ELU1:
        return _causal_phi(q, k, v, S0, z0, o, eps, S_out, z_out, ws, stream, phi)
    B, H, N, Dk, Dv = _shape4(q, k, v)
    if o is None:
        o = torch.empty_like(v)
    _need_cuda(q, k, v, o, ws, S0, z0, S_out, z_out)
    for t, shp in ((S0, (B, H, Dk, Dv)), (z0, (B, H, Dk)), (S_out, (B, H, Dk, Dv)),
                   (z_out, (B, H, Dk))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shp):
            raise ValueError(f"states must be float32 with shape {shp}")
    if ws is None:
        ws = workspace(LA_OP_CAUSAL, B, H, N, Dk, Dv, q.dtype, q.device, stream)
    _check(_lib.la_causal_fwd_state(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv, _dt(q),
                                    float(eps), _ptr(S0), _ptr(z0), _ptr(S_out), _ptr(z_out),
                                    _ptr(ws), ws.numel(), _stream(stream)),
           "la_causal_fwd_state")
    return o


def _bwd(fn, op, q, k, v, dout, dq, dk, dv, eps, ws, stream, phi=LA_PHI_ELU1):
    B, H, N, Dk, Dv = _shape4(q, k, v)
    if dout.shape != v.shape or dout.dtype != v.dtype:
        raise ValueError("dout must be shaped and typed like v")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _need_cuda(q, k, v, dout, dq, dk, dv, ws)
    if ws is None:
        ws = workspace(op, B, H, N, Dk, Dv, q.dtype, q.device, stream)
    if phi == LA_PHI_ELU1:
        _check(getattr(_lib, fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk),
                                 _ptr(dv), B, H, N, Dk, Dv, _dt(q), float(eps), _ptr(ws),
                                 ws.numel(), _stream(stream)),
               fn)
    else:
        _check(getattr(_lib, fn + "_phi")(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq),
                                          _ptr(dk), _ptr(dv), B, H, N, Dk, Dv, _dt(q), int(phi),
                                          float(eps), _ptr(ws), ws.numel(), _stream(stream)),
               fn + "_phi")
    return dq, dk, dv


def la_causal_bwd(q, k, v, dout, dq=None, dk=None, dv=None, eps=1e-6, ws=None, stream=None,
                  phi=LA_PHI_ELU1):
    """Gradients (dq, dk, dv) of sum(o * dout) for the causal forward o of (q, k, v)."""
    return _bwd("la_causal_bwd", LA_OP_CAUSAL_BWD, q, k, v, dout, dq, dk, dv, eps, ws, stream,
                phi)


def la_noncausal_bwd(q, k, v, dout, dq=None, dk=None, dv=None, eps=1e-6, ws=None, stream=None,
                     phi=LA_PHI_ELU1):
    """Gradients (dq, dk, dv) of sum(o * dout) for the non-causal forward o of (q, k, v)."""
    return _bwd("la_noncausal_bwd", LA_OP_NONCAUSAL_BWD, q, k, v, dout, dq, dk, dv, eps, ws,
                stream, phi)


def la_host_staging_size(B, H, N, Dk, Dv, dtype):
    """Device staging bytes la_causal_fwd_host needs at this shape."""
    dt = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    n = ctypes.c_size_t(0)
    _check(_lib.la_host_staging_size(B, H, N, Dk, Dv, dt, ctypes.byref(n)), "la_host_staging_size")
    return int(n.value)


def host_staging(B, H, N, Dk, Dv, dtype, device=None):
    """Allocates (through PyTorch) the device staging buffer of la_causal_fwd_host."""
    n = la_host_staging_size(B, H, N, Dk, Dv, dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def la_causal_fwd_host(q, k, v, o=None, eps=1e-6, S_out=None, z_out=None, staging=None, ws=None,
                       device=None, stream=None):
    """Causal forward on host (CPU) tensors, transfers overlapped with compute; returns o on the
    host. q, k, v should be pinned (tensor.pin_memory()); S_out, z_out are CUDA tensors."""
    B, H, N, Dk, Dv = _shape4(q, k, v)
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous host tensors")
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, pin_memory=True)
    if o.is_cuda or not o.is_contiguous() or o.shape != v.shape or o.dtype != v.dtype:
        raise ValueError("o must be a contiguous host tensor shaped and typed like v")
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    _need_cuda(S_out, z_out, staging, ws)
    for t, shp in ((S_out, (B, H, Dk, Dv)), (z_out, (B, H, Dk))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shp):
            raise ValueError(f"state outputs must be float32 with shape {shp}")
    if staging is None:
        staging = host_staging(B, H, N, Dk, Dv, q.dtype, dev)
    if ws is None:
        ws = workspace(LA_OP_CAUSAL, B, H, N, Dk, Dv, q.dtype, dev, stream)
    _check(_lib.la_causal_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, N, Dk, Dv, _dt(q),
                                   float(eps), _ptr(S_out), _ptr(z_out), _ptr(staging),
                                   staging.numel(), _ptr(ws), ws.numel(), _stream(stream)),
           "la_causal_fwd_host")
    return o


def la_decode_step(q, k, v, S, z, o=None, eps=1e-6, stream=None, phi=LA_PHI_ELU1):
    """One recurrent step on (S, z) in place; q, k [B,H,Dk], v [B,H,Dv]; returns o [B,H,Dv]."""
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError("expected q, k [B,H,Dk] and v [B,H,Dv]")
    B, H, Dk = q.shape
    Dv = v.shape[2]
    if S.dtype != torch.float32 or z.dtype != torch.float32 or tuple(S.shape) != (B, H, Dk, Dv) \
            or tuple(z.shape) != (B, H, Dk):
        raise ValueError("S must be float32 [B,H,Dk,Dv] and z float32 [B,H,Dk]")
    if o is None:
        o = torch.empty_like(v)
    _need_cuda(q, k, v, o, S, z)
    if phi == LA_PHI_ELU1:
        _check(_lib.la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(S), _ptr(z), B, H, Dk,
                                   Dv, _dt(q), float(eps), _stream(stream)),
               "la_decode_step")
    else:
        _check(_lib.la_decode_step_phi(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(S), _ptr(z), B, H,
                                       Dk, Dv, _dt(q), int(phi), float(eps), _stream(stream)),
               "la_decode_step_phi")
    return o


def la_positive_random_features(x, W, out=None, shift=0.0, stream=None):
    """exp(W x - |x|^2 / 2 - shift) / sqrt(R) over the last axis of x [..., D]; W [R, D].

    Returns out [..., R] in x's dtype: features for the LA_PHI_IDENTITY entries."""
    if W.dim() != 2 or x.shape[-1] != W.shape[1] or W.dtype != x.dtype:
        raise ValueError("expected x [..., D] and W [R, D] of one dtype")
    R, D = W.shape
    rows = x.numel() // D if D else 0
    if out is None:
        out = torch.empty(tuple(x.shape[:-1]) + (R,), dtype=x.dtype, device=x.device)
    _need_cuda(x, W, out)
    _check(_lib.la_positive_random_features(_ptr(x), _ptr(W), _ptr(out), rows, D, R, _dt(x),
                                            float(shift), _stream(stream)),
           "la_positive_random_features")
    return out


def la_layer_decode_step(x, Wqkv, Wo, S, z, H, y=None, eps=1e-6, ws=None, stream=None):
    """One decode step of a linear-attention layer: x [B, d_model] -> y [B, d_model].

    Wqkv [d_model, 3 H D] (q | k | v, head-major within each), Wo [H D, d_model];
    S [B, H, D, D] and z [B, H, D] (float32) are updated in place."""
    if x.dim() != 2 or Wqkv.dim() != 2 or Wo.dim() != 2:
        raise ValueError("expected x [B, d_model], Wqkv [d_model, 3 H D], Wo [H D, d_model]")
    B, dm = x.shape
    D = dm // H if H else 0
    if H * D != dm or tuple(Wqkv.shape) != (dm, 3 * dm) or tuple(Wo.shape) != (dm, dm):
        raise ValueError("d_model must equal H D, Wqkv be [d_model, 3 d_model], Wo [d_model, d_model]")
    if Wqkv.dtype != x.dtype or Wo.dtype != x.dtype:
        raise TypeError("x, Wqkv and Wo must share one dtype")
    if S.dtype != torch.float32 or z.dtype != torch.float32 or tuple(S.shape) != (B, H, D, D) \
            or tuple(z.shape) != (B, H, D):
        raise ValueError("S must be float32 [B,H,D,D] and z float32 [B,H,D]")
    if y is None:
        y = torch.empty_like(x)
    _need_cuda(x, Wqkv, Wo, y, S, z, ws)
    if ws is None:
        ws = workspace(LA_OP_LAYER_DECODE, B, H, 1, D, D, x.dtype, x.device, stream)
    _check(_lib.la_layer_decode_step(_ptr(x), _ptr(Wqkv), _ptr(Wo), _ptr(y), _ptr(S), _ptr(z), B,
                                     H, D, _dt(x), float(eps), _ptr(ws), ws.numel(),
                                     _stream(stream)),
           "la_layer_decode_step")
    return y


_NO_SCOPE = contextlib.nullcontext()
# The stream handle alone: the Stream object that torch.cuda.current_stream() builds
# costs a call more than the rest of its argument handling.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _device_of(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return index


def _same_device(index, *ts):
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one CUDA device")


def _scope(index, stream):
    """Context in which a call on tensors of device `index` allocates and launches: that device,
    and the given stream (so that what the call allocates belongs to the stream that uses it)."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
        return torch.cuda.stream(stream)
    return _NO_SCOPE if index == torch.cuda.current_device() else torch.cuda.device(index)


def _addr(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _inner_adjacent(t, what, inner):
    """Strides of t, whose last `inner` dimensions must be adjacent values (a column range of a
    projection's rows, for instance)."""
    strides = t.stride()
    if not t.is_contiguous():
        want = 1
        for size, stride in zip(reversed(t.shape[-inner:]), reversed(strides[-inner:])):
            if size > 1 and stride != want:
                raise ValueError(f"{what}: a token's values must be adjacent (strides {strides})")
            want *= size
    return strides


def la_rope_table(inv_freq, axis=None, device="cuda"):
    """Table of the position rotation: int64 [pairs, 2] on `device`, one (step, axis) per pair.

    inv_freq: radians per position of each rotated pair (a sequence or CPU tensor of float64);
    axis: the position axis of each pair (default: all 0)."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
    if f.dim() != 1:
        raise ValueError("inv_freq must be one-dimensional")
    ax = None
    if axis is not None:
        ax = torch.as_tensor(axis, device="cpu").to(torch.int32).contiguous()
        if ax.shape != f.shape:
            raise ValueError("axis must have one entry per pair")
    table = torch.empty(f.numel(), 2, dtype=torch.int64)
    _check(_lib.la_rope_table(_addr(f), _addr(ax), f.numel(), LA_ROPE_MAX_AXES, _addr(table)),
           "la_rope_table")
    return table.to(device)


def _rope_args(q, k, pos, table, wq, wk, norm):
    """Checks shared by both directions; returns (device index, B, N, Hq, Hk, D, axes)."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    shape, dtype = ref.shape, ref.dtype
    if len(shape) != 4:
        raise ValueError("expected q [B,N,Hq,D] and k [B,N,Hk,D]")
    B, N, Hq, D = shape
    Hk = Hq
    if q is None:
        Hq = 0
    elif k is None:
        Hk = 0
    else:
        if k.dim() != 4 or k.shape[0] != B or k.shape[1] != N or k.shape[3] != D:
            raise ValueError("expected q [B,N,Hq,D] and k [B,N,Hk,D]")
        if k.dtype != dtype:
            raise TypeError("q and k must share one dtype")
        Hk = k.shape[2]
    index = _device_of(ref)
    for w in (wq, wk):
        if w is None:
            continue
        if not norm:
            raise ValueError("norm weights need norm=True")
        if w.dtype != dtype or w.dim() != 1 or w.shape[0] != D or not w.is_contiguous():
            raise ValueError("norm weights must be contiguous [D] in q's dtype")
    pshape = pos.shape
    if pos.dtype != torch.int32 or not pos.is_contiguous() or len(pshape) not in (2, 3) or pshape[0] != B \
            or pshape[1] != N:
        raise ValueError("pos must be contiguous int32 [B,N] or [B,N,axes]")
    if table.dtype != torch.int64 or table.dim() != 2 or table.shape[1] != 2 or not table.is_contiguous():
        raise ValueError("table must come from la_rope_table (int64 [pairs, 2])")
    _same_device(index, k, pos, table, wq, wk)
    return index, B, N, Hq, Hk, D, pshape[2] if len(pshape) == 3 else 1


def _head_major(t, B, H, N, D, like, what):
    if t.shape != (B, H, N, D) or t.dtype != like.dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous [B,H,N,D] = {(B, H, N, D)} in q's dtype")


def la_qk_norm_rope_fwd(q, k, pos, table, wq=None, wk=None, norm=True, eps=1e-6, interleaved=False,
                        qo=None, ko=None, stream=None):
    """Per-head RMS norm (norm=True) and position rotation of q [B,N,Hq,D] and k [B,N,Hk,D].

    q and k may be column ranges of one projection; either may be None. pos: int32 [B,N] or
    [B,N,axes]; table: la_rope_table. Returns (qo [B,Hq,N,D], ko [B,Hk,N,D]), head-major, ready
    for the attention entries."""
    index, B, N, Hq, Hk, D, axes = _rope_args(q, k, pos, table, wq, wk, norm)
    ref = q if q is not None else k
    qs = _inner_adjacent(q, "q", 2) if q is not None else (0, 0)
    ks = _inner_adjacent(k, "k", 2) if k is not None else (0, 0)
    with _scope(index, stream):
        if q is not None:
            if qo is None:
                qo = torch.empty((B, Hq, N, D), dtype=ref.dtype, device=ref.device)
            else:
                _head_major(qo, B, Hq, N, D, ref, "qo")
        if k is not None:
            if ko is None:
                ko = torch.empty((B, Hk, N, D), dtype=ref.dtype, device=ref.device)
            else:
                _head_major(ko, B, Hk, N, D, ref, "ko")
        _same_device(index, qo, ko)
        _check(_lib.la_qk_norm_rope_fwd(
            _addr(q), qs[0], qs[1], _addr(k), ks[0], ks[1], _addr(wq), _addr(wk), pos.data_ptr(), axes,
            table.data_ptr(), table.shape[0], _addr(qo), _addr(ko), B, N, Hq, Hk, D, _dt(ref),
            1 if norm else 0, eps, 1 if interleaved else 0, _raw_stream(index)), "la_qk_norm_rope_fwd")
    return qo, ko


def la_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hk, D):
    """Workspace bytes of la_qk_norm_rope_bwd with the norm."""
    n = ctypes.c_size_t(0)
    _check(_lib.la_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hk, D, ctypes.byref(n)),
           "la_qk_norm_rope_bwd_workspace_size")
    return int(n.value)


def qk_norm_rope_workspace(B, N, Hq, Hk, D, device=None):
    """Allocates (through PyTorch) the workspace of la_qk_norm_rope_bwd; it needs no initialisation."""
    n = la_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hk, D)
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda" if device is None else device)


def la_qk_norm_rope_bwd(q, k, dqo, dko, pos, table, wq=None, wk=None, norm=True, eps=1e-6,
                        interleaved=False, dq=None, dk=None, ws=None, stream=None):
    """Gradients (dq, dk, dwq, dwk) of sum(qo * dqo) + sum(ko * dko) of la_qk_norm_rope_fwd.

    dq [B,N,Hq,D] and dk [B,N,Hk,D] may be given as column ranges of one projection gradient.
    dwq, dwk are float32 [D], None without the norm (or without weights of that side). Without
    the norm the gradient needs no inputs: q and k may be None."""
    if norm or q is not None or k is not None:
        for t, x, what in ((dqo, q, "dqo"), (dko, k, "dko")):
            if (t is None) != (x is None):
                raise ValueError(f"{what} must be given exactly when its input is")
        qx, kx = q, k
    else:
        qx, kx = (t.transpose(1, 2) if t is not None and t.dim() == 4 else t for t in (dqo, dko))
    index, B, N, Hq, Hk, D, axes = _rope_args(qx, kx, pos, table, wq, wk, norm)
    ref = qx if qx is not None else kx
    qs = _inner_adjacent(q, "q", 2) if q is not None else (0, 0)
    ks = _inner_adjacent(k, "k", 2) if k is not None else (0, 0)
    for t, H, what in ((dqo, Hq, "dqo"), (dko, Hk, "dko")):
        if t is not None:
            _head_major(t, B, H, N, D, ref, what)
    with _scope(index, stream):
        if dq is None and qx is not None:
            dq = torch.empty((B, N, Hq, D), dtype=ref.dtype, device=ref.device)
        if dk is None and kx is not None:
            dk = torch.empty((B, N, Hk, D), dtype=ref.dtype, device=ref.device)
        for t, x, what in ((dq, qx, "dq"), (dk, kx, "dk")):
            if t is not None and (x is None or t.shape != x.shape or t.dtype != ref.dtype):
                raise ValueError(f"{what} must be shaped and typed like its input")
        dqs = _inner_adjacent(dq, "dq", 2) if dq is not None else (0, 0)
        dks = _inner_adjacent(dk, "dk", 2) if dk is not None else (0, 0)
        dwq = torch.empty(D, dtype=torch.float32, device=ref.device) if wq is not None else None
        dwk = torch.empty(D, dtype=torch.float32, device=ref.device) if wk is not None else None
        if ws is None and norm:
            ws = qk_norm_rope_workspace(B, N, Hq, Hk, D, ref.device)
        _same_device(index, dqo, dko, dq, dk, ws)
        _check(_lib.la_qk_norm_rope_bwd(
            _addr(q), qs[0], qs[1], _addr(k), ks[0], ks[1], _addr(wq), _addr(wk), pos.data_ptr(), axes,
            table.data_ptr(), table.shape[0], _addr(dqo), _addr(dko), _addr(dq), dqs[0], dqs[1], _addr(dk),
            dks[0], dks[1], _addr(dwq), _addr(dwk), B, N, Hq, Hk, D, _dt(ref), 1 if norm else 0, eps,
            1 if interleaved else 0, _addr(ws), _bytes(ws), _raw_stream(index)), "la_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def _conv_args(x, w, bias, dims):
    """Checks shared by the prompt and the step; returns (device index, x's strides, C, W)."""
    wshape, dtype = w.shape, x.dtype
    if x.dim() != dims or len(wshape) != 2 or wshape[0] != x.shape[-1]:
        raise ValueError("expected x [B,N,C] (one token: [B,C]) and w [C,W]")
    _dt(x)
    index = _device_of(x)
    if w.dtype != dtype or not w.is_contiguous():
        raise ValueError("w must be contiguous [C,W] in x's dtype")
    if bias is not None and (bias.dtype != dtype or bias.dim() != 1 or bias.shape[0] != wshape[0]
                             or not bias.is_contiguous()):
        raise ValueError("bias must be contiguous [C] in x's dtype")
    return index, _inner_adjacent(x, "x", 1), wshape[0], wshape[1]


def _conv_state(t, B, C, W, x, what):
    if t is not None and (t.shape != (B, W - 1, C) or t.dtype != x.dtype or not t.is_contiguous()):
        raise ValueError(f"{what} must be contiguous [B,W-1,C] = {(B, W - 1, C)} in x's dtype")


def _like(y, x, inner):
    if y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError("y must be shaped and typed like x")
    return _inner_adjacent(y, "y", inner)


def _check_lengths(lengths, B):
    if lengths is not None and (lengths.dtype != torch.int32 or lengths.shape != (B,)
                                or not lengths.is_contiguous()):
        raise ValueError("lengths must be contiguous int32 [B]")


def la_short_conv_fwd(x, w, bias=None, silu=True, lengths=None, state0=None, state_out=None, y=None,
                      return_state=False, stream=None):
    """Causal depthwise convolution of x [B,N,C] (strided rows allowed) with w [C,W], W in 2..4.

    state0 [B,W-1,C]: the inputs before the first token; the last W - 1 inputs go to state_out
    (allocated with return_state=True). lengths (int32 [B]): rows past them are left as they are
    (zero where the call makes y). Returns y, or (y, state_out) with return_state=True."""
    index, xs, C, W = _conv_args(x, w, bias, 3)
    B, N, _ = x.shape
    _conv_state(state0, B, C, W, x, "state0")
    _check_lengths(lengths, B)
    with _scope(index, stream):
        if y is None:
            make = torch.empty if lengths is None else torch.zeros
            y = make((B, N, C), dtype=x.dtype, device=x.device)
        if state_out is None and return_state:
            state_out = torch.empty((B, W - 1, C), dtype=x.dtype, device=x.device)
        ys = _like(y, x, 1)
        _conv_state(state_out, B, C, W, x, "state_out")
        _same_device(index, w, bias, lengths, state0, state_out, y)
        _check(_lib.la_short_conv_fwd(
            x.data_ptr(), xs[0], xs[1], w.data_ptr(), _addr(bias), 1 if silu else 0, _addr(lengths),
            _addr(state0), _addr(state_out), y.data_ptr(), ys[0], ys[1], B, N, C, W, _dt(x),
            _raw_stream(index)), "la_short_conv_fwd")
    return (y, state_out) if return_state else y


def la_short_conv_step(x, w, state, bias=None, silu=True, y=None, stream=None):
    """One token of the convolution: x [B,C] -> y [B,C]; state [B,W-1,C] is shifted in place."""
    index, xs, C, W = _conv_args(x, w, bias, 2)
    B = x.shape[0]
    if state is None:
        raise ValueError("state must be given")
    _conv_state(state, B, C, W, x, "state")
    with _scope(index, stream):
        if y is None:
            y = torch.empty((B, C), dtype=x.dtype, device=x.device)
            ys = (C, 1)
        else:
            ys = _like(y, x, 1)
        _same_device(index, w, bias, state, y)
        _check(_lib.la_short_conv_step(
            x.data_ptr(), xs[0], w.data_ptr(), _addr(bias), 1 if silu else 0, state.data_ptr(), y.data_ptr(),
            ys[0], B, C, W, _dt(x), _raw_stream(index)), "la_short_conv_step")
    return y


def _scan_args(x, step, A, Bm, Cm, D, z, step_bias, lead):
    """Checks shared by the prompt (lead = 2: [B,N,..]) and the step (lead = 1: [B,..]); returns
    (device index, shape of x, G, S)."""
    xshape, bshape, dtype = x.shape, Bm.shape, x.dtype
    if len(xshape) != lead + 2 or len(bshape) != lead + 2 or Cm.shape != bshape or \
            bshape[:lead] != xshape[:lead] or step.shape != xshape[:-1] or \
            (z is not None and z.shape != xshape):
        dims = "[B,N,H,P]" if lead == 2 else "[B,H,P]"
        raise ValueError(f"expected x (and z) {dims}, step one value per head, Bm and Cm with [G,S] per token")
    if step.dtype != dtype or Bm.dtype != dtype or Cm.dtype != dtype or (z is not None and z.dtype != dtype):
        raise TypeError("x, step, Bm, Cm and z must share one dtype")
    _dt(x)
    index = _device_of(x)
    if A is None:
        raise ValueError("A must be given")
    for t, what in ((A, "A"), (D, "D"), (step_bias, "dt_bias")):
        if t is not None and (t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != xshape[-2]
                              or not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous float32 [H]")
    _same_device(index, step, A, Bm, Cm, D, z, step_bias)
    return index, xshape, bshape[-2], bshape[-1]


def _f32_state(t, shape, what):
    if t is not None and (t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what} must be contiguous float32 with shape {shape}")


def la_selective_scan_fwd(x, step, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True,
                          lengths=None, S0=None, S_out=None, y=None, ws=None, stream=None):
    """Selective scan of x [B,N,H,P] with step sizes [B,N,H], rates A [H], Bm, Cm [B,N,G,S].

    y_t = (C_t^T S_t + D x_t) silu(z_t) with S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T and
    d_t = softplus(step_t + dt_bias); a step of minus infinity masks its token. S0, S_out [B,H,S,P]
    float32 (S_out may be S0). lengths (int32 [B]): rows past them are left as they are (zero where
    the call makes y). Token rows may be strided (column ranges of a projection). Returns y
    [B,N,H,P]."""
    index, (B, N, H, P), G, S = _scan_args(x, step, A, Bm, Cm, D, z, dt_bias, 2)
    _f32_state(S0, (B, H, S, P), "S0")
    _f32_state(S_out, (B, H, S, P), "S_out")
    _check_lengths(lengths, B)
    xs, ss = _inner_adjacent(x, "x", 2), _inner_adjacent(step, "step", 1)
    bs, cs = _inner_adjacent(Bm, "Bm", 2), _inner_adjacent(Cm, "Cm", 2)
    zs = _inner_adjacent(z, "z", 2) if z is not None else (0, 0)
    with _scope(index, stream):
        if y is None:
            make = torch.empty if lengths is None else torch.zeros
            y = make((B, N, H, P), dtype=x.dtype, device=x.device)
        ys = _like(y, x, 2)
        if ws is None:
            ws = workspace(LA_OP_SELECTIVE_SCAN, B, H, N, S, P, x.dtype, x.device)
        _same_device(index, lengths, S0, S_out, y, ws)
        _check(_lib.la_selective_scan_fwd(
            x.data_ptr(), xs[0], xs[1], step.data_ptr(), ss[0], ss[1], A.data_ptr(), Bm.data_ptr(), bs[0],
            bs[1], Cm.data_ptr(), cs[0], cs[1], _addr(D), _addr(z), zs[0], zs[1], _addr(dt_bias),
            1 if softplus else 0, _addr(lengths), _addr(S0), _addr(S_out), y.data_ptr(), ys[0], ys[1], B, H,
            G, N, S, P, _dt(x), ws.data_ptr(), _bytes(ws), _raw_stream(index)), "la_selective_scan_fwd")
    return y


def la_selective_scan_step(x, step, A, Bm, Cm, S, D=None, z=None, dt_bias=None, softplus=True,
                           y=None, stream=None):
    """One token of the scan: x [B,H,P], step [B,H], Bm, Cm [B,G,S]; S [B,H,S,P] in place."""
    index, (B, H, P), G, Sn = _scan_args(x, step, A, Bm, Cm, D, z, dt_bias, 1)
    if S is None:
        raise ValueError("S must be given")
    _f32_state(S, (B, H, Sn, P), "S")
    xs, ss = _inner_adjacent(x, "x", 2), _inner_adjacent(step, "step", 1)
    bs, cs = _inner_adjacent(Bm, "Bm", 2), _inner_adjacent(Cm, "Cm", 2)
    zs = _inner_adjacent(z, "z", 2) if z is not None else (0,)
    with _scope(index, stream):
        if y is None:
            y = torch.empty((B, H, P), dtype=x.dtype, device=x.device)
        ys = _like(y, x, 2)
        _same_device(index, S, y)
        _check(_lib.la_selective_scan_step(
            x.data_ptr(), xs[0], step.data_ptr(), ss[0], A.data_ptr(), Bm.data_ptr(), bs[0], Cm.data_ptr(),
            cs[0], _addr(D), _addr(z), zs[0], _addr(dt_bias), 1 if softplus else 0, S.data_ptr(),
            y.data_ptr(), ys[0], B, H, G, Sn, P, _dt(x), _raw_stream(index)), "la_selective_scan_step")
    return y


def _decay_args(q, k, v, decay, dims):
    """Checks shared by the prompt (dims = 4: [B,H,N,D]) and the step (3: [B,H,D]); returns
    (device index, shape of q, Dv, element type)."""
    qshape, vshape, dtype = q.shape, v.shape, q.dtype
    if len(qshape) != dims or k.shape != qshape or len(vshape) != dims or vshape[:-1] != qshape[:-1]:
        lead = "B,H,N" if dims == 4 else "B,H"
        raise ValueError(f"expected q, k [{lead},Dk] and v [{lead},Dv]; got {tuple(qshape)}, "
                         f"{tuple(k.shape)}, {tuple(vshape)}")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v must share one dtype")
    dt = _dt(q)
    index = _device_of(q)
    if decay.dtype != torch.float32 or decay.shape != qshape[1:2] or not decay.is_contiguous():
        raise ValueError("decay must be contiguous float32 [H]")
    if k.get_device() != index or v.get_device() != index or decay.get_device() != index:
        raise ValueError("tensors must be on one CUDA device")
    return index, qshape, vshape[-1], dt


# Host arrays of strides: of the axes but the last, tensor by tensor.
_I64x8, _I64x12, _I64x21 = (ctypes.c_int64 * n for n in (8, 12, 21))


def _rows(t, what):
    """Strides of a tensor whose last axis' values must be adjacent."""
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what}: a row's values must be adjacent (strides {s})")
    return s


def _typed_like(t, ref, what):
    if t.shape != ref.shape or t.dtype != ref.dtype:
        raise ValueError(f"{what} must be shaped and typed like its input")


def la_decay_attn_fwd(q, k, v, decay, scale=1.0, lengths=None, S0=None, S_out=None, o=None, ws=None, stream=None):
    """Causal linear attention with a decay per head: o_t = scale S_t^T q_t, S_t = e^decay S_{t-1} + k_t v_t^T.

    q, k [B,H,N,Dk], v [B,H,N,Dv]: any batch, head and token strides (column ranges of a projection,
    transposed to head-major; a row's values adjacent). decay: float32 [H], the logarithm of the factor
    per token. S0, S_out [B,H,Dk,Dv] float32 (S_out may be S0). lengths (int32 [B]): rows past them are
    left as they are (zero where the call makes o). Returns o [B,H,N,Dv]."""
    index, (B, H, N, Dk), Dv, dt = _decay_args(q, k, v, decay, 4)
    _f32_state(S0, (B, H, Dk, Dv), "S0")
    _f32_state(S_out, (B, H, Dk, Dv), "S_out")
    _check_lengths(lengths, B)
    with _scope(index, stream):
        if o is None:
            make = torch.empty if lengths is None else torch.zeros
            o = make((B, H, N, Dv), dtype=q.dtype, device=q.device)
        _typed_like(o, v, "o")
        if ws is None:
            ws = workspace(LA_OP_DECAY_ATTN, B, H, N, Dk, Dv, q.dtype, q.device)
        _same_device(index, lengths, S0, S_out, o, ws)
        sq, sk, sv, so = _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), _rows(o, "o")
        _check(_lib.la_decay_attn_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), scale, _addr(lengths), _addr(S0),
            _addr(S_out), o.data_ptr(), _I64x12(*sq[:3], *sk[:3], *sv[:3], *so[:3]), B, H, N, Dk, Dv, dt,
            ws.data_ptr(), _bytes(ws), _raw_stream(index)), "la_decay_attn_fwd")
    return o


def la_decay_attn_bwd(q, k, v, dout, decay, scale=1.0, lengths=None, dq=None, dk=None, dv=None, ws=None,
                      stream=None):
    """Gradients (dq, dk, dv) of sum(o * dout) of la_decay_attn_fwd without states (decay a constant).

    Strides as there; dq, dk and dv may be given as column ranges of one projection gradient. Rows past
    the lengths are left as they are (zero where the call makes them)."""
    index, (B, H, N, Dk), Dv, dt = _decay_args(q, k, v, decay, 4)
    _typed_like(dout, v, "dout")
    _check_lengths(lengths, B)
    with _scope(index, stream):
        make = torch.empty if lengths is None else torch.zeros
        grads = [make(x.shape, dtype=x.dtype, device=x.device) if t is None else t
                 for t, x in ((dq, q), (dk, k), (dv, v))]
        for t, x, what in zip(grads, (q, k, v), ("dq", "dk", "dv")):
            _typed_like(t, x, what)
        dq, dk, dv = grads
        if ws is None:
            ws = workspace(LA_OP_DECAY_ATTN_BWD, B, H, N, Dk, Dv, q.dtype, q.device)
        _same_device(index, dout, lengths, dq, dk, dv, ws)
        strides = _I64x21(*(s for t, what in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv"))
                            for s in _rows(t, what)[:3]))
        _check(_lib.la_decay_attn_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(), decay.data_ptr(), scale, _addr(lengths),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), strides, B, H, N, Dk, Dv, dt, ws.data_ptr(), _bytes(ws),
            _raw_stream(index)), "la_decay_attn_bwd")
    return dq, dk, dv


def la_decay_attn_step(q, k, v, decay, S, scale=1.0, o=None, stream=None):
    """One token of la_decay_attn_fwd: q, k [B,H,Dk], v [B,H,Dv]; S [B,H,Dk,Dv] in place; returns o [B,H,Dv]."""
    index, (B, H, Dk), Dv, dt = _decay_args(q, k, v, decay, 3)
    if S is None:
        raise ValueError("S must be given")
    _f32_state(S, (B, H, Dk, Dv), "S")
    if S.get_device() != index:
        raise ValueError("tensors must be on one CUDA device")
    with _scope(index, stream):
        if o is None:
            o = torch.empty((B, H, Dv), dtype=q.dtype, device=q.device)
        else:
            _typed_like(o, v, "o")
            _same_device(index, o)
        sq, sk, sv, so = _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), _rows(o, "o")
        _check(_lib.la_decay_attn_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), scale, S.data_ptr(), o.data_ptr(),
            _I64x8(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1]), B, H, Dk, Dv, dt, _raw_stream(index)),
            "la_decay_attn_step")
    return o


def la_group_norm_workspace_size(B, N, C, G):
    """Workspace bytes of la_group_norm_fwd and la_group_norm_bwd."""
    n = ctypes.c_size_t(0)
    _check(_lib.la_group_norm_workspace_size(B, N, C, G, ctypes.byref(n)), "la_group_norm_workspace_size")
    return int(n.value)


def group_norm_workspace(B, N, C, G, device=None):
    """Allocates (through PyTorch) the workspace of the group norm, both directions; it needs no initialisation."""
    n = la_group_norm_workspace_size(B, N, C, G)
    return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda" if device is None else device)


def _norm_args(x, groups, w, b, z):
    """Checks shared by both directions; returns (device index, B, N, C, element type)."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 3 or groups < 1 or shape[2] % groups:
        raise ValueError(f"expected x [B,N,C] with C a multiple of groups; got {tuple(shape)}, {groups} groups")
    dt = _dt(x)
    index = _device_of(x)
    for t in (w, b):
        if t is not None and (t.dtype != dtype or t.shape != shape[2:] or not t.is_contiguous()):
            raise ValueError("w and b must be contiguous [C] in x's dtype")
    if z is not None:
        _typed_like(z, x, "z")
    _same_device(index, w, b, z)
    return index, shape[0], shape[1], shape[2], dt


def la_group_norm_fwd(x, groups, w=None, b=None, z=None, silu=False, eps=1e-5, y=None, stats=None,
                      return_stats=False, ws=None, stream=None):
    """Group norm of channels-last rows x [B,N,C]: y = act(w xh + b) silu(z), statistics over N and C / groups.

    silu: act is the silu (else the identity); z [B,N,C]: the gate. A row of its own per sample (the
    heads of an attention output, tokens as samples) is N = 1. Rows may be strided. Returns y, or
    (y, stats) with return_stats=True: stats [B,groups,2] float32 (mean, inverse deviation; zeros
    where there are no tokens)."""
    index, B, N, C, dt = _norm_args(x, groups, w, b, z)
    xs = _rows(x, "x")
    zs = _rows(z, "z") if z is not None else (0, 0)
    with _scope(index, stream):
        if y is None:
            y = torch.empty((B, N, C), dtype=x.dtype, device=x.device)
        else:
            _typed_like(y, x, "y")
            _same_device(index, y)
        ys = _rows(y, "y")
        if stats is not None:
            _f32_state(stats, (B, groups, 2), "stats")
            _same_device(index, stats)
        elif return_stats:
            stats = torch.empty((B, groups, 2), dtype=torch.float32, device=x.device)
        if N == 0 and stats is not None:
            stats.zero_()                       # the library writes nothing then
        if ws is None:
            if N != 1:
                ws = group_norm_workspace(B, N, C, groups, x.device)
        else:
            _same_device(index, ws)
        _check(_lib.la_group_norm_fwd(
            x.data_ptr(), xs[0], xs[1], _addr(w), _addr(b), _addr(z), zs[0], zs[1], y.data_ptr(), ys[0], ys[1],
            _addr(stats), B, N, C, groups, dt, 1 if silu else 0, eps, _addr(ws), _bytes(ws),
            _raw_stream(index)), "la_group_norm_fwd")
    return (y, stats) if return_stats else y


def la_group_norm_bwd(x, groups, dy, stats, w=None, b=None, z=None, silu=False, dx=None, dz=None, ws=None,
                      stream=None):
    """Gradients (dx, dw, db, dz) of sum(y * dy) of la_group_norm_fwd; stats: as it returns them.

    dx, dz [B,N,C] in x's dtype (dz None without a gate); dw, db float32 [C] (None without w, b)."""
    index, B, N, C, dt = _norm_args(x, groups, w, b, z)
    _typed_like(dy, x, "dy")
    if stats is None:
        raise ValueError("stats must be given")
    _f32_state(stats, (B, groups, 2), "stats")
    if dz is not None and z is None:
        raise ValueError("dz needs z")
    xs, gs = _rows(x, "x"), _rows(dy, "dy")
    zs = _rows(z, "z") if z is not None else (0, 0)
    with _scope(index, stream):
        if dx is None:
            dx = torch.empty((B, N, C), dtype=x.dtype, device=x.device)
        if dz is None and z is not None:
            dz = torch.empty((B, N, C), dtype=x.dtype, device=x.device)
        _typed_like(dx, x, "dx")
        dxs, dzs = _rows(dx, "dx"), (0, 0)
        if dz is not None:
            _typed_like(dz, x, "dz")
            dzs = _rows(dz, "dz")
        dw = torch.empty(C, dtype=torch.float32, device=x.device) if w is not None else None
        db = torch.empty(C, dtype=torch.float32, device=x.device) if b is not None else None
        if ws is None:
            ws = group_norm_workspace(B, N, C, groups, x.device)
        _same_device(index, dy, stats, dx, dz, ws)
        _check(_lib.la_group_norm_bwd(
            x.data_ptr(), xs[0], xs[1], _addr(w), _addr(b), _addr(z), zs[0], zs[1], dy.data_ptr(), gs[0], gs[1],
            stats.data_ptr(), dx.data_ptr(), dxs[0], dxs[1], _addr(dz), dzs[0], dzs[1], _addr(dw), _addr(db), B, N,
            C, groups, dt, 1 if silu else 0, _addr(ws), _bytes(ws), _raw_stream(index)), "la_group_norm_bwd")
    return dx, dw, db, dz


def la_query_status(ws, stream=None):
    """Synchronises the stream and returns (and clears) the workspace status code."""
    return int(_lib.la_query_status(_ptr(ws), _stream(stream)))

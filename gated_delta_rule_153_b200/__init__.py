"""Python binding of libgdn.so, the sm_100a gated delta-rule library.

Argument marshalling only: every function below checks tensor shapes, dtypes
and devices, allocates outputs with torch (device memory is torch's job),
and calls the C entry point of the same name through ctypes on the current
CUDA stream.  No arithmetic of the layer happens in Python, and there is no
CPU fallback: if the compiled library is missing, the first call raises.

Layouts follow the C ABI (include/gdn.h): q, k [B,T,H,dk]; v, o [B,T,H,dv];
g [B,T,H] (scalar gate) or [B,T,H,dk] (channel gate) fp32; beta [B,T,H] fp32;
states [B,H,dv,dk] fp32.
"""
from __future__ import annotations

import ctypes
import os
import threading

try:  # needed by every call, though not to build the library
    import torch
except ImportError:
    torch = None
else:
    # the current device and a device's current stream handle, by the short way where torch has it
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream",
                             lambda index: torch.cuda.current_stream(index).cuda_stream)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA, \
    GDN_ERR_DEVICE_TIMEOUT = range(6)
GDN_BF16, GDN_F32 = 0, 1
GDN_GATE_SCALAR, GDN_GATE_CHANNEL = 0, 1

# Every symbol include/gdn.h declares.
EXPORTS = ("gdn_chunk_fwd_workspace", "gdn_chunk_fwd", "gdn_chunk_bwd_workspace",
           "gdn_chunk_bwd", "gdn_chunk_fwd_save", "gdn_chunk_bwd_saved",
           "gdn_chunk_conv_saved_workspace", "gdn_chunk_fwd_save_conv", "gdn_chunk_bwd_saved_conv", "gdn_recurrent_step", "gdn_query_device_status",
           "gdn_status_string", "gdn_profile_begin", "gdn_profile_end",
           "gdn_chunk_fwd_noalloc", "gdn_noalloc_device_status", "gdn_test_stalled_fwd", "gdn_product_fwd_workspace", "gdn_product_fwd",
           "gdn_product_bwd_workspace", "gdn_product_bwd", "gdn_chunk_fwd_varlen_workspace",
           "gdn_chunk_fwd_varlen", "gdn_chunk_bwd_varlen_workspace", "gdn_chunk_bwd_varlen",
           "gdn_tree_verify", "gdn_tree_commit", "gdn_short_conv_fwd",
           "gdn_short_conv_bwd_workspace", "gdn_short_conv_bwd",
           "gdn_decay_fwd_workspace", "gdn_decay_fwd", "gdn_decay_bwd_workspace",
           "gdn_decay_bwd", "gdn_decay_step", "gdn_tree_attn_workspace", "gdn_tree_attn",
           "gdn_tree_append", "gdn_gated_norm_fwd", "gdn_gated_norm_bwd_workspace",
           "gdn_gated_norm_bwd")


class gdn_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
                ("dtype", ctypes.c_int), ("gate", ctypes.c_int), ("scale", ctypes.c_float)]


class gdn_decay_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("Hk", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgdn.so with argument types set.  Raises if it is absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m gated_delta_rule_153_b200.build` (nvcc, sm_100a)")
            L = ctypes.CDLL(LIB_PATH)
            vp, fp, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
            dp = ctypes.POINTER(gdn_dims)
            i, f = ctypes.c_int, ctypes.c_float
            L.gdn_chunk_fwd_workspace.argtypes = [dp]
            L.gdn_chunk_fwd_workspace.restype = sz
            L.gdn_chunk_bwd_workspace.argtypes = [dp]
            L.gdn_chunk_bwd_workspace.restype = sz
            L.gdn_chunk_fwd.argtypes = [dp, vp, vp, vp, fp, fp, fp, vp, fp, vp, sz, vp]
            L.gdn_chunk_fwd.restype = i
            L.gdn_chunk_bwd.argtypes = [dp, vp, vp, vp, fp, fp, fp, vp, fp, vp, vp, vp,
                                        fp, fp, fp, vp, sz, vp]
            L.gdn_chunk_bwd.restype = i
            L.gdn_chunk_fwd_save.argtypes = L.gdn_chunk_fwd.argtypes
            L.gdn_chunk_fwd_save.restype = i
            L.gdn_chunk_bwd_saved.argtypes = L.gdn_chunk_bwd.argtypes
            L.gdn_chunk_bwd_saved.restype = i
            L.gdn_chunk_conv_saved_workspace.argtypes = [dp, i]
            L.gdn_chunk_conv_saved_workspace.restype = sz
            L.gdn_chunk_fwd_save_conv.argtypes = [dp, i, vp, vp, vp, fp, fp, fp, fp, fp, fp, vp, fp,
                                                  vp, sz, vp]
            L.gdn_chunk_fwd_save_conv.restype = i
            L.gdn_chunk_bwd_saved_conv.argtypes = [dp, i, vp, vp, vp, fp, fp, fp, fp, fp, fp, vp, fp,
                                                   vp, vp, vp, fp, fp, fp, fp, fp, fp, vp, sz, vp]
            L.gdn_chunk_bwd_saved_conv.restype = i
            L.gdn_recurrent_step.argtypes = [i, i, i, i, i, i, f, vp, vp, vp, fp, fp, fp,
                                             vp, vp]
            L.gdn_recurrent_step.restype = i
            L.gdn_query_device_status.argtypes = [vp, vp]
            L.gdn_query_device_status.restype = i
            L.gdn_chunk_fwd_noalloc.argtypes = [dp, vp, vp, vp, fp, fp, fp, vp, fp, vp]
            L.gdn_chunk_fwd_noalloc.restype = i
            L.gdn_test_stalled_fwd.argtypes = [dp, vp, vp, vp, fp, fp, fp, vp, fp, vp, sz, i,
                                               ctypes.c_ulonglong, vp]
            L.gdn_test_stalled_fwd.restype = i
            L.gdn_noalloc_device_status.argtypes = [vp]
            L.gdn_noalloc_device_status.restype = i
            L.gdn_product_fwd_workspace.argtypes = [dp, i]
            L.gdn_product_fwd_workspace.restype = sz
            L.gdn_product_bwd_workspace.argtypes = [dp, i]
            L.gdn_product_bwd_workspace.restype = sz
            L.gdn_product_fwd.argtypes = [dp, i, vp, vp, vp, fp, fp, fp, vp, fp, vp, sz, vp]
            L.gdn_product_fwd.restype = i
            L.gdn_product_bwd.argtypes = [dp, i, vp, vp, vp, fp, fp, fp, vp, fp, vp, vp, vp,
                                          fp, fp, fp, vp, sz, vp]
            L.gdn_product_bwd.restype = i
            L.gdn_chunk_fwd_varlen_workspace.argtypes = [dp, i]
            L.gdn_chunk_fwd_varlen_workspace.restype = sz
            L.gdn_chunk_bwd_varlen_workspace.argtypes = [dp, i]
            L.gdn_chunk_bwd_varlen_workspace.restype = sz
            L.gdn_chunk_fwd_varlen.argtypes = [dp, vp, i, vp, vp, vp, fp, fp, fp, vp, fp, vp,
                                               sz, vp]
            L.gdn_chunk_fwd_varlen.restype = i
            L.gdn_chunk_bwd_varlen.argtypes = [dp, vp, i, vp, vp, vp, fp, fp, fp, vp, fp, vp,
                                               vp, vp, fp, fp, fp, vp, sz, vp]
            L.gdn_chunk_bwd_varlen.restype = i
            L.gdn_tree_verify.argtypes = [i, i, i, i, i, i, i, f, vp, vp, vp, vp, fp, fp, fp,
                                          vp, vp, vp]
            L.gdn_tree_verify.restype = i
            L.gdn_tree_commit.argtypes = [i, i, i, i, i, i, i, vp, vp, vp, vp, fp, fp, fp, vp,
                                          vp]
            L.gdn_tree_commit.restype = i
            L.gdn_short_conv_fwd.argtypes = [i, i, i, i, i, i, i, vp, fp, vp, vp]
            L.gdn_short_conv_fwd.restype = i
            L.gdn_short_conv_bwd_workspace.argtypes = [i, i, i, i, i]
            L.gdn_short_conv_bwd_workspace.restype = sz
            L.gdn_short_conv_bwd.argtypes = [i, i, i, i, i, i, i, vp, fp, vp, vp, fp, vp, sz, vp]
            L.gdn_short_conv_bwd.restype = i
            dd, ll = ctypes.POINTER(gdn_decay_dims), ctypes.c_longlong
            L.gdn_decay_fwd_workspace.argtypes = [dd, i]
            L.gdn_decay_fwd_workspace.restype = sz
            L.gdn_decay_fwd.argtypes = [dd, vp, i, vp, vp, vp, fp, fp, vp, fp, vp, sz, vp]
            L.gdn_decay_fwd.restype = i
            L.gdn_decay_bwd_workspace.argtypes = [dd, i]
            L.gdn_decay_bwd_workspace.restype = sz
            L.gdn_decay_bwd.argtypes = [dd, vp, i, vp, vp, vp, fp, fp, vp, fp, vp, vp, vp, fp, fp,
                                        vp, sz, vp]
            L.gdn_decay_bwd.restype = i
            L.gdn_decay_step.argtypes = [i, i, i, i, i, i, f, vp, vp, vp, fp, fp, vp, vp]
            L.gdn_decay_step.restype = i
            L.gdn_tree_attn_workspace.argtypes = [i, i, i, i, i, i, i, i]
            L.gdn_tree_attn_workspace.restype = sz
            L.gdn_tree_attn.argtypes = [i, i, i, i, i, i, f, i, vp, vp, vp, vp, i, i, i, vp, vp, vp,
                                        vp, vp, vp, sz, vp]
            L.gdn_tree_attn.restype = i
            L.gdn_tree_append.argtypes = [i, i, i, i, i, vp, vp, vp, vp, i, i, i, vp, vp, vp, vp,
                                          vp, vp, vp]
            L.gdn_tree_append.restype = i
            L.gdn_gated_norm_fwd.argtypes = [ll, i, i, i, i, i, f, vp, vp, fp, vp, vp]
            L.gdn_gated_norm_fwd.restype = i
            L.gdn_gated_norm_bwd_workspace.argtypes = [ll, i, i, i]
            L.gdn_gated_norm_bwd_workspace.restype = sz
            L.gdn_gated_norm_bwd.argtypes = [ll, i, i, i, i, i, f, vp, vp, fp, vp, vp, vp, fp, vp,
                                             sz, vp]
            L.gdn_gated_norm_bwd.restype = i
            L.gdn_profile_begin.argtypes = [i]
            L.gdn_profile_begin.restype = i
            L.gdn_profile_end.argtypes = [ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(ctypes.c_char_p), i]
            L.gdn_profile_end.restype = i
            L.gdn_status_string.argtypes = [i]
            L.gdn_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdn_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != GDN_OK:
        raise GdnError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t, name, dtype=None, shape=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def make_dims(q, v, g, chunk=64, scale=1.0) -> gdn_dims:
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    gate = GDN_GATE_CHANNEL if g.dim() == 4 else GDN_GATE_SCALAR
    return gdn_dims(B, T, H, dk, dv, int(chunk), _dtype_code(q), gate, float(scale))


def gdn_chunk_fwd_workspace(dims: gdn_dims) -> int:
    return int(lib().gdn_chunk_fwd_workspace(ctypes.byref(dims)))


def gdn_chunk_bwd_workspace(dims: gdn_dims) -> int:
    return int(lib().gdn_chunk_bwd_workspace(ctypes.byref(dims)))


def _validate_chunk_inputs(q, k, v, g, beta, h0):
    import torch
    _need(q, "q")
    B, T, H, dk = q.shape
    _need(k, "k", q.dtype, (B, T, H, dk))
    _need(v, "v", q.dtype)
    if v.shape[:3] != (B, T, H):
        raise ValueError("v must be [B,T,H,dv] matching q")
    dv = v.shape[3]
    _need(g, "g", torch.float32)
    if tuple(g.shape) not in ((B, T, H), (B, T, H, dk)):
        raise ValueError("g must be [B,T,H] or [B,T,H,dk]")
    _need(beta, "beta", torch.float32, (B, T, H))
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, H, dv, dk))
    return B, T, H, dk, dv


def _workspace(nbytes, device, workspace):
    import torch
    if nbytes == 0:
        return None
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, *, chunk=64, scale=1.0,
                  output_final_state=True, o=None, hT=None, workspace=None, stream=None):
    """Chunkwise forward.  Returns (o, hT); hT is None unless requested."""
    import torch
    B, T, H, dk, dv = _validate_chunk_inputs(q, k, v, g, beta, h0)
    dims = make_dims(q, v, g, chunk, scale)
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if output_final_state and hT is None:
        hT = torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device)
    nbytes = gdn_chunk_fwd_workspace(dims)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_chunk_fwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                             _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT), _ptr(ws),
                             nbytes if ws is None else ws.numel() * ws.element_size(),
                             _stream(stream))
    _check(st, "gdn_chunk_fwd")
    return o, hT


def gdn_chunk_bwd(q, k, v, g, beta, dO, h0=None, dhT=None, *, chunk=64, scale=1.0,
                  workspace=None, stream=None):
    """Chunkwise backward of <dO,o> + <dhT,hT>.  Returns a dict with dq, dk,
    dv (dtype of q), dg (shape of g), dbeta, dh0 (None when h0 is None)."""
    import torch
    B, T, H, dk, dv = _validate_chunk_inputs(q, k, v, g, beta, h0)
    _need(dO, "dO", q.dtype, (B, T, H, dv))
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (B, H, dv, dk))
    dims = make_dims(q, v, g, chunk, scale)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
               dh0=None if h0 is None else torch.empty_like(h0))
    nbytes = gdn_chunk_bwd_workspace(dims)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_chunk_bwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                             _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(out["dq"]),
                             _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                             _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws),
                             nbytes if ws is None else ws.numel() * ws.element_size(),
                             _stream(stream))
    _check(st, "gdn_chunk_bwd")
    return out


def gdn_chunk_saved_workspace(dims: gdn_dims) -> int:
    """Bytes of the workspace gdn_chunk_fwd_save fills and gdn_chunk_bwd_saved reads."""
    return max(gdn_chunk_bwd_workspace(dims), gdn_chunk_fwd_workspace(dims))


def gdn_chunk_fwd_save(q, k, v, g, beta, h0=None, *, chunk=64, scale=1.0,
                       output_final_state=True, o=None, hT=None, workspace=None, stream=None):
    """Forward of a training step.  Returns (o, hT, workspace): pass the
    workspace, and the same inputs, to gdn_chunk_bwd_saved."""
    import torch
    B, T, H, dk, dv = _validate_chunk_inputs(q, k, v, g, beta, h0)
    dims = make_dims(q, v, g, chunk, scale)
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if output_final_state and hT is None:
        hT = torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device)
    nbytes = gdn_chunk_saved_workspace(dims)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_chunk_fwd_save(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                  _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT), _ptr(ws),
                                  nbytes if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(st, "gdn_chunk_fwd_save")
    return o, hT, ws


def gdn_chunk_bwd_saved(q, k, v, g, beta, dO, workspace, h0=None, dhT=None, *, chunk=64,
                        scale=1.0, out=None, stream=None):
    """Backward from gdn_chunk_fwd_save's workspace; results as gdn_chunk_bwd.
    ``out``: optional dict of preallocated result tensors (dq, dk, dv, dg,
    dbeta, dh0), filled in place."""
    import torch
    B, T, H, dk, dv = _validate_chunk_inputs(q, k, v, g, beta, h0)
    _need(dO, "dO", q.dtype, (B, T, H, dv))
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (B, H, dv, dk))
    dims = make_dims(q, v, g, chunk, scale)
    if out is None:
        out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                   dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
                   dh0=None if h0 is None else torch.empty_like(h0))
    else:
        for n, ref in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
            _need(out[n], n, ref.dtype, tuple(ref.shape))
        if h0 is not None:
            _need(out["dh0"], "dh0", torch.float32, tuple(h0.shape))
    nbytes = gdn_chunk_saved_workspace(dims)
    if nbytes and (workspace is None or workspace.numel() * workspace.element_size() < nbytes):
        raise ValueError(f"workspace must be gdn_chunk_fwd_save's ({nbytes} bytes)")
    st = lib().gdn_chunk_bwd_saved(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                   _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(out["dq"]),
                                   _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                   _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(workspace),
                                   0 if workspace is None else workspace.numel() * workspace.element_size(),
                                   _stream(stream))
    _check(st, "gdn_chunk_bwd_saved")
    return out


def _validate_conv_chunk(xq, xk, xv, wq, wk, wv, g, beta, h0):
    import torch
    B, T, H, dk, dv = _validate_chunk_inputs(xq, xk, xv, g, beta, h0)
    K = wq.shape[-1] if wq.dim() == 3 else 0
    for w, name, d in ((wq, "wq", dk), (wk, "wk", dk), (wv, "wv", dv)):
        _need(w, name, torch.float32, (H, d, K))
    return B, T, H, dk, dv, K


def gdn_chunk_fwd_save_conv(xq, xk, xv, wq, wk, wv, g, beta, h0=None, *, chunk=64, scale=1.0,
                            output_final_state=True, o=None, hT=None, workspace=None, stream=None):
    """Forward of a training step from the raw projections: the short
    convolution, SiLU and (q, k) L2 norm, then the gated delta rule.  Returns
    (o, hT, workspace); pass the workspace to gdn_chunk_bwd_saved_conv."""
    import torch
    B, T, H, dk, dv, K = _validate_conv_chunk(xq, xk, xv, wq, wk, wv, g, beta, h0)
    dims = make_dims(xq, xv, g, chunk, scale)
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=xq.dtype, device=xq.device)
    if output_final_state and hT is None:
        hT = torch.empty(B, H, dv, dk, dtype=torch.float32, device=xq.device)
    nbytes = int(lib().gdn_chunk_conv_saved_workspace(ctypes.byref(dims), K))
    ws = _workspace(nbytes, xq.device, workspace)
    st = lib().gdn_chunk_fwd_save_conv(ctypes.byref(dims), K, _ptr(xq), _ptr(xk), _ptr(xv),
                                       _ptr(wq), _ptr(wk), _ptr(wv), _ptr(g), _ptr(beta), _ptr(h0),
                                       _ptr(o), _ptr(hT), _ptr(ws),
                                       0 if ws is None else ws.numel() * ws.element_size(),
                                       _stream(stream))
    _check(st, "gdn_chunk_fwd_save_conv")
    return o, hT, ws


def gdn_chunk_bwd_saved_conv(xq, xk, xv, wq, wk, wv, g, beta, dO, workspace, h0=None, dhT=None,
                             *, chunk=64, scale=1.0, stream=None):
    """Backward from gdn_chunk_fwd_save_conv's workspace.  Returns a dict with
    dxq, dxk, dxv, dwq, dwk, dwv, dg, dbeta, dh0."""
    import torch
    B, T, H, dk, dv, K = _validate_conv_chunk(xq, xk, xv, wq, wk, wv, g, beta, h0)
    _need(dO, "dO", xq.dtype, (B, T, H, dv))
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (B, H, dv, dk))
    dims = make_dims(xq, xv, g, chunk, scale)
    out = dict(dxq=torch.empty_like(xq), dxk=torch.empty_like(xk), dxv=torch.empty_like(xv),
               dwq=torch.empty_like(wq), dwk=torch.empty_like(wk), dwv=torch.empty_like(wv),
               dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
               dh0=None if h0 is None else torch.empty_like(h0))
    st = lib().gdn_chunk_bwd_saved_conv(
        ctypes.byref(dims), K, _ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(g),
        _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(out["dxq"]), _ptr(out["dxk"]),
        _ptr(out["dxv"]), _ptr(out["dwq"]), _ptr(out["dwk"]), _ptr(out["dwv"]), _ptr(out["dg"]),
        _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "gdn_chunk_bwd_saved_conv")
    return out


def gdn_recurrent_step(q, k, v, g, beta, state, *, scale=1.0, o=None, stream=None):
    """One decode token, in place on ``state`` [N,H,dv,dk] fp32.  q,k [N,H,dk];
    v [N,H,dv]; g [N,H] or [N,H,dk]; beta [N,H].  Returns o [N,H,dv]."""
    import torch
    _need(q, "q")
    N, H, dk = q.shape
    _need(k, "k", q.dtype, (N, H, dk))
    _need(v, "v", q.dtype)
    dv = v.shape[-1]
    _need(g, "g", torch.float32)
    gate = GDN_GATE_CHANNEL if g.dim() == 3 else GDN_GATE_SCALAR
    _need(beta, "beta", torch.float32, (N, H))
    _need(state, "state", torch.float32, (N, H, dv, dk))
    if o is None:
        o = torch.empty(N, H, dv, dtype=q.dtype, device=q.device)
    st = lib().gdn_recurrent_step(N, H, dk, dv, _dtype_code(q), gate, float(scale), _ptr(q),
                                  _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                  _ptr(o), _stream(stream))
    _check(st, "gdn_recurrent_step")
    return o


def gdn_profile_begin(capacity: int) -> None:
    """Start bracketing this thread's next ``capacity`` library launches with
    CUDA events (a profiling aid)."""
    _check(lib().gdn_profile_begin(int(capacity)), "gdn_profile_begin")


def gdn_profile_end(capacity: int):
    """Stop recording; returns (launch count, [(kernel name, ms), ...])."""
    ms = (ctypes.c_float * capacity)()
    names = (ctypes.c_char_p * capacity)()
    n = lib().gdn_profile_end(ms, names, int(capacity))
    if n < 0:
        raise RuntimeError("gdn_profile_end: recording was not on or a CUDA call failed")
    return n, [(names[i].decode(), float(ms[i])) for i in range(min(n, capacity))]


def gdn_query_device_status(workspace, stream=None) -> int:
    """Status word of the most recent chunkwise call that used ``workspace``."""
    return int(lib().gdn_query_device_status(_ptr(workspace), _stream(stream)))


# ---- gated DeltaProduct (n delta-rule steps per token) ---------------------
def _validate_product_inputs(q, k, v, g, beta, h0):
    import torch
    _need(q, "q")
    B, T, H, dk = q.shape
    if k.dim() != 5:
        raise ValueError("k must be [B,T,n,H,dk]")
    n = k.shape[2]
    _need(k, "k", q.dtype, (B, T, n, H, dk))
    _need(v, "v", q.dtype)
    if v.dim() != 5 or v.shape[:4] != (B, T, n, H):
        raise ValueError("v must be [B,T,n,H,dv] matching k")
    dv = v.shape[4]
    _need(g, "g", torch.float32)
    if tuple(g.shape) not in ((B, T, H), (B, T, H, dk)):
        raise ValueError("g must be [B,T,H] or [B,T,H,dk]")
    _need(beta, "beta", torch.float32, (B, T, n, H))
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, H, dv, dk))
    return B, T, n, H, dk, dv


def gdn_product_fwd(q, k, v, g, beta, h0=None, *, chunk=64, scale=1.0,
                    output_final_state=True, workspace=None, stream=None):
    """Gated DeltaProduct forward: k [B,T,n,H,dk], v [B,T,n,H,dv],
    beta [B,T,n,H]; q, g, h0 as for gdn_chunk_fwd.  Returns (o, hT)."""
    import torch
    B, T, n, H, dk, dv = _validate_product_inputs(q, k, v, g, beta, h0)
    dims = make_dims(q, v, g, chunk, scale)
    o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    hT = torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device) \
        if output_final_state else None
    nbytes = int(lib().gdn_product_fwd_workspace(ctypes.byref(dims), n))
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_product_fwd(ctypes.byref(dims), n, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                               _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT), _ptr(ws),
                               nbytes if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream))
    _check(st, "gdn_product_fwd")
    return o, hT


def gdn_product_bwd(q, k, v, g, beta, dO, h0=None, dhT=None, *, chunk=64, scale=1.0,
                    workspace=None, stream=None):
    """Gated DeltaProduct backward of <dO,o> + <dhT,hT>: gradients in the
    shapes of their primals (dh0 None when h0 is None)."""
    import torch
    B, T, n, H, dk, dv = _validate_product_inputs(q, k, v, g, beta, h0)
    _need(dO, "dO", q.dtype, (B, T, H, dv))
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (B, H, dv, dk))
    dims = make_dims(q, v, g, chunk, scale)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
               dh0=None if h0 is None else torch.empty_like(h0))
    nbytes = int(lib().gdn_product_bwd_workspace(ctypes.byref(dims), n))
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_product_bwd(ctypes.byref(dims), n, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                               _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dhT), _ptr(out["dq"]),
                               _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                               _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws),
                               nbytes if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream))
    _check(st, "gdn_product_bwd")
    return out


# ---- packed variable-length batches ----------------------------------------
def _validate_varlen(q, k, v, g, beta, cu_seqlens, h0):
    import torch
    B, T, H, dk, dv = _validate_chunk_inputs(q, k, v, g, beta, None)
    if B != 1:
        raise ValueError("packed sequences take q [1, total_tokens, H, dk]")
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [nseq + 1] int32")
    nseq = cu_seqlens.numel() - 1
    if h0 is not None:
        _need(h0, "h0", torch.float32, (nseq, H, dv, dk))
    return nseq, T, H, dk, dv


def gdn_chunk_fwd_varlen(q, k, v, g, beta, cu_seqlens, h0=None, *, scale=1.0,
                         output_final_state=True, workspace=None, stream=None):
    """Chunkwise forward over packed sequences: q [1,T,H,dk] etc. hold nseq
    sequences back to back, sequence s at tokens cu_seqlens[s]..cu_seqlens[s+1]-1
    (cu_seqlens int32 on the device).  h0 / hT are [nseq,H,dv,dk].  Returns
    (o, hT)."""
    import torch
    nseq, T, H, dk, dv = _validate_varlen(q, k, v, g, beta, cu_seqlens, h0)
    dims = make_dims(q, v, g, 64, scale)
    o = torch.empty(1, T, H, dv, dtype=q.dtype, device=q.device)
    hT = torch.empty(nseq, H, dv, dk, dtype=torch.float32, device=q.device) \
        if output_final_state else None
    nbytes = int(lib().gdn_chunk_fwd_varlen_workspace(ctypes.byref(dims), nseq))
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_chunk_fwd_varlen(ctypes.byref(dims), _ptr(cu_seqlens), nseq, _ptr(q),
                                    _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
                                    _ptr(hT), _ptr(ws),
                                    nbytes if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream))
    _check(st, "gdn_chunk_fwd_varlen")
    return o, hT


def gdn_chunk_bwd_varlen(q, k, v, g, beta, cu_seqlens, dO, h0=None, dhT=None, *, scale=1.0,
                         workspace=None, stream=None):
    """Backward of gdn_chunk_fwd_varlen: gradients in the shapes of their
    primals (dh0 None when h0 is None)."""
    import torch
    nseq, T, H, dk, dv = _validate_varlen(q, k, v, g, beta, cu_seqlens, h0)
    _need(dO, "dO", q.dtype, (1, T, H, dv))
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (nseq, H, dv, dk))
    dims = make_dims(q, v, g, 64, scale)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
               dh0=None if h0 is None else torch.empty_like(h0))
    nbytes = int(lib().gdn_chunk_bwd_varlen_workspace(ctypes.byref(dims), nseq))
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().gdn_chunk_bwd_varlen(ctypes.byref(dims), _ptr(cu_seqlens), nseq, _ptr(q),
                                    _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(dO),
                                    _ptr(dhT), _ptr(out["dq"]), _ptr(out["dk"]),
                                    _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]),
                                    _ptr(out["dh0"]), _ptr(ws),
                                    nbytes if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream))
    _check(st, "gdn_chunk_bwd_varlen")
    return out


# ---- draft-tree verification and commit ------------------------------------
def _validate_tree(parent, k, v, g, beta, state):
    import torch
    _need(parent, "parent", torch.int32)
    if parent.dim() != 2:
        raise ValueError("parent must be [N, M] int32")
    N, M = parent.shape
    _need(k, "k")
    if k.dim() != 4 or tuple(k.shape[:2]) != (N, M):
        raise ValueError("k must be [N, M, H, dk]")
    H, dk = k.shape[2], k.shape[3]
    _need(v, "v", k.dtype)
    if v.dim() != 4 or tuple(v.shape[:3]) != (N, M, H):
        raise ValueError("v must be [N, M, H, dv]")
    dv = v.shape[3]
    gate = GDN_GATE_CHANNEL if g.dim() == 4 else GDN_GATE_SCALAR
    _need(g, "g", torch.float32)
    if tuple(g.shape[:3]) != (N, M, H):
        raise ValueError("g must be [N, M, H]")
    _need(beta, "beta", torch.float32, (N, M, H))
    _need(state, "state", torch.float32, (N, H, dv, dk))
    return N, M, H, dk, dv, gate


def gdn_tree_verify(parent, q, k, v, g, beta, state, *, scale=1.0, o=None, status=None,
                    stream=None):
    """Outputs of every draft-tree node: o [N,M,H,dv], node i read out after
    the tokens of its root path, from ``state`` [N,H,dv,dk] (not modified)."""
    import torch
    N, M, H, dk, dv, gate = _validate_tree(parent, k, v, g, beta, state)
    _need(q, "q", k.dtype, tuple(k.shape))
    if o is None:
        o = torch.empty(N, M, H, dv, dtype=q.dtype, device=q.device)
    st = lib().gdn_tree_verify(N, M, H, dk, dv, _dtype_code(q), gate, float(scale),
                               _ptr(parent), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                               _ptr(state), _ptr(o), _ptr(status), _stream(stream))
    _check(st, "gdn_tree_verify")
    return o


def gdn_tree_commit(parent, accepted, k, v, g, beta, state, *, status=None, stream=None):
    """In place on ``state``: the state after the root path of node
    accepted[n] (int32 [N]; -1 leaves state[n] as it is)."""
    import torch
    N, M, H, dk, dv, gate = _validate_tree(parent, k, v, g, beta, state)
    _need(accepted, "accepted", torch.int32, (N,))
    st = lib().gdn_tree_commit(N, M, H, dk, dv, _dtype_code(k), gate, _ptr(parent),
                               _ptr(accepted), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                               _ptr(state), _ptr(status), _stream(stream))
    _check(st, "gdn_tree_commit")
    return state


# ---- q/k/v prologue: short causal convolution, SiLU, L2 norm ---------------
def _validate_conv(x, w):
    import torch
    _need(x, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, d]")
    B, T, H, d = x.shape
    _need(w, "w", torch.float32)
    if w.dim() != 3 or tuple(w.shape[:2]) != (H, d):
        raise ValueError("w must be [H, d, K] fp32")
    return B, T, H, d, w.shape[2]


def gdn_short_conv_fwd(x, w, *, l2norm=True, y=None, stream=None):
    """y = (L2-normalised) SiLU(causal depthwise conv of x with w): x
    [B,T,H,d] bf16/fp32, w [H,d,K] fp32.  Returns y (shape and dtype of x)."""
    import torch
    B, T, H, d, K = _validate_conv(x, w)
    if y is None:
        y = torch.empty_like(x)
    st = lib().gdn_short_conv_fwd(B, T, H, d, K, _dtype_code(x), int(bool(l2norm)), _ptr(x),
                                  _ptr(w), _ptr(y), _stream(stream))
    _check(st, "gdn_short_conv_fwd")
    return y


def gdn_short_conv_bwd(x, w, dy, *, l2norm=True, workspace=None, stream=None):
    """Gradients of <dy, y> for gdn_short_conv_fwd: returns (dx, dw)."""
    import torch
    B, T, H, d, K = _validate_conv(x, w)
    _need(dy, "dy", x.dtype, tuple(x.shape))
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    nbytes = int(lib().gdn_short_conv_bwd_workspace(B, T, H, d, K))
    ws = _workspace(nbytes, x.device, workspace)
    st = lib().gdn_short_conv_bwd(B, T, H, d, K, _dtype_code(x), int(bool(l2norm)), _ptr(x),
                                  _ptr(w), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(ws),
                                  nbytes if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(st, "gdn_short_conv_bwd")
    return dx, dw


# ---- linear attention with a decay per head ----------------------------------
class _On:
    """The device of a call's tensors and, when the caller names a stream, that
    stream: what the call allocates then belongs to the stream it runs on.
    Entering gives the stream's handle; where device and stream are the current
    ones that is all it does."""

    def __init__(self, device, stream):
        self.ctx, self.handle = None, None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream of {stream.device} for tensors on {device}")
            self.ctx, self.handle = torch.cuda.stream(stream), stream.cuda_stream  # sets its device too
        else:
            if device.index != _current_device():
                self.ctx = torch.cuda.device(device)
            self.handle = _stream_handle(device.index)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _want(t, name, dtype, shape, device):
    """A contiguous CUDA tensor of this dtype and shape on this device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


_CODES = {}  # torch dtypes of q, k, v and the like, filled on first use
_INT = 2 ** 31 - 1  # the library's sizes are C ints, and ctypes would drop the higher bits


def _int(n, name):
    """A size that fits a C int."""
    if n > _INT:
        raise ValueError(f"{name} = {n} is more than {_INT}")
    return n


def _lead(t, name, dims):
    """The first tensor of a call: (dtype code, device, shape)."""
    try:
        code, shape = _CODES[t.dtype], t.shape
        if len(shape) == dims and t.is_cuda and t.is_contiguous() and max(shape) <= _INT:
            return code, t.device, shape
    except (KeyError, AttributeError):
        pass
    _need(t, name)
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    _int(max(t.shape), f"a size of {name}")
    _CODES[t.dtype] = _dtype_code(t)
    return _CODES[t.dtype], t.device, t.shape


def _given(t, name, shape, dtype, device):
    """``t`` checked as an output, or a new tensor when it is None."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(t, name, dtype, shape, device)
    return t


def _like(t, name, ref):
    """``t`` checked as an output of ``ref``'s kind, or a new one."""
    if t is None:
        return torch.empty_like(ref)
    _want(t, name, ref.dtype, ref.shape, ref.device)
    return t


def _at(t):
    return None if t is None else t.data_ptr()


def _nbytes(t):
    return t.numel() * t.element_size()


def _scratch(nbytes, device, workspace):
    """The caller's workspace, checked, or a new one."""
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device:
        raise TypeError(f"workspace must be a tensor on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if _nbytes(workspace) < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace


def _decay_inputs(q, k, v, g, h0, cu_seqlens, scale):
    code, dev, (B, T, Hk, dk) = _lead(q, "q", 4)
    _want(k, "k", q.dtype, q.shape, dev)
    _, vdev, (Bv, Tv, H, dv) = _lead(v, "v", 4)
    if Bv != B or Tv != T or v.dtype is not q.dtype or vdev != dev:
        raise ValueError(f"v must be {q.dtype} [B, T, H, dv] matching q, on {dev}")
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} value heads cannot share {Hk} key heads")
    _want(g, "g", torch.float32, (B, T, H), dev)
    nseq = 0
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2 or cu_seqlens.device != dev:
            raise ValueError(f"cu_seqlens must be [nseq + 1] int32 on {dev}")
        if B != 1:
            raise ValueError("packed sequences take q [1, total_tokens, Hk, dk]")
        nseq = _int(cu_seqlens.shape[0] - 1, "nseq")
    states = (nseq or B, H, dv, dk)
    if h0 is not None:
        _want(h0, "h0", torch.float32, states, dev)
    return gdn_decay_dims(B, T, H, Hk, dk, dv, code, scale), nseq, states


def gdn_decay_fwd_workspace(dims: gdn_decay_dims, nseq: int = 0) -> int:
    return lib().gdn_decay_fwd_workspace(dims, nseq)


def gdn_decay_bwd_workspace(dims: gdn_decay_dims, nseq: int = 0) -> int:
    return lib().gdn_decay_bwd_workspace(dims, nseq)


def gdn_decay_fwd(q, k, v, g, h0=None, *, cu_seqlens=None, scale=1.0, output_final_state=True,
                  o=None, hT=None, workspace=None, stream=None):
    """Linear attention S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t (scale q_t):
    q, k [B,T,Hk,dk]; v [B,T,H,dv] (Hk divides H); g [B,T,H] fp32; h0
    [B,H,dv,dk] fp32.  With ``cu_seqlens`` (int32 on the device) B is 1, the row
    holds packed sequences and the states are [nseq,H,dv,dk].  Returns (o, hT);
    hT is None unless requested."""
    dims, nseq, states = _decay_inputs(q, k, v, g, h0, cu_seqlens, scale)
    dev = q.device
    with _On(dev, stream) as s:
        o = _like(o, "o", v)
        if output_final_state or hT is not None:
            hT = _given(hT, "hT", states, torch.float32, dev)
        ws = _scratch(gdn_decay_fwd_workspace(dims, nseq), dev, workspace)
        st = lib().gdn_decay_fwd(dims, _at(cu_seqlens), nseq, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                 g.data_ptr(), _at(h0), o.data_ptr(), _at(hT), ws.data_ptr(),
                                 _nbytes(ws), s)
    _check(st, "gdn_decay_fwd")
    return o, hT


def gdn_decay_bwd(q, k, v, g, dO, h0=None, dhT=None, *, cu_seqlens=None, scale=1.0, out=None,
                  workspace=None, stream=None):
    """Backward of <dO,o> + <dhT,hT> for gdn_decay_fwd.  Returns a dict with dq,
    dk, dv (dtype of q), dg, dh0 (None when h0 is None).  ``out``: optional dict
    of preallocated results, filled in place."""
    dims, nseq, states = _decay_inputs(q, k, v, g, h0, cu_seqlens, scale)
    dev = q.device
    _want(dO, "dO", q.dtype, v.shape, dev)
    if dhT is not None:
        _want(dhT, "dhT", torch.float32, states, dev)
    with _On(dev, stream) as s:
        out = {} if out is None else dict(out)
        for n, ref in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dh0", h0)):
            out[n] = None if ref is None else _like(out.get(n), n, ref)
        ws = _scratch(gdn_decay_bwd_workspace(dims, nseq), dev, workspace)
        st = lib().gdn_decay_bwd(dims, _at(cu_seqlens), nseq, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                 g.data_ptr(), _at(h0), dO.data_ptr(), _at(dhT), out["dq"].data_ptr(),
                                 out["dk"].data_ptr(), out["dv"].data_ptr(), out["dg"].data_ptr(),
                                 _at(out["dh0"]), ws.data_ptr(), _nbytes(ws), s)
    _check(st, "gdn_decay_bwd")
    return out


def gdn_decay_step(q, k, v, g, state, *, scale=1.0, o=None, stream=None):
    """One decode token of gdn_decay_fwd's recurrence, in place on ``state``
    [N,H,dv,dk] fp32: q, k [N,Hk,dk]; v [N,H,dv]; g [N,H] fp32.  Returns o."""
    code, dev, (N, Hk, dk) = _lead(q, "q", 3)
    _want(k, "k", q.dtype, q.shape, dev)
    _, vdev, (Nv, H, dv) = _lead(v, "v", 3)
    if Nv != N or v.dtype is not q.dtype or vdev != dev:
        raise ValueError(f"v must be {q.dtype} [N, H, dv] matching q, on {dev}")
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} value heads cannot share {Hk} key heads")
    _want(g, "g", torch.float32, (N, H), dev)
    _want(state, "state", torch.float32, (N, H, dv, dk), dev)
    with _On(dev, stream) as s:
        o = _like(o, "o", v)
        st = lib().gdn_decay_step(N, H, Hk, dk, dv, code, scale, q.data_ptr(), k.data_ptr(),
                                  v.data_ptr(), g.data_ptr(), state.data_ptr(), o.data_ptr(), s)
    _check(st, "gdn_decay_step")
    return o


# ---- draft-tree attention over a paged cache ---------------------------------
def _tree_cache(parent, k, v, k_cache, v_cache, block_table, cache_len):
    code, dev, (N, M, Hkv, d) = _lead(k, "k", 4)
    _want(parent, "parent", torch.int32, (N, M), dev)
    _want(v, "v", k.dtype, k.shape, dev)
    _, cdev, (pages, page, Hc, dc) = _lead(k_cache, "k_cache", 4)
    if Hc != Hkv or dc != d or k_cache.dtype is not k.dtype or cdev != dev:
        raise ValueError(f"k_cache must be {k.dtype} [pages, page, Hkv, d] on {dev}")
    _want(v_cache, "v_cache", k.dtype, k_cache.shape, dev)
    width = block_table.shape[-1] if isinstance(block_table, torch.Tensor) and block_table.dim() == 2 else 0
    _want(block_table, "block_table", torch.int32, (N, width), dev)
    _int(width, "block_table's width")
    _want(cache_len, "cache_len", torch.int32, (N,), dev)
    return code, dev, N, M, Hkv, d, pages, page, width


def gdn_tree_attn(parent, q, k, v, k_cache, v_cache, block_table, cache_len, *, scale=1.0, window=0,
                  o=None, workspace=None, stream=None):
    """Softmax attention of every draft-tree node over its sequence's cached
    tokens, its ancestors and itself: parent [N,M] int32; q [N,M,Hq,d]; k, v
    [N,M,Hkv,d]; k_cache, v_cache [pages,page,Hkv,d]; block_table [N,width] and
    cache_len [N] int32.  window > 0: only positions less than ``window`` back.
    Returns o [N,M,Hq,d]."""
    window = max(-1, min(window, _INT))  # no position is further back
    dt, dev, N, M, Hkv, d, pages, page, width = _tree_cache(parent, k, v, k_cache, v_cache, block_table,
                                                            cache_len)
    Hq = _int(q.shape[2], "Hq") if isinstance(q, torch.Tensor) and q.dim() == 4 else 0
    _want(q, "q", k.dtype, (N, M, Hq, d), dev)
    with _On(dev, stream) as s:
        o = _like(o, "o", q)
        ws = _scratch(lib().gdn_tree_attn_workspace(N, M, Hq, Hkv, d, dt, page, width), dev, workspace)
        st = lib().gdn_tree_attn(N, M, Hq, Hkv, d, dt, scale, window, parent.data_ptr(), q.data_ptr(),
                                 k.data_ptr(), v.data_ptr(), pages, page, width, k_cache.data_ptr(),
                                 v_cache.data_ptr(), block_table.data_ptr(), cache_len.data_ptr(),
                                 o.data_ptr(), ws.data_ptr(), _nbytes(ws), s)
    _check(st, "gdn_tree_attn")
    return o


def gdn_tree_append(parent, accepted, k, v, k_cache, v_cache, block_table, cache_len, *, new_len=None,
                    status=None, stream=None):
    """Appends the k and v rows of the root path of node accepted[n] (int32 [N];
    -1: nothing) to sequence n's pages, in place on k_cache and v_cache.  Returns
    the new lengths (``new_len`` may be ``cache_len``)."""
    code, dev, N, M, Hkv, d, pages, page, width = _tree_cache(parent, k, v, k_cache, v_cache, block_table,
                                                              cache_len)
    _want(accepted, "accepted", torch.int32, (N,), dev)
    if status is not None:
        _need(status, "status", torch.int32)
        if status.numel() < 1 or status.device != dev:
            raise ValueError(f"status must hold a word on {dev}")
    with _On(dev, stream) as s:
        new_len = _like(new_len, "new_len", cache_len)
        st = lib().gdn_tree_append(N, M, Hkv, d, code, parent.data_ptr(), accepted.data_ptr(),
                                   k.data_ptr(), v.data_ptr(), pages, page, width, k_cache.data_ptr(),
                                   v_cache.data_ptr(), block_table.data_ptr(), cache_len.data_ptr(),
                                   new_len.data_ptr(), _at(status), s)
    _check(st, "gdn_tree_append")
    return new_len


# ---- output norm and gate ----------------------------------------------------
def _norm_inputs(x, z, w):
    _need(x, "x")
    if x.dim() < 2:
        raise ValueError("x must be [..., H, d]")
    H, d = _int(x.shape[-2], "H"), _int(x.shape[-1], "d")
    _want(z, "z", x.dtype, x.shape, x.device)
    shared = isinstance(w, torch.Tensor) and w.dim() == 1
    _want(w, "w", torch.float32, (d,) if shared else (H, d), x.device)
    return x.numel() // max(d, 1), H, d, 1 if shared else H


def gdn_gated_norm_fwd(x, z, w, *, eps=1e-6, center=False, y=None, stream=None):
    """y = w * norm(x) * SiLU(z), the norm over the last axis of x [...,H,d]: RMS,
    or mean and variance with ``center``; w [d] or [H,d] fp32."""
    rows, H, d, wheads = _norm_inputs(x, z, w)
    with _On(x.device, stream) as s:
        y = _like(y, "y", x)
        st = lib().gdn_gated_norm_fwd(rows, H, d, wheads, _dtype_code(x), bool(center), eps, x.data_ptr(),
                                      z.data_ptr(), w.data_ptr(), y.data_ptr(), s)
    _check(st, "gdn_gated_norm_fwd")
    return y


def gdn_gated_norm_bwd(x, z, w, dy, *, eps=1e-6, center=False, dx=None, dz=None, dw=None, workspace=None,
                       stream=None):
    """Gradients of <dy, y> for gdn_gated_norm_fwd: returns (dx, dz, dw)."""
    rows, H, d, wheads = _norm_inputs(x, z, w)
    dev, dt = x.device, _dtype_code(x)
    _want(dy, "dy", x.dtype, x.shape, dev)
    with _On(dev, stream) as s:
        dx = _like(dx, "dx", x)
        dz = _like(dz, "dz", x)
        dw = _like(dw, "dw", w)
        ws = _scratch(lib().gdn_gated_norm_bwd_workspace(rows, H, d, dt), dev, workspace)
        st = lib().gdn_gated_norm_bwd(rows, H, d, wheads, dt, bool(center), eps, x.data_ptr(), z.data_ptr(),
                                      w.data_ptr(), dy.data_ptr(), dx.data_ptr(), dz.data_ptr(),
                                      dw.data_ptr(), ws.data_ptr(), _nbytes(ws), s)
    _check(st, "gdn_gated_norm_bwd")
    return dx, dz, dw

"""Thin ctypes binding of libmhc_gb300.so (argument marshalling only).

Each function takes CUDA tensors, allocates the outputs with torch (device
memory is PyTorch's job here), and calls the C entry point of the same name on
the current torch stream.  Every step of the layer runs in the library's CUDA
kernels; there is no CPU path.  If the library is missing, the first call
raises: build it with ``python -m mhc_pre_gb300.build`` (or
``__graft_entry__.build()``).
"""

from __future__ import annotations

import ctypes
import os
from collections import namedtuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libmhc_gb300.so")

MHC_OK, MHC_ERR_INVALID_ARG, MHC_ERR_UNSUPPORTED = 0, 1, 2
MHC_ERR_MISALIGNED, MHC_ERR_CUDA, MHC_ERR_TIMEOUT = 3, 4, 5
MHC_ERR_RANGE = 6
MHC_F32, MHC_BF16 = 0, 1
MAX_ITERS = 64

EXPORTS = ("mhc_status_string", "mhc_version", "mhc_get_last_device_error",
           "mhc_pre", "mhc_post", "mhc_post_norm", "mhc_post_norm_bwd",
           "mhc_post_pre", "mhc_post_pre_workspace_bytes",
           "mhc_post_bwd", "mhc_kernel_launches",
           "mhc_pre_bwd_workspace_bytes", "mhc_pre_bwd", "mhc_pre_bwd_noalloc",
           "mhc_pre_gates", "mhc_layer_bwd_recompute_workspace_bytes",
           "mhc_layer_bwd_recompute", "mhc_test_force_timeout", "mhc_pre_critical",
           "mhc_post_res_gates",
           "mhc_qk_norm_rope", "mhc_qk_norm_rope_bwd", "mhc_qk_norm_rope_bwd_workspace_bytes",
           "mhc_qk_norm_rope_append", "mhc_paged_attn_plan", "mhc_paged_attn",
           "mhc_paged_attn_workspace_bytes")

PreOut = namedtuple("PreOut", "x_in H_pre H_post H_res proj inv_rms")
PostPreOut = namedtuple("PostPreOut", "x_next x_in H_pre H_post H_res proj inv_rms")
PostNormOut = namedtuple("PostNormOut", "x_next inv_rms_y inv_rms_out")
SANDWICH_NORM, BLOCK_NORM = 1, 2
PostBwdOut = namedtuple("PostBwdOut", "dx dy dH_post dH_res")
PreBwdOut = namedtuple("PreBwdOut", "dx dphi db dalpha")
PreGatesOut = namedtuple("PreGatesOut", "H_pre H_post H_res proj inv_rms")
PreCriticalOut = namedtuple("PreCriticalOut", "x_in H_pre proj inv_rms")
PostResGatesOut = namedtuple("PostResGatesOut", "H_post H_res")
LayerBwdOut = namedtuple("LayerBwdOut", "dx dy dphi db dalpha")
QKOut = namedtuple("QKOut", "q k")
QKBwdOut = namedtuple("QKBwdOut", "dq dk dw_q dw_k")
PagedAttnOut = namedtuple("PagedAttnOut", "o lse")
PagedAttnPlan = namedtuple("PagedAttnPlan", "workspace sizes")
ROPE_ADJACENT = 1

_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_SIGS = {
    "mhc_status_string": ([_I], ctypes.c_char_p),
    "mhc_version": ([], ctypes.c_char_p),
    "mhc_get_last_device_error": ([_P], _I),
    "mhc_pre": ([_I, _P, _P, _P, _P, _I64, _I, _I64, _I, _F,
                 _P, _P, _P, _P, _P, _P, _P], _I),
    "mhc_post": ([_I, _P, _P, _P, _P, _I64, _I, _I64, _P, _P], _I),
    "mhc_post_pre": ([_I, _P, _P, _P, _P, _P, _P, _P, _I64, _I, _I64, _I, _F,
                      _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], _I),
    "mhc_post_pre_workspace_bytes": ([_I, _I64, _I, _I64], ctypes.c_size_t),
    "mhc_post_norm": ([_I, _P, _P, _P, _P, _I, _F, _I64, _I, _I64, _P, _P, _P, _P], _I),
    "mhc_post_norm_bwd": ([_I, _P, _P, _P, _P, _P, _I, _F, _P, _P, _I64, _I, _I64,
                           _P, _P, _P, _P, _P], _I),
    "mhc_post_bwd": ([_I, _P, _P, _P, _P, _P, _I64, _I, _I64,
                      _P, _P, _P, _P, _P], _I),
    "mhc_kernel_launches": ([ctypes.c_char_p, _I, _I64, _I, _I64], _I),
    "mhc_pre_bwd_workspace_bytes": ([_I, _I64, _I, _I64], ctypes.c_size_t),
    "mhc_pre_bwd": ([_I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I, _I64,
                     _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], _I),
    "mhc_pre_bwd_noalloc": ([_I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I,
                             _I64, _I, _P, _P, _P, _P, _P], _I),
    "mhc_pre_gates": ([_I, _P, _P, _P, _P, _I64, _I, _I64, _I, _F,
                       _P, _P, _P, _P, _P, _P], _I),
    "mhc_layer_bwd_recompute_workspace_bytes": ([_I, _I64, _I, _I64], ctypes.c_size_t),
    "mhc_test_force_timeout": ([_I], _I),
    "mhc_pre_critical": ([_I, _P, _P, _P, _P, _I64, _I, _I64, _F, _P, _P, _P, _P, _P], _I),
    "mhc_post_res_gates": ([_P, _P, _P, _I64, _I, _I, _P, _P, _P], _I),
    "mhc_layer_bwd_recompute": ([_I, _P, _P, _P, _P, _P, _P, _P, _I64, _I, _I64, _I, _F,
                                 _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], _I),
    "mhc_qk_norm_rope": ([_I, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I, _I, _I, _I, _I, _F,
                          _P, _I64, _P, _I64, _P], _I),
    "mhc_qk_norm_rope_bwd": ([_I, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64,
                              _I, _I, _I, _I, _I, _F, _P, _I64, _P, _I64, _P, _P, _P, ctypes.c_size_t,
                              _P], _I),
    "mhc_qk_norm_rope_bwd_workspace_bytes": ([_I64, _I], ctypes.c_size_t),
    "mhc_qk_norm_rope_append": ([_I, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _I64,
                                 _I, _I, _I, _I, _I, _F, _P, _I64, _P, _I64, _I64, _I64,
                                 _P, _I64, _I64, _I64, _I64, _I, _P], _I),
    "mhc_paged_attn_plan": ([_I, _P, _P, _I64, _I, _I, _I, _I, _I, _I64, _I64, _I, _P,
                             ctypes.c_size_t, _P], _I),
    "mhc_paged_attn": ([_I, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I,
                        _P, _I64, _P, _P, _I64, _I, _I, _I, _I, _I64, _I64, _I, _F, _F, _P, _P,
                        _P, ctypes.c_size_t, _P], _I),
    "mhc_paged_attn_workspace_bytes": ([_I, _I64, _I, _I, _I, _I, _I, _I64], ctypes.c_size_t),
}

_lib = None


def _empty(shape, dtype=None, device=None):
    """Allocates every output and workspace buffer this module hands to the
    library.  Plain torch.empty; the guard-band tests put an allocator that
    surrounds each buffer with sentinel bytes in its place."""
    return torch.empty(shape, dtype=dtype, device=device)


_torch_empty = _empty


class MhcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads the library once and declares every exported signature."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: the mHC layer has no CPU path; build the "
            "CUDA library with `python -m mhc_pre_gb300.build`")
    handle = ctypes.CDLL(path)
    for name, (args, res) in _SIGS.items():
        fn = getattr(handle, name)
        fn.argtypes = args
        fn.restype = res
    if path == LIB_PATH:
        _lib = handle
    return handle


def status_string(status: int) -> str:
    return lib().mhc_status_string(status).decode()


def version() -> str:
    return lib().mhc_version().decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MHC_BF16
    if t.dtype == torch.float32:
        return MHC_F32
    raise TypeError(f"activations must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("the mHC library takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("the mHC library takes contiguous tensors only")
    return t.data_ptr()


def _stream(dev) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _check(status: int, where: str):
    if status != MHC_OK:
        raise MhcError(status, where)


def _f32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    return t


def mhc_pre(x, phi, b, alpha, iters: int = 20, eps: float = 1e-6):
    """Forward of the read side.  x [T, n, D] (bf16 or f32, CUDA)."""
    T, n, D = x.shape
    G = 2 * n + n * n
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PreOut(_empty((T, D), dtype=x.dtype, device=x.device),
                 _empty((T, n), **f32), _empty((T, n), **f32),
                 _empty((T, n, n), **f32), _empty((T, G), **f32),
                 _empty((T,), **f32))
    st = lib().mhc_pre(_dtype_code(x), _ptr(x), _ptr(_f32(phi, "phi")),
                       _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")), T, n, D,
                       iters, eps, *[_ptr(o) for o in out], _stream(x.device))
    _check(st, "mhc_pre")
    return out


def mhc_pre_gates(x, phi, b, alpha, iters: int = 20, eps: float = 1e-6):
    """mhc_pre without the H_pre mix (no x_in): the gates and the saved state,
    bit for bit as mhc_pre writes them."""
    T, n, D = x.shape
    G = 2 * n + n * n
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PreGatesOut(_empty((T, n), **f32), _empty((T, n), **f32),
                      _empty((T, n, n), **f32), _empty((T, G), **f32),
                      _empty((T,), **f32))
    st = lib().mhc_pre_gates(_dtype_code(x), _ptr(x), _ptr(_f32(phi, "phi")),
                             _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")), T, n, D,
                             iters, eps, *[_ptr(o) for o in out], _stream(x.device))
    _check(st, "mhc_pre_gates")
    return out


def layer_bwd_recompute_workspace_bytes(dtype, T: int, n: int, D: int) -> int:
    code = MHC_BF16 if dtype == torch.bfloat16 else MHC_F32
    return int(lib().mhc_layer_bwd_recompute_workspace_bytes(code, T, n, D))


def mhc_pre_critical(x, phi, b, alpha, eps: float = 1e-6, stream=None):
    """The inference critical path of mhc_pre: x_in, H_pre, proj, inv_rms (no
    Sinkhorn).  ``stream``: a torch.cuda.Stream (default: the current one)."""
    T, n, D = x.shape
    G = 2 * n + n * n
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PreCriticalOut(_empty((T, D), dtype=x.dtype, device=x.device), _empty((T, n), **f32),
                         _empty((T, G), **f32), _empty((T,), **f32))
    s = stream.cuda_stream if stream is not None else _stream(x.device)
    st = lib().mhc_pre_critical(_dtype_code(x), _ptr(x), _ptr(_f32(phi, "phi")), _ptr(_f32(b, "b")),
                                _ptr(_f32(alpha, "alpha")), T, n, D, eps, *[_ptr(o) for o in out], s)
    _check(st, "mhc_pre_critical")
    return out


def mhc_post_res_gates(proj, b, alpha, iters: int = 20, stream=None):
    """H_post and H_res from a saved projection (the side of the critical-path
    split).  ``stream``: a torch.cuda.Stream (default: the current one)."""
    T, G = proj.shape
    n = 4
    f32 = dict(dtype=torch.float32, device=proj.device)
    out = PostResGatesOut(_empty((T, n), **f32), _empty((T, n, n), **f32))
    s = stream.cuda_stream if stream is not None else _stream(proj.device)
    st = lib().mhc_post_res_gates(_ptr(_f32(proj, "proj")), _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")),
                                  T, n, iters, *[_ptr(o) for o in out], s)
    _check(st, "mhc_post_res_gates")
    return out


def mhc_layer_bwd_recompute(g_in, g_next, x, y, phi, b, alpha, iters: int = 20,
                            eps: float = 1e-6, workspace=None):
    """The layer's backward from its inputs x and y alone (the gates and the
    saved state recomputed).  Returns dx, dy, dphi, db, dalpha."""
    T, n, D = x.shape
    G = 2 * n + n * n
    if not (g_in.dtype == g_next.dtype == x.dtype == y.dtype):
        raise TypeError("g_in, g_next, x and y must share a dtype")
    need = layer_bwd_recompute_workspace_bytes(x.dtype, T, n, D)
    if workspace is None:
        workspace = _empty((max(need, 16),), dtype=torch.uint8, device=x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    dx = _empty(x.shape, x.dtype, x.device)
    dy = _empty(y.shape, y.dtype, y.device)
    dphi = _empty((n * D, G), **f32)
    db = _empty((G,), **f32)
    dalpha = _empty((3,), **f32)
    st = lib().mhc_layer_bwd_recompute(
        _dtype_code(x), _ptr(g_in), _ptr(g_next), _ptr(x), _ptr(y), _ptr(_f32(phi, "phi")),
        _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")), T, n, D, iters, eps, _ptr(dx), _ptr(dy),
        _ptr(dphi), _ptr(db), _ptr(dalpha), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(x.device))
    _check(st, "mhc_layer_bwd_recompute")
    return LayerBwdOut(dx, dy, dphi, db, dalpha)


def mhc_post_pre(x, y, H_post_l, H_res_l, phi, b, alpha, iters: int = 20,
                 eps: float = 1e-6):
    """mhc_post of layer l, then mhc_pre of layer l + 1 on the stored x_next."""
    T, n, D = x.shape
    G = 2 * n + n * n
    if y.dtype != x.dtype:
        raise TypeError("x and y must share a dtype")
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PostPreOut(_empty(x.shape, x.dtype, x.device),
                     _empty((T, D), dtype=x.dtype, device=x.device),
                     _empty((T, n), **f32), _empty((T, n), **f32),
                     _empty((T, n, n), **f32), _empty((T, G), **f32),
                     _empty((T,), **f32))
    nws = int(lib().mhc_post_pre_workspace_bytes(_dtype_code(x), T, n, D))
    ws = _empty((max(nws, 1),), dtype=torch.uint8, device=x.device)
    st = lib().mhc_post_pre(_dtype_code(x), _ptr(x), _ptr(y), _ptr(_f32(H_post_l, "H_post_l")),
                            _ptr(_f32(H_res_l, "H_res_l")), _ptr(_f32(phi, "phi")),
                            _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")), T, n, D, iters, eps,
                            *[_ptr(o) for o in out], _ptr(ws), nws, _stream(x.device))
    _check(st, "mhc_post_pre")
    return out


def mhc_post_norm(x, y, H_post, H_res, flags: int, eps: float = 1e-6):
    """mhc_post with the sandwich (flag 1) and block (flag 2) normalisations."""
    T, n, D = x.shape
    if y.dtype != x.dtype:
        raise TypeError("x and y must share a dtype")
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PostNormOut(_empty(x.shape, x.dtype, x.device), _empty((T,), **f32), _empty((T,), **f32))
    st = lib().mhc_post_norm(_dtype_code(x), _ptr(x), _ptr(y), _ptr(_f32(H_post, "H_post")),
                             _ptr(_f32(H_res, "H_res")), flags, eps, T, n, D, *[_ptr(o) for o in out],
                             _stream(x.device))
    _check(st, "mhc_post_norm")
    return out


def mhc_post_norm_bwd(g_next, x, y, H_post, H_res, flags: int, inv_rms_y, inv_rms_out,
                      eps: float = 1e-6):
    """Gradients of <g_next, x_next> for mhc_post_norm: (dx, dy, dH_post, dH_res)."""
    T, n, D = x.shape
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PostBwdOut(_empty(x.shape, x.dtype, x.device), _empty(y.shape, y.dtype, y.device),
                     _empty((T, n), **f32), _empty((T, n, n), **f32))
    st = lib().mhc_post_norm_bwd(_dtype_code(x), _ptr(g_next), _ptr(x), _ptr(y),
                                 _ptr(_f32(H_post, "H_post")), _ptr(_f32(H_res, "H_res")), flags, eps,
                                 _ptr(_f32(inv_rms_y, "inv_rms_y")), _ptr(_f32(inv_rms_out, "inv_rms_out")),
                                 T, n, D, *[_ptr(o) for o in out], _stream(x.device))
    _check(st, "mhc_post_norm_bwd")
    return out


def mhc_post(x, y, H_post, H_res):
    """x_next [T, n, D] = H_res x + H_post (x) y."""
    T, n, D = x.shape
    if y.dtype != x.dtype:
        raise TypeError("x and y must share a dtype")
    x_next = _empty(x.shape, x.dtype, x.device)
    st = lib().mhc_post(_dtype_code(x), _ptr(x), _ptr(y), _ptr(_f32(H_post, "H_post")),
                        _ptr(_f32(H_res, "H_res")), T, n, D, _ptr(x_next),
                        _stream(x.device))
    _check(st, "mhc_post")
    return x_next


def mhc_post_bwd(g_next, x, y, H_post, H_res):
    """Gradients of <g_next, x_next>: (dx, dy, dH_post, dH_res)."""
    T, n, D = x.shape
    if not (g_next.dtype == x.dtype == y.dtype):
        raise TypeError("g_next, x and y must share a dtype")
    f32 = dict(dtype=torch.float32, device=x.device)
    out = PostBwdOut(_empty(x.shape, x.dtype, x.device), _empty(y.shape, y.dtype, y.device),
                     _empty((T, n), **f32), _empty((T, n, n), **f32))
    st = lib().mhc_post_bwd(_dtype_code(x), _ptr(g_next), _ptr(x), _ptr(y),
                            _ptr(_f32(H_post, "H_post")), _ptr(_f32(H_res, "H_res")),
                            T, n, D, *[_ptr(o) for o in out], _stream(x.device))
    _check(st, "mhc_post_bwd")
    return out


def kernel_launches(op: str, dtype, T: int, n: int, D: int) -> int:
    """Kernels the entry point ``op`` launches for these sizes."""
    code = MHC_BF16 if dtype in (torch.bfloat16, "bf16") else MHC_F32
    return int(lib().mhc_kernel_launches(op.encode(), code, T, n, D))


def pre_bwd_workspace_bytes(dtype, T: int, n: int, D: int) -> int:
    code = MHC_BF16 if dtype == torch.bfloat16 else MHC_F32
    return int(lib().mhc_pre_bwd_workspace_bytes(code, T, n, D))


def mhc_pre_bwd(g_in, dH_post, dH_res, x, phi, b, alpha, proj, inv_rms, dx,
                iters: int = 20, workspace=None):
    """Backward of mhc_pre.  ``dx`` is accumulated in place (dx += pre part)."""
    T, n, D = x.shape
    G = 2 * n + n * n
    if not (g_in.dtype == x.dtype == dx.dtype):
        raise TypeError("g_in, x and dx must share a dtype")
    need = pre_bwd_workspace_bytes(x.dtype, T, n, D)
    if workspace is None:
        workspace = _empty((max(need, 16),), dtype=torch.uint8, device=x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    dphi = _empty((n * D, G), **f32)
    db = _empty((G,), **f32)
    dalpha = _empty((3,), **f32)
    st = lib().mhc_pre_bwd(_dtype_code(x), _ptr(g_in), _ptr(_f32(dH_post, "dH_post")),
                           _ptr(_f32(dH_res, "dH_res")), _ptr(x), _ptr(_f32(phi, "phi")),
                           _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")),
                           _ptr(_f32(proj, "proj")), _ptr(_f32(inv_rms, "inv_rms")),
                           T, n, D, iters, _ptr(dx), _ptr(dphi), _ptr(db), _ptr(dalpha),
                           _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(x.device))
    _check(st, "mhc_pre_bwd")
    return PreBwdOut(dx, dphi, db, dalpha)


def mhc_pre_bwd_noalloc(g_in, dH_post, dH_res, x, phi, b, alpha, proj, inv_rms,
                        dx, iters: int = 20):
    """mhc_pre_bwd with the library's fixed scratch array instead of a
    caller workspace (for callers that cannot allocate device memory).
    ``dx`` is accumulated in place; the outputs dphi, db, dalpha are allocated
    here by torch only because this binding returns new tensors."""
    T, n, D = x.shape
    G = 2 * n + n * n
    if not (g_in.dtype == x.dtype == dx.dtype):
        raise TypeError("g_in, x and dx must share a dtype")
    f32 = dict(dtype=torch.float32, device=x.device)
    dphi = _empty((n * D, G), **f32)
    db = _empty((G,), **f32)
    dalpha = _empty((3,), **f32)
    st = lib().mhc_pre_bwd_noalloc(
        _dtype_code(x), _ptr(g_in), _ptr(_f32(dH_post, "dH_post")), _ptr(_f32(dH_res, "dH_res")),
        _ptr(x), _ptr(_f32(phi, "phi")), _ptr(_f32(b, "b")), _ptr(_f32(alpha, "alpha")),
        _ptr(_f32(proj, "proj")), _ptr(_f32(inv_rms, "inv_rms")), T, n, D, iters, _ptr(dx),
        _ptr(dphi), _ptr(db), _ptr(dalpha), _stream(x.device))
    _check(st, "mhc_pre_bwd_noalloc")
    return PreBwdOut(dx, dphi, db, dalpha)


# ------------------------------------------------------ attention sublayer
#
# These calls are made once per layer in a decoding step, where the host's time
# is the call's time: their checks and marshalling are in a CPython module
# (csrc/py_attn.cpp), which is given the addresses of the library's entry points.

CALLS_PATH = os.path.join(os.path.dirname(LIB_PATH), "_attn_calls.so")
# the entry points that it calls, in its order
CALLS_ENTRIES = ("mhc_qk_norm_rope", "mhc_qk_norm_rope_bwd", "mhc_qk_norm_rope_bwd_workspace_bytes",
                 "mhc_qk_norm_rope_append", "mhc_paged_attn", "mhc_paged_attn_workspace_bytes")
_calls_module = None


def _calls():
    """The module, loaded once."""
    global _calls_module
    if _calls_module is None:
        handle = lib()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} is missing: build it with `python -m mhc_pre_gb300.build`")
        from . import _attn_calls, build
        made_for, here = _attn_calls.made_for, build.calls_made_for()
        if made_for != here:
            raise RuntimeError(f"{CALLS_PATH} was built for {made_for}, this is {here}: build it again with "
                               "`python -m mhc_pre_gb300.build`")
        _attn_calls.bind(*(ctypes.cast(getattr(handle, n), _P).value for n in CALLS_ENTRIES))
        _calls_module = _attn_calls
    return _calls_module


def _allocator():
    """What _calls() allocates with: None (torch's empty) unless _empty has been replaced."""
    return None if _empty is _torch_empty else _empty


def mhc_qk_norm_rope(q, k, w_q, w_k, positions=None, cos_sin=None, eps: float = 1e-6,
                     interleaved: bool = False):
    """Per-head RMSNorm of q [T, Hq, Dh] and k [T, Hk, Dh], then the rotation of
    the first cos_sin.shape[1] values of each head by cos_sin[positions]
    (cosines, then sines).  ``interleaved``: pairs (2j, 2j + 1)."""
    st, qo, ko = (_calls_module or _calls()).qk_norm_rope(_allocator(), q, k, w_q, w_k, positions, cos_sin, eps,
                                                          ROPE_ADJACENT if interleaved else 0)
    if st:
        _check(st, "mhc_qk_norm_rope")
    return QKOut(qo, ko)


def mhc_qk_norm_rope_bwd(g_q, g_k, q, k, w_q, w_k, positions=None, cos_sin=None, eps: float = 1e-6,
                         interleaved: bool = False, dq=None, dk=None):
    """Gradients of <g_q, q_out> + <g_k, k_out> for mhc_qk_norm_rope.  ``dq`` and
    ``dk`` (parts of a packed gradient, say) are written when given."""
    st, dq, dk, dw_q, dw_k = (_calls_module or _calls()).qk_norm_rope_bwd(
        _allocator(), g_q, g_k, q, k, w_q, w_k, positions, cos_sin, eps, ROPE_ADJACENT if interleaved else 0, dq, dk)
    if st:
        _check(st, "mhc_qk_norm_rope_bwd")
    return QKBwdOut(dq, dk, dw_q, dw_k)


def mhc_qk_norm_rope_append(q, k, v, w_q, w_k, k_cache, v_cache, slots, positions=None, cos_sin=None,
                            eps: float = 1e-6, interleaved: bool = False):
    """The serving form: returns the normalised, rotated q; the keys (likewise)
    and the values go to slots[t] = page * page_size + place of the caches
    [pages, page_size, Hk, Dh] (-1: nowhere), in place."""
    st, out = (_calls_module or _calls()).qk_norm_rope_append(
        _allocator(), q, k, v, w_q, w_k, k_cache, v_cache, slots, positions, cos_sin, eps,
        ROPE_ADJACENT if interleaved else 0)
    if st:
        _check(st, "mhc_qk_norm_rope_append")
    return out


def mhc_paged_attn_plan(cu_q, kv_lens, dtype, T: int, Hq: int, Hk: int, Dh: int, page_size: int,
                        max_q: int, max_kv: int, window: int = 0):
    """Splits a batch over the GPU once, for every mhc_paged_attn call of the
    same sizes (the layers of one step).  Calls that share a plan share its
    workspace: they must not overlap.  After a call that timed out the batch has
    to be planned again."""
    B = kv_lens.numel()
    for t, name, n in ((cu_q, "cu_q", B + 1), (kv_lens, "kv_lens", B)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be {torch.int32}, got {t.dtype}")
        if t.numel() != n:
            raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"activations must be bfloat16 or float32, got {dtype}")
    code = MHC_BF16 if dtype == torch.bfloat16 else MHC_F32
    need = int(lib().mhc_paged_attn_workspace_bytes(code, T, B, Hq, Hk, Dh, page_size, max_q))
    ws = _empty((max(need, 16),), dtype=torch.uint8, device=cu_q.device)
    st = lib().mhc_paged_attn_plan(code, _ptr(cu_q), _ptr(kv_lens), T, B, Hq, Hk, Dh, page_size, max_q, max_kv,
                                   window, _ptr(ws), need, _stream(cu_q.device))
    _check(st, "mhc_paged_attn_plan")
    return PagedAttnPlan(ws, (code, T, B, Hq, Hk, Dh, page_size, max_q, max_kv, window))


def mhc_paged_attn(q, k_cache, v_cache, page_table, cu_q=None, kv_lens=None, max_q: int = None,
                   max_kv: int = None, scale: float = None, window: int = None, softcap: float = 0.0,
                   plan=None, out=None):
    """Causal attention of the new tokens q [T, Hq, Dh] over a paged cache
    [pages, page_size, Hk, Dh]: sequence b has the rows cu_q[b]:cu_q[b+1] and
    kv_lens[b] cached tokens, the new ones last.  ``max_q`` and ``max_kv`` bound
    the new and the cached tokens of a sequence (default: all rows of q, the
    page table's width); ``window`` 0 or None: unlimited.  ``plan`` (from
    mhc_paged_attn_plan) takes the place of cu_q and kv_lens and brings its own
    max_q, max_kv and window.  ``out``: a tensor for o; rows of no sequence stay
    as they are.  Returns o and lse [T, Hq]."""
    ws = None
    if plan is not None:
        ws, sizes = plan
        max_q, max_kv, window = (a if b is None else b for a, b in zip(sizes[7:], (max_q, max_kv, window)))
        code = MHC_BF16 if q.dtype == torch.bfloat16 else MHC_F32
        want = (code, q.shape[0], page_table.shape[0], q.shape[1], k_cache.shape[2], q.shape[2], k_cache.shape[1],
                max_q, max_kv, window)
        if want != sizes or cu_q is not None or kv_lens is not None:
            raise ValueError(f"the plan has its own lengths and sizes: {sizes}, not {want}")
    st, o, lse = (_calls_module or _calls()).paged_attn(
        _allocator(), q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window or 0, softcap, ws, out)
    if st:
        _check(st, "mhc_paged_attn")
    return PagedAttnOut(o, lse)


def get_last_device_error(device=None) -> int:
    """Synchronises the current stream and returns the device error status."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    return int(lib().mhc_get_last_device_error(_stream(dev)))

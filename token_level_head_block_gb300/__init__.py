"""MHLA forward pass (token-level multi-head linear attention) on GB300, sm_103a.

Thin Python binding of the C ABI in ``include/mhla.h`` (``lib/libmhla.so``):
argument marshalling only.  Every step of the forward pass runs in the
library's CUDA kernels; PyTorch supplies device memory and streams.  There is
no CPU fallback: calls raise when the library is missing or a call fails.
"""

from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

__all__ = [
    "MhlaError", "lib", "library_path", "num_blocks", "init_mixing", "workspace_size",
    "select_path", "forward", "forward_causal", "causal_workspace_size", "backward", "backward_workspace_size",
    "backward_causal", "backward_causal_workspace_size",
    "device_status", "profile_begin", "layer_norm", "lepe_add", "module_forward",
    "module_workspace_size",
    "profile_end", "tensor_desc", "shape3",
    "gated_forward", "gated_workspace_size", "gated_backward", "gated_backward_workspace_size", "gated_step",
    "init_rotation", "qk_norm", "qk_norm_backward", "qk_norm_backward_workspace_size",
    "PATHS", "TRANSFORMS", "ROTATION_LAYOUTS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "lib", "libmhla.so")

PATHS = {"auto": 0, "simt": 1, "tc": 2, "fused": 3, "tc_fused": 4}
TRANSFORMS = {"linear": 0, "cos": 1, "exp": 2, "gaussian": 3, "local": 4}
PHIS = {"relu": 0, "relu_eps": 1}
DTYPES = {"bf16": 0, "f32": 1}
ROTATION_LAYOUTS = {"half": 0, "interleaved": 1}

STATUS = {
    0: "ok", 1: "invalid argument", 2: "shape mismatch", 3: "unsupported by the selected path",
    4: "CUDA error", 5: "device wait timed out", 6: "workspace missing, too small or misaligned",
}


class MhlaError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = int(status)
        super().__init__(f"{what}: {STATUS.get(self.status, 'unknown status')} ({self.status})")


class Shape3(ctypes.Structure):
    _fields_ = [("ndim", ctypes.c_int32), ("pad_", ctypes.c_int32), ("extent", ctypes.c_int64 * 3)]


class Phi(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_float)]


class Tensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("pad_", ctypes.c_int32),
        ("B", ctypes.c_int64), ("N", ctypes.c_int64), ("H", ctypes.c_int64), ("d", ctypes.c_int64),
        ("stride_b", ctypes.c_int64), ("stride_n", ctypes.c_int64), ("stride_h", ctypes.c_int64),
    ]


class ModuleParams(ctypes.Structure):
    """mhla_module_params_t: device pointers of the module's parameters."""
    _fields_ = [
        ("ln_weight", ctypes.c_void_p), ("ln_bias", ctypes.c_void_p),
        ("qkv_weight", ctypes.c_void_p), ("qkv_bias", ctypes.c_void_p),
        ("lepe_weight", ctypes.c_void_p), ("lepe_bias", ctypes.c_void_p),
        ("out_weight", ctypes.c_void_p), ("out_bias", ctypes.c_void_p),
        ("ln_eps", ctypes.c_float), ("heads", ctypes.c_int32),
    ]


class Rotation(ctypes.Structure):
    """mhla_rotation_t: the table, the rows of the tokens and which channels pair up."""
    _fields_ = [
        ("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rows", ctypes.c_int64),
        ("pairs", ctypes.c_int32), ("layout", ctypes.c_int32),
    ]


_lib = None


def library_path():
    return _LIB_PATH


def lib():
    """The loaded libmhla (raises when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise MhlaError(4, f"{_LIB_PATH} is missing; build it with "
                           "`python -m token_level_head_block_gb300.build`")
    L = ctypes.CDLL(_LIB_PATH)
    P = ctypes.POINTER
    L.mhla_num_blocks.argtypes = [P(Shape3), P(Shape3)]
    L.mhla_num_blocks.restype = ctypes.c_int64
    L.mhla_init_mixing.argtypes = [P(Shape3), P(Shape3), ctypes.c_int32, ctypes.c_double, ctypes.c_double,
                                   P(ctypes.c_float), ctypes.c_int64]
    L.mhla_init_mixing.restype = ctypes.c_int
    L.mhla_workspace_size.argtypes = [P(Tensor), P(Shape3), P(Shape3), ctypes.c_int32, P(ctypes.c_size_t)]
    L.mhla_workspace_size.restype = ctypes.c_int
    L.mhla_select_path.argtypes = [P(Tensor), P(Tensor), P(Tensor), P(Tensor), P(Shape3), P(Shape3)]
    L.mhla_select_path.restype = ctypes.c_int32
    L.mhla_forward.argtypes = [P(Tensor), P(Tensor), P(Tensor), ctypes.c_void_p, P(Shape3), P(Shape3), P(Phi),
                               P(Tensor), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int32]
    L.mhla_forward.restype = ctypes.c_int
    L.mhla_causal_workspace_size.argtypes = [P(Tensor), P(Shape3), P(Shape3), ctypes.c_int32, P(ctypes.c_size_t)]
    L.mhla_causal_workspace_size.restype = ctypes.c_int
    L.mhla_forward_causal.argtypes = [P(Tensor), P(Tensor), P(Tensor), ctypes.c_void_p, P(Shape3), P(Shape3),
                                      P(Phi), P(Tensor), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                      ctypes.c_int32]
    L.mhla_forward_causal.restype = ctypes.c_int
    L.mhla_backward_workspace_size.argtypes = [P(Tensor), P(Shape3), P(Shape3), ctypes.c_int32,
                                               P(ctypes.c_size_t)]
    L.mhla_backward_workspace_size.restype = ctypes.c_int
    L.mhla_backward.argtypes = [P(Tensor), P(Tensor), P(Tensor), ctypes.c_void_p, P(Shape3), P(Shape3), P(Phi),
                                P(Tensor), P(Tensor), P(Tensor), P(Tensor), ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int32]
    L.mhla_backward.restype = ctypes.c_int
    L.mhla_backward_causal_workspace_size.argtypes = [P(Tensor), P(Shape3), P(Shape3), ctypes.c_int32,
                                                      P(ctypes.c_size_t)]
    L.mhla_backward_causal_workspace_size.restype = ctypes.c_int
    L.mhla_backward_causal.argtypes = L.mhla_backward.argtypes
    L.mhla_backward_causal.restype = ctypes.c_int
    L.mhla_layer_norm.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p]
    L.mhla_layer_norm.restype = ctypes.c_int
    L.mhla_lepe_add.argtypes = [P(Tensor), P(Tensor), P(Shape3), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    L.mhla_lepe_add.restype = ctypes.c_int
    L.mhla_linear.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                              ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
    L.mhla_linear.restype = ctypes.c_int
    L.mhla_module_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                             P(Shape3), P(Shape3), P(ctypes.c_size_t)]
    L.mhla_module_workspace_size.restype = ctypes.c_int
    L.mhla_module_forward.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, P(ModuleParams), ctypes.c_void_p, P(Shape3), P(Shape3),
                                      P(Phi), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    L.mhla_module_forward.restype = ctypes.c_int
    V = T = ctypes.c_void_p   # tensors as packed bytes or by reference
    L.mhla_gated_workspace_size.argtypes = [T, P(ctypes.c_size_t)]
    L.mhla_gated_backward_workspace_size.argtypes = [T, P(ctypes.c_size_t)]
    L.mhla_gated_forward.argtypes = [T, T, T, T, ctypes.c_float, V, T, V, V, ctypes.c_size_t, V]
    L.mhla_gated_backward.argtypes = [T, T, T, T, T, ctypes.c_float, V, V, T, T, T, T, V, V, ctypes.c_size_t, V]
    L.mhla_gated_step.argtypes = [T, T, T, T, ctypes.c_float, V, T, V]
    L.mhla_init_rotation.argtypes = [P(Shape3), P(ctypes.c_int32), ctypes.c_double, P(ctypes.c_float),
                                     ctypes.c_int64]
    L.mhla_qk_norm.argtypes = [T, T, V, V, ctypes.c_float, P(Rotation), T, T, V]
    L.mhla_qk_norm_backward_workspace_size.argtypes = [T, P(ctypes.c_size_t)]
    L.mhla_qk_norm_backward.argtypes = [T, T, V, V, ctypes.c_float, P(Rotation), T, T, T, T, V, V, V,
                                        ctypes.c_size_t, V]
    for name in ("mhla_gated_workspace_size", "mhla_gated_backward_workspace_size", "mhla_gated_forward",
                 "mhla_gated_backward", "mhla_gated_step", "mhla_init_rotation", "mhla_qk_norm",
                 "mhla_qk_norm_backward_workspace_size", "mhla_qk_norm_backward"):
        getattr(L, name).restype = ctypes.c_int
    L.mhla_debug_stall_waits.argtypes = [ctypes.c_int32, ctypes.c_uint64]
    L.mhla_debug_stall_waits.restype = ctypes.c_int
    L.mhla_device_status.argtypes = [ctypes.c_void_p, P(ctypes.c_uint32)]
    L.mhla_device_status.restype = ctypes.c_int
    L.mhla_status_string.argtypes = [ctypes.c_int32]
    L.mhla_status_string.restype = ctypes.c_char_p
    L.mhla_profile_begin.argtypes = []
    L.mhla_profile_begin.restype = ctypes.c_int
    L.mhla_profile_end.argtypes = [P(KernelTime), ctypes.c_int32, P(ctypes.c_int32)]
    L.mhla_profile_end.restype = ctypes.c_int
    L.mhla_version.argtypes = []
    L.mhla_version.restype = ctypes.c_char_p
    _lib = L
    return L


def shape3(ext):
    ext = tuple(int(e) for e in ext)
    s = Shape3()
    s.ndim = len(ext)
    for a, e in enumerate(ext[:3]):
        s.extent[a] = e
    return s


def tensor_desc(ptr, dtype, shape, strides):
    """mhla_tensor_t for a [B, N, H, d] operand given its address and element strides."""
    t = Tensor()
    t.data = ctypes.c_void_p(int(ptr)) if ptr else None
    t.dtype = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    t.B, t.N, t.H, t.d = (int(x) for x in shape)
    t.stride_b, t.stride_n, t.stride_h = (int(x) for x in strides[:3])
    return t


def _desc(x):
    import torch
    if x.dim() != 4:
        raise ValueError("expected a [B, N, H, d] tensor")
    if x.shape[3] > 1 and x.stride(3) != 1:
        raise ValueError("the d dimension must be contiguous")
    if x.dtype == torch.bfloat16:
        dt = "bf16"
    elif x.dtype == torch.float32:
        dt = "f32"
    else:
        raise ValueError(f"unsupported dtype {x.dtype}")
    return tensor_desc(x.data_ptr(), dt, tuple(x.shape), (x.stride(0), x.stride(1), x.stride(2)))


def _check(status, what):
    if status != 0:
        raise MhlaError(status, what)


def num_blocks(grid, block):
    m = lib().mhla_num_blocks(ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)))
    if m < 0:
        raise MhlaError(-m, "mhla_num_blocks")
    return int(m)


def init_mixing(grid, block, transform="linear", local_thres=1.5, exp_sigma=3.0):
    """M x M float32 mixing matrix from block-centre distances (host computation)."""
    M = num_blocks(grid, block)
    W = np.empty((M, M), dtype=np.float32)
    st = lib().mhla_init_mixing(ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)),
                                TRANSFORMS[transform], float(local_thres), float(exp_sigma),
                                W.ctypes.data_as(ctypes.POINTER(ctypes.c_float)), W.size)
    _check(st, "mhla_init_mixing")
    return W


def workspace_size(q, grid, block, path="auto"):
    n = ctypes.c_size_t(0)
    _check(lib().mhla_workspace_size(ctypes.byref(_desc(q) if not isinstance(q, Tensor) else q),
                                     ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)), PATHS[path],
                                     ctypes.byref(n)), "mhla_workspace_size")
    return int(n.value)


def select_path(q, k, v, out, grid, block):
    r = lib().mhla_select_path(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)),
                               ctypes.byref(_desc(out)), ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)))
    if r < 0:
        raise MhlaError(-r, "mhla_select_path")
    return {1: "simt", 2: "tc", 3: "fused"}[r]


def forward(q, k, v, W, grid, block, phi="relu", eps=1e-6, out=None, workspace=None, stream=None,
            path="auto"):
    """MHLA forward of device tensors q, k, v [B, N, H, d]; returns ``out``.

    W is a float32 CUDA tensor (M x M, contiguous), shared by all batches and
    heads.  ``workspace`` is an optional uint8 CUDA tensor of at least
    ``workspace_size`` bytes; without it the call takes stream-ordered memory.
    Asynchronous on ``stream`` (default: torch's current stream).
    """
    import torch
    if out is None:
        out = torch.empty_like(q)
    if not W.is_contiguous() or W.dtype != torch.float32:
        raise ValueError("W must be a contiguous float32 tensor")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() *
                                                            workspace.element_size())
    st = lib().mhla_forward(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)),
                            ctypes.c_void_p(W.data_ptr()), ctypes.byref(shape3(grid)),
                            ctypes.byref(shape3(block)), ctypes.byref(Phi(PHIS[phi], float(eps))),
                            ctypes.byref(_desc(out)), ctypes.c_void_p(ws_ptr) if ws_ptr else None,
                            ws_bytes, ctypes.c_void_p(sptr) if sptr else None, PATHS[path])
    _check(st, "mhla_forward")
    return out


def causal_workspace_size(q, grid, block, path="auto"):
    n = ctypes.c_size_t(0)
    _check(lib().mhla_causal_workspace_size(ctypes.byref(_desc(q) if not isinstance(q, Tensor) else q),
                                            ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)), PATHS[path],
                                            ctypes.byref(n)), "mhla_causal_workspace_size")
    return int(n.value)


def forward_causal(q, k, v, W, grid, block, phi="relu", eps=1e-6, out=None, workspace=None, stream=None,
                   path="auto"):
    """Causal (chunkwise) MHLA of device tensors [B, N, H, d]; blocks must be
    contiguous token ranges (e.g. grid (1, N), block (1, w)).  Returns ``out``."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    if not W.is_contiguous() or W.dtype != torch.float32:
        raise ValueError("W must be a contiguous float32 tensor")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() *
                                                            workspace.element_size())
    st = lib().mhla_forward_causal(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)),
                                   ctypes.c_void_p(W.data_ptr()), ctypes.byref(shape3(grid)),
                                   ctypes.byref(shape3(block)), ctypes.byref(Phi(PHIS[phi], float(eps))),
                                   ctypes.byref(_desc(out)), ctypes.c_void_p(ws_ptr) if ws_ptr else None,
                                   ws_bytes, ctypes.c_void_p(sptr) if sptr else None, PATHS[path])
    _check(st, "mhla_forward_causal")
    return out


def backward_workspace_size(q, grid, block, path="auto"):
    n = ctypes.c_size_t(0)
    _check(lib().mhla_backward_workspace_size(ctypes.byref(_desc(q) if not isinstance(q, Tensor) else q),
                                              ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)),
                                              PATHS[path], ctypes.byref(n)), "mhla_backward_workspace_size")
    return int(n.value)


def backward(q, k, v, W, dout, grid, block, phi="relu", eps=1e-6, dq=None, dk=None, dv=None, dW=None,
             workspace=None, stream=None, path="auto"):
    """Gradients (dq, dk, dv, dW) of the MHLA forward given dout = dL/d(out).

    Device tensors [B, N, H, d] like ``forward``; dW is a float32 M x M CUDA
    tensor (allocated when not given) holding the sum over batches and heads.
    Asynchronous on ``stream`` (default: torch's current stream).
    """
    import torch
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dW is None:
        dW = torch.empty_like(W)
    for name, x in (("W", W), ("dW", dW)):
        if not x.is_contiguous() or x.dtype != torch.float32:
            raise ValueError(f"{name} must be a contiguous float32 tensor")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() *
                                                            workspace.element_size())
    st = lib().mhla_backward(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)),
                             ctypes.c_void_p(W.data_ptr()), ctypes.byref(shape3(grid)),
                             ctypes.byref(shape3(block)), ctypes.byref(Phi(PHIS[phi], float(eps))),
                             ctypes.byref(_desc(dout)), ctypes.byref(_desc(dq)), ctypes.byref(_desc(dk)),
                             ctypes.byref(_desc(dv)), ctypes.c_void_p(dW.data_ptr()),
                             ctypes.c_void_p(ws_ptr) if ws_ptr else None, ws_bytes,
                             ctypes.c_void_p(sptr) if sptr else None, PATHS[path])
    _check(st, "mhla_backward")
    return dq, dk, dv, dW


def backward_causal_workspace_size(q, grid, block, path="auto"):
    n = ctypes.c_size_t(0)
    _check(lib().mhla_backward_causal_workspace_size(ctypes.byref(_desc(q) if not isinstance(q, Tensor) else q),
                                                     ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)),
                                                     PATHS[path], ctypes.byref(n)),
           "mhla_backward_causal_workspace_size")
    return int(n.value)


def backward_causal(q, k, v, W, dout, grid, block, phi="relu", eps=1e-6, dq=None, dk=None, dv=None, dW=None,
                    workspace=None, stream=None, path="auto"):
    """Gradients (dq, dk, dv, dW) of ``forward_causal`` given dout = dL/d(out).

    Arguments as for ``backward``; the blocks must be contiguous token ranges
    as for ``forward_causal``.  dW is zero above the diagonal."""
    import torch
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dW is None:
        dW = torch.empty_like(W)
    for name, x in (("W", W), ("dW", dW)):
        if not x.is_contiguous() or x.dtype != torch.float32:
            raise ValueError(f"{name} must be a contiguous float32 tensor")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() *
                                                            workspace.element_size())
    st = lib().mhla_backward_causal(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)),
                                    ctypes.c_void_p(W.data_ptr()), ctypes.byref(shape3(grid)),
                                    ctypes.byref(shape3(block)), ctypes.byref(Phi(PHIS[phi], float(eps))),
                                    ctypes.byref(_desc(dout)), ctypes.byref(_desc(dq)), ctypes.byref(_desc(dk)),
                                    ctypes.byref(_desc(dv)), ctypes.c_void_p(dW.data_ptr()),
                                    ctypes.c_void_p(ws_ptr) if ws_ptr else None, ws_bytes,
                                    ctypes.c_void_p(sptr) if sptr else None, PATHS[path])
    _check(st, "mhla_backward_causal")
    return dq, dk, dv, dW


def _stream_ptr(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(sptr) if sptr else None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def layer_norm(x, weight, bias, eps=1e-5, out=None, stream=None):
    """LayerNorm over the last axis of a contiguous bf16 CUDA tensor (float32
    weight and bias of that size); returns ``out`` (may be ``x``)."""
    import torch
    out = torch.empty_like(x) if out is None else out
    C = x.shape[-1]
    st = lib().mhla_layer_norm(_ptr(x), _ptr(out), x.numel() // C, C, _ptr(weight), _ptr(bias), float(eps),
                               _stream_ptr(stream, x.device))
    _check(st, "mhla_layer_norm")
    return out


def linear(x, w, bias=None, out=None, stream=None):
    """y = x w^T (+ bias) for a contiguous bf16 CUDA tensor x [..., k] and an
    nn.Linear-layout weight w [n_out, k] (bias [n_out] or None); returns ``out``."""
    import torch
    k = x.shape[-1]
    n_out = w.shape[0]
    rows = x.numel() // k if k else 0
    if out is None:
        out = torch.empty(*x.shape[:-1], n_out, dtype=x.dtype, device=x.device)
    st = lib().mhla_linear(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), rows, k, n_out, _stream_ptr(stream, x.device))
    _check(st, "mhla_linear")
    return out


def lepe_add(v, out, grid, weight, bias, stream=None):
    """out += 5 x 5 depthwise convolution of v (+ bias) over the token image, for
    bf16 [B, N, H, d] CUDA views; weight float32 [H * d, 5, 5], bias [H * d]."""
    st = lib().mhla_lepe_add(ctypes.byref(_desc(v)), ctypes.byref(_desc(out)), ctypes.byref(shape3(grid)),
                             _ptr(weight), _ptr(bias), _stream_ptr(stream, v.device))
    _check(st, "mhla_lepe_add")
    return out


def module_workspace_size(B, N, C, heads, grid, block):
    n = ctypes.c_size_t(0)
    _check(lib().mhla_module_workspace_size(B, N, C, heads, ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)),
                                            ctypes.byref(n)), "mhla_module_workspace_size")
    return int(n.value)


def module_forward(x, params, W, grid, block, heads, phi="relu_eps", eps=1e-6, ln_eps=1e-5, out=None,
                   workspace=None, stream=None):
    """The MHLA module (LayerNorm, qkv projection, MHLA, 5 x 5 positional term,
    output projection) on a contiguous bf16 CUDA tensor x [B, N, C].

    ``params``: CUDA tensors ln_weight, ln_bias (float32 [C]); qkv_weight (bf16
    [3C, C]) and optional qkv_bias (bf16 [3C]); optional lepe_weight (float32
    [C, 5, 5]) with lepe_bias (float32 [C]); out_weight (bf16 [C, C]) and
    optional out_bias (bf16 [C]).  Returns ``out`` ([B, N, C], bf16).
    """
    import torch
    B, N, C = x.shape
    out = torch.empty_like(x) if out is None else out
    p = ModuleParams(_ptr(params["ln_weight"]), _ptr(params["ln_bias"]), _ptr(params["qkv_weight"]),
                     _ptr(params.get("qkv_bias")), _ptr(params.get("lepe_weight")), _ptr(params.get("lepe_bias")),
                     _ptr(params["out_weight"]), _ptr(params.get("out_bias")), float(ln_eps), int(heads))
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() *
                                                            workspace.element_size())
    st = lib().mhla_module_forward(_ptr(x), _ptr(out), B, N, C, ctypes.byref(p), _ptr(W),
                                   ctypes.byref(shape3(grid)), ctypes.byref(shape3(block)),
                                   ctypes.byref(Phi(PHIS[phi], float(eps))),
                                   ctypes.c_void_p(ws_ptr) if ws_ptr else None, ws_bytes,
                                   _stream_ptr(stream, x.device))
    _check(st, "mhla_module_forward")
    return out


# --------------------------------------------------- gated recurrence, query/key norm


_PACK_TENSOR = struct.Struct("Pii7q").pack   # mhla_tensor_t
_CODES = {}


def _dtype_code(x):
    code = _CODES.get(x.dtype)
    if code is None:
        import torch
        _CODES.update({torch.bfloat16: 0, torch.float32: 1})
        code = _CODES.get(x.dtype)
        if code is None:
            raise ValueError(f"unsupported dtype {x.dtype}")
    return code


# These two pack the C struct directly, and _launch takes its arguments as they are: serving
# makes such a call per token, and filling a ctypes structure field by field costs
# more than the launch.
def _heads(x):
    """mhla_tensor_t of a [B, N, H, d] tensor."""
    B, N, H, d = x.shape
    sb, sn, sh, sd = x.stride()
    if sd != 1 and d > 1:
        raise ValueError("the d dimension must be contiguous")
    return _PACK_TENSOR(x.data_ptr(), _dtype_code(x), 0, B, N, H, d, sb, sn, sh)


def _gates(x):
    """mhla_tensor_t of a [B, N, H] tensor of one value per token and head."""
    B, N, H = x.shape
    sb, sn, sh = x.stride()
    return _PACK_TENSOR(x.data_ptr(), _dtype_code(x), 0, B, N, H, 1, sb, sn, sh)


def _float_array(name, x, shape, like):
    """Address of a contiguous float32 tensor of this shape on like's device, or None."""
    if x is None:
        return None
    if _dtype_code(x) != 1 or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {list(shape)}")
    if x.get_device() != like.get_device():
        raise ValueError(f"{name} is on {x.device}, not on {like.device}")
    return x.data_ptr()


def _new_float(shape, twin, like):
    """A float32 tensor of this shape on like's device, by its twin if there is one (the shorter call)."""
    import torch
    return torch.empty(shape, dtype=torch.float32, device=like.device) if twin is None else torch.empty_like(twin)


def _same_device(like, *tensors):
    index = like.get_device()
    if index < 0:
        raise ValueError("expected CUDA tensors")
    for x in tensors:
        if x.get_device() != index:
            raise ValueError(f"a tensor is on {x.device}, not on {like.device}")


def _on(stream, x):
    """The given stream (torch's, or a handle) as torch's current one on x's device: a call made under it allocates
    its outputs and its workspace there, so that their memory is not handed on before that stream is through with it."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=x.device)
    if stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, not on {x.device}")
    return torch.cuda.stream(stream)


def _launch(what, fn, args, x, workspace=None, need=None):
    """fn(*args, [workspace, bytes,] stream) on torch's current stream with x's device current.  need() tells the
    workspace's bytes (None: the call takes none); they come from torch's allocator when the caller brings
    no workspace."""
    import torch
    index = x.get_device()
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _launch(what, fn, args, x, workspace, need)
    s = torch._C._cuda_getCurrentRawStream(index)
    if need is None:
        st = fn(*args, s)
    elif workspace is not None:
        st = fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
    else:
        n = need()
        if n == 0:
            st = fn(*args, None, 0, s)
        else:
            scratch = torch.empty(n, dtype=torch.uint8, device=x.device)
            st = fn(*args, scratch.data_ptr(), n, s)
    if st != 0:
        raise MhlaError(st, what)


def _size(fn, what, desc):
    n = ctypes.c_size_t(0)
    _check(fn(desc, ctypes.byref(n)), what)
    return n.value


def gated_workspace_size(q):
    return _size(lib().mhla_gated_workspace_size, "mhla_gated_workspace_size", _heads(q))


def gated_backward_workspace_size(q):
    return _size(lib().mhla_gated_backward_workspace_size, "mhla_gated_backward_workspace_size", _heads(q))


def gated_forward(q, k, v, g, scale=1.0, state=None, out=None, state_out=None, workspace=None, stream=None):
    """Gated causal linear attention S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k, v: CUDA tensors [B, N, H, d]; g: log decays [B, N, H] of the same
    dtype; state: float32 [B, H, d, d] before the first token (None: zero).
    Returns (out, state_out); state_out (allocated when not given) may be state.
    ``stream`` (default: torch's current one) runs the call and owns what it allocates; the
    caller orders it behind the writers of its inputs and in front of the readers of its outputs.
    """
    import torch
    if stream is not None:
        with _on(stream, q):
            return gated_forward(q, k, v, g, scale, state, out, state_out, workspace)
    B, N, H, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if state_out is None:
        state_out = _new_float((B, H, d, d), state, q)
    dq = _heads(q)
    args = (dq, _heads(k), _heads(v), _gates(g), scale, _float_array("state", state, (B, H, d, d), q), _heads(out),
            _float_array("state_out", state_out, (B, H, d, d), q))
    _same_device(q, k, v, g, out)
    L = lib()
    _launch("mhla_gated_forward", L.mhla_gated_forward, args, q, workspace,
            lambda: _size(L.mhla_gated_workspace_size, "mhla_gated_workspace_size", dq))
    return out, state_out


def gated_backward(q, k, v, g, dout, scale=1.0, state=None, dstate_out=None, dq=None, dk=None, dv=None, dg=None,
                   dstate=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv, dg, dstate) of ``gated_forward`` given dout and,
    when the last state is used, dstate_out (float32 [B, H, d, d]).  ``stream`` as for ``gated_forward``."""
    import torch
    if stream is not None:
        with _on(stream, q):
            return gated_backward(q, k, v, g, dout, scale, state, dstate_out, dq, dk, dv, dg, dstate, workspace)
    B, N, H, d = q.shape
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    dg = torch.empty_like(g) if dg is None else dg
    if dstate is None:
        dstate = _new_float((B, H, d, d), state if dstate_out is None else dstate_out, q)
    desc = _heads(q)
    square = (B, H, d, d)
    args = (desc, _heads(k), _heads(v), _gates(g), _heads(dout), scale, _float_array("state", state, square, q),
            _float_array("dstate_out", dstate_out, square, q), _heads(dq), _heads(dk), _heads(dv), _gates(dg),
            _float_array("dstate", dstate, square, q))
    _same_device(q, k, v, g, dout, dq, dk, dv, dg)
    L = lib()
    _launch("mhla_gated_backward", L.mhla_gated_backward, args, q, workspace,
            lambda: _size(L.mhla_gated_backward_workspace_size, "mhla_gated_backward_workspace_size", desc))
    return dq, dk, dv, dg, dstate


def gated_step(q, k, v, g, state, scale=1.0, out=None, stream=None):
    """One token for every sequence: tensors [B, 1, H, d], g [B, 1, H]; ``state``
    (float32 [B, H, d, d]) is updated in place.  Returns ``out``.  ``stream`` as for ``gated_forward``."""
    if stream is not None:
        with _on(stream, q):
            return gated_step(q, k, v, g, state, scale, out)
    B, _, H, d = q.shape
    if out is None:
        import torch
        out = torch.empty_like(q)
    args = (_heads(q), _heads(k), _heads(v), _gates(g), scale, _float_array("state", state, (B, H, d, d), q), _heads(out))
    _same_device(q, k, v, g, out)
    _launch("mhla_gated_step", lib().mhla_gated_step, args, q)
    return out


def init_rotation(grid, pairs, base=10000.0):
    """Rotation table [prod(grid), sum(pairs), 2] (cos, sin; float32, host) of the token
    coordinates on a grid; ``pairs`` gives the rotated pairs of each grid axis
    (a sequence of N tokens: grid (1, N), pairs (0, n))."""
    grid = tuple(int(e) for e in grid)
    if len(pairs) != len(grid):
        raise ValueError("pairs needs one count per grid axis")
    n = 1
    for e in grid:
        n *= e
    total = sum(int(p) for p in pairs)
    table = np.empty((max(n, 0), max(total, 0), 2), dtype=np.float32)
    st = lib().mhla_init_rotation(ctypes.byref(shape3(grid)), (ctypes.c_int32 * 3)(*pairs), float(base),
                                  table.ctypes.data_as(ctypes.POINTER(ctypes.c_float)), table.size)
    _check(st, "mhla_init_rotation")
    return table


def _rotation(x, table, positions, layout):
    import torch
    if layout not in ROTATION_LAYOUTS:
        raise ValueError(f"unknown rotation layout {layout!r}")
    if table is None:
        return None
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("the rotation table is [rows, pairs, 2]")
    if table.shape[0] == 0 and table.shape[1] > 0:   # whose address would read as no table
        raise ValueError("the rotation table has no rows")
    ptr = _float_array("table", table, table.shape, x)
    pos = None
    if positions is not None:
        if positions.dtype != torch.int32 or tuple(positions.shape) != tuple(x.shape[:2]) \
                or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 tensor of shape {list(x.shape[:2])}")
        _same_device(x, positions)
        pos = positions.data_ptr()
    return Rotation(ptr or None, pos, table.shape[0], table.shape[1], ROTATION_LAYOUTS[layout])


def qk_norm(q, k, q_weight=None, k_weight=None, eps=1e-6, table=None, positions=None, layout="half", q_out=None,
            k_out=None, stream=None):
    """Root-mean-square norm of every head of q [B, N, H, d] and k [B, N, Hk, d] (float32
    weights [d]) and its rotation by ``table`` ([rows, pairs, 2], see ``init_rotation``) at
    ``positions`` (int32 [B, N]; None: 0 .. N-1).  Returns (q_out, k_out), which may be q and k.
    ``stream`` as for ``gated_forward``."""
    import torch
    if stream is not None:
        with _on(stream, q):
            return qk_norm(q, k, q_weight, k_weight, eps, table, positions, layout, q_out, k_out)
    if q_out is None:
        q_out = torch.empty_like(q)
    if k_out is None:
        k_out = torch.empty_like(k)
    d = q.shape[3]
    args = (_heads(q), _heads(k), _float_array("q_weight", q_weight, (d,), q), _float_array("k_weight", k_weight, (d,), q),
            eps, _rotation(q, table, positions, layout), _heads(q_out), _heads(k_out))
    _same_device(q, k, q_out, k_out)
    _launch("mhla_qk_norm", lib().mhla_qk_norm, args, q)
    return q_out, k_out


def qk_norm_backward_workspace_size(q):
    return _size(lib().mhla_qk_norm_backward_workspace_size, "mhla_qk_norm_backward_workspace_size", _heads(q))


def qk_norm_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, eps=1e-6, table=None, positions=None,
                     layout="half", dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qk_norm`` for its inputs q, k;
    dq may be dq_out and dk dk_out.  ``stream`` as for ``gated_forward``."""
    import torch
    if stream is not None:
        with _on(stream, q):
            return qk_norm_backward(q, k, dq_out, dk_out, q_weight, k_weight, eps, table, positions, layout, dq, dk,
                                    dq_weight, dk_weight, workspace)
    d = q.shape[3]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    if dq_weight is None:
        dq_weight = _new_float((d,), q_weight, q)
    if dk_weight is None:
        dk_weight = _new_float((d,), k_weight, q)
    desc = _heads(q)
    args = (desc, _heads(k), _float_array("q_weight", q_weight, (d,), q), _float_array("k_weight", k_weight, (d,), q), eps,
            _rotation(q, table, positions, layout), _heads(dq_out), _heads(dk_out), _heads(dq), _heads(dk),
            _float_array("dq_weight", dq_weight, (d,), q), _float_array("dk_weight", dk_weight, (d,), q))
    _same_device(q, k, dq_out, dk_out, dq, dk)
    L = lib()
    _launch("mhla_qk_norm_backward", L.mhla_qk_norm_backward, args, q, workspace,
            lambda: _size(L.mhla_qk_norm_backward_workspace_size, "mhla_qk_norm_backward_workspace_size", desc))
    return dq, dk, dq_weight, dk_weight


def profile_begin():
    """Start bracketing every kernel launch with CUDA events on its stream."""
    _check(lib().mhla_profile_begin(), "mhla_profile_begin")


def profile_end():
    """Stop collecting; {kernel name: (launches, total milliseconds)}."""
    buf = (KernelTime * 32)()
    n = ctypes.c_int32(0)
    _check(lib().mhla_profile_end(buf, 32, ctypes.byref(n)), "mhla_profile_end")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(min(n.value, 32))}


def debug_stall_waits(warp, limit_ns=1_000_000):
    """Diagnostic hook of the timeout path: warp >= 0 makes every bounded wait
    of that warp index give up after limit_ns (the kernels then stop and report
    MHLA_ERR_TIMEOUT through device_status); warp = -1 turns it off."""
    _check(lib().mhla_debug_stall_waits(int(warp), int(limit_ns)), "mhla_debug_stall_waits")


def device_status(stream=None):
    """Reads and clears the device error word; raises MhlaError on a timeout flag."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    sptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    flags = ctypes.c_uint32(0)
    st = lib().mhla_device_status(ctypes.c_void_p(sptr) if sptr else None, ctypes.byref(flags))
    _check(st, f"mhla_device_status (flags={flags.value:#x})")
    return int(flags.value)

"""Thin Python binding of libgbla.so (include/gbla.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory (outputs, workspace) and the current
CUDA stream.  There is no CPU path: if the library is missing this module
raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgbla.so")

GBLA_OK, GBLA_ERR_INVALID_ARG, GBLA_ERR_UNSUPPORTED, GBLA_ERR_WORKSPACE, GBLA_ERR_CUDA, GBLA_ERR_DEVICE_CHECK = \
    0, -1, -2, -3, -4, -5
GBLA_ERR_DEVICE_TIMEOUT = -6
GBLA_POLICY_AUTO, GBLA_POLICY_TC, GBLA_POLICY_MMA = 0, 1, 2
GBLA_F32, GBLA_BF16 = 0, 1
GBLA_GATE_SIGMOID, GBLA_GATE_SOFTMAX = 0, 1
GBLA_OP_FORWARD, GBLA_OP_BACKWARD, GBLA_OP_CORE_FORWARD, GBLA_OP_CORE_BACKWARD, GBLA_OP_DECAY_FORWARD = 0, 1, 2, 3, 4
GBLA_OP_SA_FORWARD, GBLA_OP_GLR_FORWARD, GBLA_OP_GLR_BACKWARD = 5, 6, 7

EXPORTS = ("gbla_workspace_size", "gbla_saved_size", "gbla_validate_shape", "gbla_forward", "gbla_backward",
           "bla_core_forward", "bla_core_backward", "gbla_check_device_status", "gbla_status_string",
           "gbla_last_error", "gbla_version", "gbla_profiling_enable", "gbla_profiling_read",
           "bla_core_forward_noalloc", "bla_core_noalloc_check_device_status", "gbla_diag_bounded_wait",
           "gbla_set_kernel_policy", "bla_decay_core_forward", "sa_core_forward",
           "glr_forward", "glr_backward", "glr_saved_size", "gbla_adamw_workspace_size", "gbla_grad_norm",
           "gbla_adamw_step", "embed_forward", "embed_backward", "embed_workspace_size", "layer_norm_forward",
           "layer_norm_backward", "layer_norm_workspace_size", "beam_select", "beam_workspace_size", "beam_reorder")
NOALLOC_SCRATCH_BYTES = 64 << 20
ADAMW_BLOCK = 256


class GblaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().gbla_status_string(status).decode()
        if status == GBLA_ERR_CUDA:
            msg += " (" + lib().gbla_last_error().decode() + ")"
        super().__init__(f"{what}: {msg}")


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("L", ctypes.c_int), ("d", ctypes.c_int), ("H", ctypes.c_int),
                ("d_h", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("seq_lens", ctypes.c_void_p), ("io_dtype", ctypes.c_int), ("gate", ctypes.c_int),
                ("rms_eps", ctypes.c_float)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("param_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("weight_decay", ctypes.c_double)]


class AdamWConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("max_norm", ctypes.c_double), ("seed", ctypes.c_uint32)]


class Beam(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int), ("n_out", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("eos", ctypes.c_int), ("over_allowed", ctypes.c_int)]


class BeamState(ctypes.Structure):
    _fields_ = [("dst", ctypes.c_void_p), ("src", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libgbla.so (built by build.py).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgbla.so not built ({LIB_PATH}); run generative_retrieval_encoder_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p
        sp = ctypes.POINTER(Shape)
        L.gbla_workspace_size.argtypes = [sp, ctypes.c_int]
        L.gbla_workspace_size.restype = sz
        L.gbla_saved_size.argtypes = [sp]
        L.gbla_saved_size.restype = sz
        L.gbla_validate_shape.argtypes = [sp]
        L.gbla_validate_shape.restype = ctypes.c_int
        L.gbla_forward.argtypes = [sp] + [vp] * 13 + [sz, vp]
        L.gbla_forward.restype = ctypes.c_int
        L.gbla_backward.argtypes = [sp] + [vp] * 13 + [f] * 9 + [vp, sz, vp]
        L.gbla_backward.restype = ctypes.c_int
        L.bla_core_forward.argtypes = [sp] + [vp] * 8 + [sz, vp]
        L.bla_core_forward.restype = ctypes.c_int
        L.bla_core_backward.argtypes = [sp] + [vp] * 10 + [sz, vp]
        L.bla_core_backward.restype = ctypes.c_int
        L.bla_decay_core_forward.argtypes = [sp] + [vp] * 8 + [sz, vp]
        L.bla_decay_core_forward.restype = ctypes.c_int
        L.sa_core_forward.argtypes = [sp] + [vp] * 5 + [sz, vp]
        L.sa_core_forward.restype = ctypes.c_int
        L.glr_forward.argtypes = [sp, vp, vp, vp, ctypes.c_int64, vp, ctypes.c_float, ctypes.c_int] + [vp] * 5 + [sz, vp]
        L.glr_forward.restype = ctypes.c_int
        L.glr_backward.argtypes = [sp, vp, vp, vp, ctypes.c_int64, vp, ctypes.c_float, ctypes.c_int] + [vp] * 7 + \
            [ctypes.c_int64] + [vp] * 3 + [sz, vp]
        L.glr_backward.restype = ctypes.c_int
        L.glr_saved_size.argtypes = [sp]
        L.glr_saved_size.restype = sz
        tp = ctypes.POINTER(AdamWTensor)
        L.gbla_adamw_workspace_size.argtypes = [tp, ctypes.c_int]
        L.gbla_adamw_workspace_size.restype = sz
        L.gbla_grad_norm.argtypes = [tp, ctypes.c_int, vp, vp, sz, vp]
        L.gbla_grad_norm.restype = ctypes.c_int
        L.gbla_adamw_step.argtypes = [tp, ctypes.c_int, ctypes.POINTER(AdamWConfig), vp, vp, vp, sz, vp]
        L.gbla_adamw_step.restype = ctypes.c_int
        i64, i32, fl = ctypes.c_int64, ctypes.c_int, ctypes.c_float
        L.embed_workspace_size.argtypes = [sp, i64, i32, i32]
        L.embed_workspace_size.restype = sz
        L.embed_forward.argtypes = [sp, vp, i32, i32, vp, i64, fl, vp, vp, sz, vp]
        L.embed_forward.restype = i32
        L.embed_backward.argtypes = [sp, vp, i32, i32, vp, i64, fl, vp, vp, sz, vp]
        L.embed_backward.restype = i32
        L.layer_norm_workspace_size.argtypes = [sp, i32]
        L.layer_norm_workspace_size.restype = sz
        L.layer_norm_forward.argtypes = [sp, vp, i64, vp, vp, vp, fl, vp, vp, vp, vp, sz, vp]
        L.layer_norm_forward.restype = i32
        L.layer_norm_backward.argtypes = [sp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.layer_norm_backward.restype = i32
        bp = ctypes.POINTER(Beam)
        L.beam_workspace_size.argtypes = [bp]
        L.beam_workspace_size.restype = sz
        L.beam_select.argtypes = [bp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_select.restype = i32
        L.beam_reorder.argtypes = [bp, ctypes.POINTER(BeamState), i32, vp, vp, sz, vp]
        L.beam_reorder.restype = i32
        L.bla_core_forward_noalloc.argtypes = [sp] + [vp] * 8
        L.bla_core_forward_noalloc.restype = ctypes.c_int
        L.bla_core_noalloc_check_device_status.argtypes = [vp]
        L.bla_core_noalloc_check_device_status.restype = ctypes.c_int
        L.gbla_diag_bounded_wait.argtypes = [vp, sz, ctypes.c_uint, vp]
        L.gbla_diag_bounded_wait.restype = ctypes.c_int
        L.gbla_set_kernel_policy.argtypes = [ctypes.c_int]
        L.gbla_set_kernel_policy.restype = ctypes.c_int
        L.gbla_check_device_status.argtypes = [vp, vp]
        L.gbla_check_device_status.restype = ctypes.c_int
        L.gbla_status_string.argtypes = [ctypes.c_int]
        L.gbla_status_string.restype = ctypes.c_char_p
        L.gbla_last_error.restype = ctypes.c_char_p
        L.gbla_version.restype = ctypes.c_int
        L.gbla_profiling_enable.argtypes = [ctypes.c_int]
        L.gbla_profiling_enable.restype = None
        L.gbla_profiling_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float),
                                          ctypes.c_int]
        L.gbla_profiling_read.restype = ctypes.c_int
        _lib = L
    return _lib


def make_shape(B: int, L: int, d: int, H: int, d_h: int, dtype: str = "bf16", gate: str = "sigmoid",
               eps: float = 1e-6, cu_seqlens: torch.Tensor | None = None,
               seq_lens: torch.Tensor | None = None) -> Shape:
    """Builds a gbla_shape.  cu_seqlens / seq_lens are int32 CUDA tensors (kept
    alive by the returned object).  With cu_seqlens, B = 1 and L = total rows."""
    s = Shape()
    s.B, s.L, s.d, s.H, s.d_h = B, L, d, H, d_h
    s.io_dtype = GBLA_F32 if dtype in ("f32", "fp32", torch.float32) else GBLA_BF16
    s.gate = GBLA_GATE_SOFTMAX if gate == "softmax" else GBLA_GATE_SIGMOID
    s.rms_eps = eps
    s._keep = []
    if cu_seqlens is not None:
        assert cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda
        s.cu_seqlens = cu_seqlens.data_ptr()
        s.num_seqs = cu_seqlens.numel() - 1
        s._keep.append(cu_seqlens)
    if seq_lens is not None:
        assert seq_lens.dtype == torch.int32 and seq_lens.is_cuda
        s.seq_lens = seq_lens.data_ptr()
        s._keep.append(seq_lens)
    return s


def io_dtype(shape: Shape) -> torch.dtype:
    return torch.float32 if shape.io_dtype == GBLA_F32 else torch.bfloat16


def rows(shape: Shape) -> int:
    return shape.L if shape.cu_seqlens else shape.B * shape.L


def n_seq(shape: Shape) -> int:
    return shape.num_seqs if shape.cu_seqlens else shape.B


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, what: str):
    if status != GBLA_OK:
        raise GblaError(status, what)


def gbla_workspace_size(shape: Shape, op: int) -> int:
    return lib().gbla_workspace_size(ctypes.byref(shape), op)


def gbla_saved_size(shape: Shape) -> int:
    return lib().gbla_saved_size(ctypes.byref(shape))


def gbla_validate_shape(shape: Shape) -> int:
    return lib().gbla_validate_shape(ctypes.byref(shape))


def workspace(shape: Shape, op: int, device="cuda") -> torch.Tensor:
    n = gbla_workspace_size(shape, op)
    if n == 0 and op in (GBLA_OP_GLR_FORWARD, GBLA_OP_GLR_BACKWARD):
        _check(GBLA_ERR_INVALID_ARG, "gbla_workspace_size")
    if n == 0:
        _check(gbla_validate_shape(shape) or GBLA_ERR_INVALID_ARG, "gbla_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


PARAMS = ("conv_w", "conv_b", "W_q", "W_k", "W_v", "W_r", "w_g", "b_g", "rms_w")


def gbla_forward(shape: Shape, x: torch.Tensor, params: dict, y: torch.Tensor | None = None,
                 saved: torch.Tensor | bool | None = None, ws: torch.Tensor | None = None):
    """Layer forward.  Returns (y, saved); pass saved=True to allocate the
    activation buffer that gbla_backward needs."""
    if y is None:
        y = torch.empty(rows(shape), shape.H * shape.d_h, dtype=io_dtype(shape), device=x.device)
    if saved is True:
        saved = torch.empty(gbla_saved_size(shape), dtype=torch.uint8, device=x.device)
    if ws is None:
        ws = workspace(shape, GBLA_OP_FORWARD, x.device)
    P = [params.get(n) for n in PARAMS]
    st = lib().gbla_forward(ctypes.byref(shape), _ptr(x), *[_ptr(p) for p in P], _ptr(y),
                            _ptr(saved if isinstance(saved, torch.Tensor) else None), _ptr(ws), ws.numel(), _stream())
    _check(st, "gbla_forward")
    return y, (saved if isinstance(saved, torch.Tensor) else None)


def gbla_backward(shape: Shape, x: torch.Tensor, params: dict, saved: torch.Tensor, dy: torch.Tensor,
                  ws: torch.Tensor | None = None, out: dict | None = None) -> dict:
    """Layer backward for <dy, y>.  Returns dx (io dtype) and fp32 parameter
    gradients d<name>."""
    dev = x.device
    d, H, dh = shape.d, shape.H, shape.d_h
    f = dict(dtype=torch.float32, device=dev)
    g = out if out is not None else {
        "dx": torch.empty_like(x), "dconv_w": torch.empty(d, 4, **f), "dconv_b": torch.empty(d, **f),
        "dW_q": torch.empty(d, H * dh, **f), "dW_k": torch.empty(d, H * dh, **f),
        "dW_v": torch.empty(d, H * dh, **f), "dW_r": torch.empty(d, H * dh, **f),
        "dw_g": torch.empty(d, H, **f), "db_g": torch.empty(H, **f), "drms_w": torch.empty(dh, **f)}
    if ws is None:
        ws = workspace(shape, GBLA_OP_BACKWARD, dev)
    P = [params.get(n) for n in PARAMS]
    names = ("dconv_w", "dconv_b", "dW_q", "dW_k", "dW_v", "dW_r", "dw_g", "db_g", "drms_w")
    st = lib().gbla_backward(ctypes.byref(shape), _ptr(x), *[_ptr(p) for p in P], _ptr(saved), _ptr(dy),
                             _ptr(g["dx"]), *[_ptr(g.get(n)) for n in names], _ptr(ws), ws.numel(), _stream())
    _check(st, "gbla_backward")
    return g


def bla_core_forward(shape: Shape, q, k, v, g, o=None, den=None, state=None, ws=None):
    """The gated BLA core alone: returns (o, den, state); den/state are filled
    when tensors are passed (True allocates them)."""
    dev = q.device
    if o is None:
        o = torch.empty_like(q)
    if den is True:
        den = torch.empty(rows(shape), shape.H, dtype=torch.float32, device=dev)
    if state is True:
        state = torch.empty(n_seq(shape), shape.H, shape.d_h, shape.d_h + 1, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(shape, GBLA_OP_CORE_FORWARD, dev)
    st = lib().bla_core_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o),
                                _ptr(den if isinstance(den, torch.Tensor) else None),
                                _ptr(state if isinstance(state, torch.Tensor) else None), _ptr(ws), ws.numel(),
                                _stream())
    _check(st, "bla_core_forward")
    return o, den, state


def bla_decay_core_forward(shape: Shape, q, k, v, g, lam, o=None, den=None, ws=None):
    """The core under LION's decay masks (see gbla.h): returns (o, den)."""
    dev = q.device
    if o is None:
        o = torch.empty_like(q)
    if den is True:
        den = torch.empty(rows(shape), shape.H, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(shape, GBLA_OP_DECAY_FORWARD, dev)
    st = lib().bla_decay_core_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lam), _ptr(o),
                                      _ptr(den if isinstance(den, torch.Tensor) else None), _ptr(ws), ws.numel(),
                                      _stream())
    _check(st, "bla_decay_core_forward")
    return o, den


def sa_core_forward(shape: Shape, q, k, v, o=None, ws=None):
    """The bidirectional softmax attention of the SA blocks (Eq. 1, see gbla.h): returns o."""
    if o is None:
        o = torch.empty_like(q)
    if ws is None:
        ws = workspace(shape, GBLA_OP_SA_FORWARD, q.device)
    st = lib().sa_core_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(ws), ws.numel(),
                               _stream())
    _check(st, "sa_core_forward")
    return o


def glr_shape(B: int, L: int, d: int, dtype: str = "bf16", cu_seqlens: torch.Tensor | None = None,
              seq_lens: torch.Tensor | None = None) -> Shape:
    """make_shape for the gated linear recurrence, which has channels but no heads."""
    for name, t, n in (("cu_seqlens", cu_seqlens, 2), ("seq_lens", seq_lens, B)):
        if t is not None and (t.dtype != torch.int32 or not t.is_cuda or t.dim() != 1 or not t.is_contiguous()
                              or (t.numel() < n if name == "cu_seqlens" else t.numel() != n)):
            raise ValueError(f"{name}: want a contiguous int32 CUDA tensor of {n} values{' at least' if n == 2 else ''}, "
                             f"got {t.dtype} {list(t.shape)} on {t.device}")
    return make_shape(B, L, d, 1, 1, dtype=dtype, cu_seqlens=cu_seqlens, seq_lens=seq_lens)


def glr_saved_size(shape: Shape) -> int:
    return lib().glr_saved_size(ctypes.byref(shape))


def _glr_arg(name, t, n, d, dtype, device, ld):
    """t's address.  Raises unless t is an [n, d] tensor of this dtype and device with contiguous rows of stride ld."""
    if t.dtype is not dtype or t.device != device or t.shape != (n, d):
        raise ValueError(f"{name}: want {dtype} {[n, d]} on {device}, got {t.dtype} {list(t.shape)} on {t.device}")
    if t.stride() != (ld, 1) and (n > 1 and t.stride(0) != ld or d > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: strides {t.stride()}, want {(ld, 1)}: rows are contiguous, and of one stride in x, r and i, "
                         "in dx, dr and di, and d in all else")
    return t.data_ptr()


def _glr_vec(name, t, d, device):
    if t.dtype is not torch.float32 or t.device != device or t.shape != (d,) or (d > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: want contiguous fp32 [{d}] on {device}, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _glr_bytes(name, t, n, device):
    if t.device != device or not t.is_contiguous() or t.numel() * t.element_size() < n:
        raise ValueError(f"{name}: want {n} contiguous bytes on {device}, got {t.numel() * t.element_size()} on {t.device}")
    return t.data_ptr()


def _glr_inputs(shape, x, r, i, lam, h0):
    T, N, d, io = rows(shape), n_seq(shape), shape.d, io_dtype(shape)
    dev = x.device
    if not x.is_cuda:
        raise ValueError(f"x: want a CUDA tensor, got {x.device}")
    ld = x.stride(0) if T > 1 and x.dim() == 2 else d
    return (dev, T, N, d, ld, _glr_arg("x", x, T, d, io, dev, ld), _glr_arg("r", r, T, d, io, dev, ld), _glr_arg("i", i, T, d, io, dev, ld),
            _glr_vec("lam", lam, d, dev), None if h0 is None else _glr_arg("h0", h0, N, d, torch.float32, dev, d))


# The current stream's handle of a device (by index): torch's own short way where it has one, 2 us less a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(device, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    if device.index == torch.cuda.current_device():
        return fn(*args, _raw_stream(device.index))
    with torch.cuda.device(device):
        return fn(*args, _raw_stream(device.index))


def glr_forward(shape: Shape, x, r, i, lam, c: float = 8.0, reverse: bool = False, h0=None, y=None, hT=None,
                saved: torch.Tensor | bool | None = None, ws=None):
    """The gated linear recurrence (see gbla.h): returns (y, hT, saved).  x, r and i share their row stride (they may
    be columns of one tensor).  hT: a tensor to fill (h0 itself to update it in place), or True to allocate it; saved =
    True allocates what glr_backward needs.  Tensors are on x's device, the call on that device's current stream."""
    dev, T, N, d, ld, px, pr, pi, pl, ph = _glr_inputs(shape, x, r, i, lam, h0)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=dev)
    py = _glr_arg("y", y, T, d, x.dtype, dev, d)
    if hT is True:
        hT = torch.empty((N, d), dtype=torch.float32, device=dev)
    pT = None if hT is None else ph if hT is h0 else _glr_arg("hT", hT, N, d, torch.float32, dev, d)
    if saved is True:
        saved = torch.empty(glr_saved_size(shape), dtype=torch.uint8, device=dev)
    saved = saved if isinstance(saved, torch.Tensor) else None
    ps = None if saved is None else _glr_bytes("saved", saved, glr_saved_size(shape), dev)
    if ws is None:
        ws = workspace(shape, GBLA_OP_GLR_FORWARD, dev)
    st = _call(dev, lib().glr_forward, ctypes.byref(shape), px, pr, pi, ld, pl, c, int(reverse), ph, py, pT, ps,
               _glr_bytes("ws", ws, 0, dev), ws.numel() * ws.element_size())
    if st != GBLA_OK:
        raise GblaError(st, "glr_forward")
    return y, hT, saved


def glr_backward(shape: Shape, x, r, i, lam, saved, dy, c: float = 8.0, reverse: bool = False, h0=None, dhT=None,
                 ws=None, out: dict | None = None) -> dict:
    """Backward of glr_forward for <dy, y> + <dhT, hT>.  Returns dx, dr, di (io dtype), dlam fp32 and, where h0 or dhT
    is given, dh0 fp32.  out: tensors to fill (dx, dr and di of one row stride)."""
    dev, T, N, d, ld, px, pr, pi, pl, ph = _glr_inputs(shape, x, r, i, lam, h0)
    f32 = torch.float32
    g = out
    if g is None:
        g = {n: torch.empty((T, d), dtype=x.dtype, device=dev) for n in ("dx", "dr", "di")}
        g["dlam"] = torch.empty(d, dtype=f32, device=dev)
        if h0 is not None or dhT is not None:
            g["dh0"] = torch.empty((N, d), dtype=f32, device=dev)
    ldd = g["dx"].stride(0) if T > 1 and g["dx"].dim() == 2 else d
    pg = [_glr_arg(n, g[n], T, d, x.dtype, dev, ldd) for n in ("dx", "dr", "di")]
    dl, dh = g.get("dlam"), g.get("dh0")
    if ws is None:
        ws = workspace(shape, GBLA_OP_GLR_BACKWARD, dev)
    st = _call(dev, lib().glr_backward, ctypes.byref(shape), px, pr, pi, ld, pl, c, int(reverse), ph,
               _glr_bytes("saved", saved, glr_saved_size(shape), dev), _glr_arg("dy", dy, T, d, x.dtype, dev, d),
               None if dhT is None else _glr_arg("dhT", dhT, N, d, f32, dev, d), *pg, ldd,
               None if dl is None else _glr_vec("dlam", dl, d, dev), None if dh is None else _glr_arg("dh0", dh, N, d, f32, dev, d),
               _glr_bytes("ws", ws, 0, dev), ws.numel() * ws.element_size())
    if st != GBLA_OK:
        raise GblaError(st, "glr_backward")
    return g


_ADAMW_DTYPE = {torch.float32: GBLA_F32, torch.bfloat16: GBLA_BF16}
_ADAMW_ROW = np.dtype([(n, {ctypes.c_void_p: np.uint64, ctypes.c_int64: np.int64, ctypes.c_int: np.int32, ctypes.c_double: np.float64}[t])
                       for n, t in AdamWTensor._fields_], align=True)


def _named(tensors):
    """(names or None, list) of a dict or a sequence of tensors."""
    return (list(tensors), list(tensors.values())) if isinstance(tensors, dict) else (None, list(tensors))


def gbla_adamw_state(params, bits: int = 32, master: bool | None = None) -> dict:
    """The state of an AdamW run over params (a dict or a sequence), before its first step: step (int64 [1]), m and v per
    parameter, fp32 (bits = 32) or e4m3 with m_scale and v_scale (bits = 8), and, where a parameter is bf16 (master =
    False: nowhere), master, the fp32 copy it is rounded from."""
    if bits not in (8, 32):
        raise ValueError(f"bits: 8 or 32, got {bits}")
    P = _named(params)[1]
    dev = P[0].device if P else torch.device("cuda", torch.cuda.current_device())
    dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
    zeros = lambda n, t: torch.zeros(n, dtype=torch.uint8 if t is torch.float8_e4m3fn else t, device=dev).view(t)  # noqa: E731
    s = {"step": torch.zeros(1, dtype=torch.int64, device=dev), "m": [zeros(p.numel(), dt) for p in P],
         "v": [zeros(p.numel(), dt) for p in P]}
    if bits == 8:
        for k in ("m_scale", "v_scale"):
            s[k] = [zeros(-(-p.numel() // ADAMW_BLOCK), torch.float32) for p in P]
    if master is not False:
        s["master"] = [p.detach().float() if p.dtype == torch.bfloat16 else None for p in P]
    return s


class AdamWPlan:
    """Which tensors an AdamW step updates, by which gradients and states (gbla_adamw_plan); it keeps them alive, also where
    the caller puts others in their place (which another plan is needed for)."""

    def __init__(self, params, grads, state):
        names, P = _named(params)
        self.names, self.n, self.step = names, len(P), state["step"]
        self.device = self.step.device
        if self.step.dtype != torch.int64 or self.step.numel() != 1 or not self.step.is_cuda:
            raise ValueError(f"step: want one int64 on a CUDA device, got {self.step.dtype} on {self.step.device}")
        self.sizes = [p.numel() for p in P]
        none = [None] * self.n
        M, V, MS, VS, MA = (list(state.get(k) or none) for k in ("m", "v", "m_scale", "v_scale", "master"))
        self._keep, self._decay = [P, M, V, MS, VS, MA], None  # the lists' own copies: the caller's may change
        for k, t in (("m", M), ("v", V), ("m_scale", MS), ("v_scale", VS), ("master", MA)):
            if len(t) != self.n:
                raise ValueError(f"{k}: {len(t)} tensors for {self.n} parameters")
        written = [(self.step.data_ptr(), 8, "step")]
        blocks = [-(-n // ADAMW_BLOCK) for n in self.sizes]
        kind = [torch.float32 if s is None else torch.float8_e4m3fn for s in MS]
        cols = {"param": self._column("parameter", P, self.sizes, None, written),
                "m": self._column("m", M, self.sizes, kind, written), "v": self._column("v", V, self.sizes, kind, written),
                "m_scale": self._column("m_scale", MS, blocks, [torch.float32] * self.n, written, VS),
                "v_scale": self._column("v_scale", VS, blocks, [torch.float32] * self.n, written, MS),
                "master": self._column("master", MA, self.sizes, [torch.float32] * self.n, written, MA)}
        for p, t in zip(P, MA):
            if t is not None and p.dtype is not torch.bfloat16:
                raise ValueError("master: only a bf16 parameter has one")
        written.sort()
        end, who = 0, None
        for at, size, name in written:
            if at < end:
                raise ValueError(f"{who} and {name} overlap")
            end, who = at + size, name
        self.tensors = (AdamWTensor * self.n)()
        self._rows = np.frombuffer(self.tensors, dtype=_ADAMW_ROW) if self.n else np.empty(0, _ADAMW_ROW)
        for k, col in cols.items():
            self._rows[k] = col
        self._rows["n"] = self.sizes
        self._rows["param_dtype"] = [_ADAMW_DTYPE[p.dtype] for p in P]
        self.set_grads(grads)
        size = lib().gbla_adamw_workspace_size(self.tensors, self.n)
        if size == 0:
            _check(GBLA_ERR_INVALID_ARG, "gbla_adamw_workspace_size")
        self.ws = torch.empty(size, dtype=torch.uint8, device=self.device)

    def _column(self, what, tensors, sizes, dtypes, written=None, like=None):
        """The addresses of one tensor for every parameter; dtypes: what each has to be (None: fp32 or bf16); where `like` is
        given a parameter may have none, if it has none of `like` either."""
        dev, col = self.device, []
        for j, (t, n) in enumerate(zip(tensors, sizes)):
            if t is None and like is not None and like[j] is None:
                col.append(0)
                continue
            if (t is None or t.numel() != n or t.device != dev or not t.is_contiguous()
                    or (t.dtype not in _ADAMW_DTYPE if dtypes is None else t.dtype is not dtypes[j])):
                want = "fp32 or bf16" if dtypes is None else dtypes[j]
                got = "none" if t is None else f"{list(t.shape)} {t.dtype} on {t.device}"
                raise ValueError(f"{what} of {self.names[j] if self.names else j}: want {n} contiguous values of {want} on {dev}, got {got}")
            at = t.data_ptr() if n else 0
            col.append(at)
            if n and written is not None:
                written.append((at, n * t.element_size(), what))
        return col

    def set_grads(self, grads):
        """Other gradient tensors for the same parameters: a sequence in their order, or a dict by their names (with or
        without the leading d of gbla_backward's: d<name> first, unless another parameter has that name).  A captured call
        keeps to those of its capture, which are the caller's to keep."""
        if isinstance(grads, dict):
            if self.names is None:
                raise ValueError("grads by name need params by name")
            G, taken = [], set(self.names)
            for k in self.names:
                at = "d" + k if "d" + k in grads and "d" + k not in taken else k
                if at not in grads:
                    raise ValueError(f"no gradient of {k}")
                G.append(grads[at])
        else:
            G = list(grads)
        if len(G) != self.n:
            raise ValueError(f"{len(G)} gradients for {self.n} parameters")
        self._rows["grad"] = self._column("gradient", G, self.sizes, None)
        self._rows["grad_dtype"] = [_ADAMW_DTYPE[g.dtype] for g in G]
        self._grads = G


def gbla_adamw_plan(params, grads, state: dict) -> AdamWPlan:
    """The plan of AdamW steps on params (a dict or a sequence of fp32 or bf16 tensors) by grads (fp32 or bf16; a dict
    may be gbla_backward's) with a state of gbla_adamw_state.  Its workspace orders its calls on one stream."""
    return AdamWPlan(params, grads, state)


def gbla_grad_norm(plan: AdamWPlan, norm: torch.Tensor | None = None) -> torch.Tensor:
    """The global 2-norm of the plan's gradients (fp32, on the device)."""
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=plan.device)
    else:
        plan._column("norm", [norm], [1], [torch.float32])
    _check(_call(plan.device, lib().gbla_grad_norm, plan.tensors, plan.n, norm.data_ptr(), plan.ws.data_ptr(), plan.ws.numel()),
           "gbla_grad_norm")
    return norm


def gbla_adamw_step(plan: AdamWPlan, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                    norm: torch.Tensor | None = None, max_norm: float | None = None, seed: int = 0) -> None:
    """One AdamW step of the plan's tensors, in place (see gbla.h).  weight_decay: one value, or one per parameter; norm:
    gbla_grad_norm's, which gradients are clipped by (max_norm) and which skips the step where it is not finite; seed: of
    the 8-bit states' rounding."""
    if norm is not None:
        plan._column("norm", [norm], [1], [torch.float32])
    if max_norm is not None and norm is None:
        raise ValueError("max_norm needs norm (gbla_grad_norm)")
    wd = tuple(weight_decay) if isinstance(weight_decay, (list, tuple)) else weight_decay
    if wd != plan._decay:
        each = wd if isinstance(wd, tuple) else (wd,) * plan.n
        if len(each) != plan.n:
            raise ValueError(f"weight_decay: {len(each)} values for {plan.n} parameters")
        plan._rows["weight_decay"] = each
        plan._decay = wd
    cfg = AdamWConfig(lr, betas[0], betas[1], eps, max_norm or 0.0, seed)
    _check(_call(plan.device, lib().gbla_adamw_step, plan.tensors, plan.n, ctypes.byref(cfg), plan.step.data_ptr(),
                 None if norm is None else norm.data_ptr(), plan.ws.data_ptr(), plan.ws.numel()), "gbla_adamw_step")


def _arg(name, t, shape, dtype, device):
    """t's address (None: of none).  Raises unless t is a contiguous tensor of this shape, dtype and device."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: want contiguous {dtype} {list(shape)} on {device}, got {t.dtype} {list(t.shape)} with strides "
                     f"{t.stride()} on {t.device}")


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name}: want a CUDA tensor, got {t.device}")
    return t.device


def _ws(ws, device):
    """A workspace's address and bytes."""
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws: want contiguous bytes on {device}, got strides {ws.stride()} on {ws.device}")
    return ws.data_ptr(), ws.nbytes


# Outputs that a call allocates need no check: (tensor, its address).
def _new(shape, dtype, device):
    t = torch.empty(shape, dtype=dtype, device=device)
    return t, t.data_ptr()


def embed_workspace_size(shape: Shape, vocab: int, k: int = 1, backward: bool = False) -> int:
    return lib().embed_workspace_size(ctypes.byref(shape), vocab, k, int(backward))


def embed_workspace(shape: Shape, vocab: int, k: int = 1, backward: bool = False, device="cuda") -> torch.Tensor:
    n = embed_workspace_size(shape, vocab, k, backward)
    if n == 0:
        _check(GBLA_ERR_INVALID_ARG, "embed_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _embed_ids(shape, ids):
    dev, T = _cuda("ids", ids), rows(shape)
    k = ids.shape[1] if ids.dim() == 2 else 1
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() not in (1, 2) or ids.shape[0] != T or k < 1 or not ids.is_contiguous():
        raise ValueError(f"ids: want contiguous int32 or int64 [{T}] or [{T}, k], got {ids.dtype} {list(ids.shape)}")
    return dev, T, k, ids.data_ptr(), int(ids.dtype is torch.int64)


def embed_forward(shape: Shape, ids, table, scale: float = 1.0, y=None, ws=None):
    """Rows of table [V, d] by ids [rows] or [rows, k] (int32 or int64; below 0: none), times scale (see gbla.h): returns y
    [rows, k d].  shape: glr_shape or make_shape, whose d is the width of a table row."""
    dev, T, k, pi, wide = _embed_ids(shape, ids)
    io, d = io_dtype(shape), shape.d
    if table.dim() != 2:
        raise ValueError(f"table: want [V, {d}], got {list(table.shape)}")
    V = table.shape[0]
    pt = _arg("table", table, (V, d), io, dev)
    if y is None:
        y, py = _new((T, k * d), io, dev)
    else:
        py = _arg("y", y, (T, k * d), io, dev)
    if ws is None:
        ws = torch.empty(256, dtype=torch.uint8, device=dev)  # the error word alone
    st = _call(dev, lib().embed_forward, ctypes.byref(shape), pi, wide, k, pt, V, scale, py, *_ws(ws, dev))
    if st != GBLA_OK:
        raise GblaError(st, "embed_forward")
    return y


def embed_backward(shape: Shape, ids, dy, vocab: int, scale: float = 1.0, dtable=None, ws=None):
    """The table's gradient for <dy, y>: fp32 [vocab, d], rows without a token 0."""
    dev, T, k, pi, wide = _embed_ids(shape, ids)
    d = shape.d
    pd = _arg("dy", dy, (T, k * d), io_dtype(shape), dev)
    if dtable is None:
        dtable, pg = _new((vocab, d), torch.float32, dev)
    else:
        pg = _arg("dtable", dtable, (vocab, d), torch.float32, dev)
    if ws is None:
        ws = embed_workspace(shape, vocab, k, True, dev)
    st = _call(dev, lib().embed_backward, ctypes.byref(shape), pi, wide, k, pd, vocab, scale, pg, *_ws(ws, dev))
    if st != GBLA_OK:
        raise GblaError(st, "embed_backward")
    return dtable


def layer_norm_workspace_size(shape: Shape, backward: bool = False) -> int:
    return lib().layer_norm_workspace_size(ctypes.byref(shape), int(backward))


def layer_norm_workspace(shape: Shape, backward: bool = False, device="cuda") -> torch.Tensor:
    n = layer_norm_workspace_size(shape, backward)
    if n == 0:
        _check(GBLA_ERR_INVALID_ARG, "layer_norm_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _norm_input(shape, x):
    """(device, rows, d, io dtype, row stride, address) of what is normed: rows of any stride."""
    dev, T, d, io = _cuda("x", x), rows(shape), shape.d, io_dtype(shape)
    ld = x.stride(0) if T > 1 and x.dim() == 2 else d
    return dev, T, d, io, ld, _glr_arg("x", x, T, d, io, dev, ld)


def layer_norm_forward(shape: Shape, x, w=None, b=None, eps: float = 1e-5, res=None, total: torch.Tensor | bool | None = None, y=None,
                       stats: torch.Tensor | bool | None = None, ws=None):
    """Layer norm of x, or of x + res (see gbla.h): returns (y, total, stats).  total: x + res as it is normed, allocated
    where there is a res (False: not wanted; res itself, or x, to update it in place); stats = True allocates what
    layer_norm_backward needs."""
    dev, T, d, io, ld, px = _norm_input(shape, x)
    full, f32 = (T, d), torch.float32
    if y is None:
        y, py = _new(full, io, dev)
    else:
        py = _arg("y", y, full, io, dev)
    if total is True or (total is None and res is not None):
        total, pt = _new(full, io, dev)
    else:
        total = None if total is False else total
        pt = _arg("total", total, full, io, dev)
    if stats is True:
        stats, ps = _new((T, 2), f32, dev)
    else:
        stats = None if stats is False else stats
        ps = _arg("stats", stats, (T, 2), f32, dev)
    if ws is None:
        ws = torch.empty(256, dtype=torch.uint8, device=dev)  # the error word alone
    st = _call(dev, lib().layer_norm_forward, ctypes.byref(shape), px, ld, _arg("res", res, full, io, dev), _arg("w", w, (d,), io, dev),
               _arg("b", b, (d,), io, dev), eps, pt, py, ps, *_ws(ws, dev))
    if st != GBLA_OK:
        raise GblaError(st, "layer_norm_forward")
    return y, total, stats


def layer_norm_backward(shape: Shape, x, w, stats, dy, ds=None, affine: bool = True, ws=None, out: dict | None = None) -> dict:
    """Backward of layer_norm_forward for <dy, y> + <ds, total>: x is what was normed (total, where there was a res).  Returns
    dx (the gradient of x and of res) and, with affine, dw and db fp32.  out: tensors to fill (dx may be ds)."""
    dev, T, d, io, ld, px = _norm_input(shape, x)
    full, f32 = (T, d), torch.float32
    if out is None:
        dx, pdx = _new(full, io, dev)
        g = {"dx": dx}
        pdw = pdb = None
        if affine:
            g["dw"], pdw = _new(d, f32, dev)
            g["db"], pdb = _new(d, f32, dev)
    else:
        g = out
        pdx, pdw, pdb = (_arg("dx", g["dx"], full, io, dev), _arg("dw", g.get("dw"), (d,), f32, dev), _arg("db", g.get("db"), (d,), f32, dev))
    if ws is None:
        ws = layer_norm_workspace(shape, True, dev)
    if stats is None:
        raise ValueError("stats: layer_norm_forward's (stats = True)")
    st = _call(dev, lib().layer_norm_backward, ctypes.byref(shape), px, ld, _arg("w", w, (d,), io, dev), _arg("stats", stats, (T, 2), f32, dev),
               _arg("dy", dy, full, io, dev), _arg("ds", ds, full, io, dev), pdx, pdw, pdb, *_ws(ws, dev))
    if st != GBLA_OK:
        raise GblaError(st, "layer_norm_backward")
    return g


def beam_shape(B: int, K: int, V: int, n_out: int | None = None, dtype: str = "bf16", eos: int = -1, over_allowed: bool = False) -> Beam:
    """A step of beam search over B groups of K beams and V tokens, of which n_out (K) beams go on; dtype: of the logits."""
    return Beam(B, K, V, K if n_out is None else n_out, GBLA_F32 if dtype in ("f32", "fp32", torch.float32) else GBLA_BF16, eos,
                int(over_allowed))


def beam_workspace_size(beam: Beam) -> int:
    return lib().beam_workspace_size(ctypes.byref(beam))


def beam_workspace(beam: Beam, device="cuda") -> torch.Tensor:
    n = beam_workspace_size(beam)
    if n == 0:
        _check(GBLA_ERR_INVALID_ARG, "beam_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def beam_select(beam: Beam, logits, scores, allowed=None, done=None, out: tuple | None = None, ws=None):
    """The n_out best of each group's K x V candidates (see gbla.h): returns (scores, tokens, parents, done), each [B, n_out],
    done (bool) where beam has an eos.  logits [B K, V] of any row stride; scores fp32 [B, K]; allowed int32 [B K,
    ceil(V / 32)], the bits of the tokens that may follow; done bool [B, K].  out: such a tuple to fill, of other tensors than
    the inputs."""
    B, K, V, n = beam.B, beam.K, beam.V, beam.n_out
    dev, dt = _cuda("logits", logits), torch.float32 if beam.io_dtype == GBLA_F32 else torch.bfloat16
    ld = logits.stride(0) if B * K > 1 and logits.dim() == 2 else V
    pl = _glr_arg("logits", logits, B * K, V, dt, dev, ld)
    if out is None:
        shape, i32 = (B, n), torch.int32
        s, ps = _new(shape, torch.float32, dev)
        t, pt = _new(shape, i32, dev)
        p, pp = _new(shape, i32, dev)
        e, pe = _new(shape, torch.bool, dev) if beam.eos >= 0 else (None, None)
        out = (s, t, p, e)
    else:
        ps, pt, pp, pe = (_arg(name, t, (B, n), kind, dev) for name, t, kind in
                          zip(("scores", "tokens", "parents", "done"), out, (torch.float32, torch.int32, torch.int32, torch.bool)))
    if ws is None:
        ws = beam_workspace(beam, dev)
    st = _call(dev, lib().beam_select, ctypes.byref(beam), pl, ld, _arg("scores", scores, (B, K), torch.float32, dev),
               _arg("allowed", allowed, (B * K, -(-V // 32)), torch.int32, dev), _arg("done", done, (B, K), torch.bool, dev), ps, pt, pp, pe,
               *_ws(ws, dev))
    if st != GBLA_OK:
        raise GblaError(st, "beam_select")
    return out


class BeamReorderPlan:
    """Which tensors follow their beams' parents (beam_reorder_plan); it keeps them alive."""

    def __init__(self, beam: Beam, states, out=None):
        S, D = list(states), list(states if out is None else out)
        if len(S) != len(D):
            raise ValueError(f"{len(D)} tensors to fill for {len(S)} states")
        if out is None and beam.n_out != beam.K:
            raise ValueError(f"in place needs as many beams out ({beam.n_out}) as in ({beam.K})")
        self.beam, self.B, self.n = Beam.from_buffer_copy(beam), beam.B, beam.n_out  # a copy: the caller's may change
        self.device = _cuda("state", S[0]) if S else torch.device("cuda", torch.cuda.current_device())
        self._keep = (S, D)
        self.states = (BeamState * len(S))()
        taken = []
        for j, (a, b) in enumerate(zip(S, D)):
            row = a.numel() // (beam.B * beam.K) * a.element_size()
            for name, t, n in (("state", a, beam.B * beam.K), ("tensor to fill", b, beam.B * beam.n_out)):
                if t.device != self.device or t.dtype is not a.dtype or not t.is_contiguous() or t.numel() * t.element_size() != n * row:
                    raise ValueError(f"{name} {j}: want {n} contiguous rows of {row} bytes of {a.dtype} on {self.device}, got {t.dtype} "
                                     f"{list(t.shape)} on {t.device}")
            if row:
                taken.append((a.data_ptr(), beam.B * beam.K * row, f"state {j}"))
                if out is not None:
                    taken.append((b.data_ptr(), beam.B * beam.n_out * row, f"tensor to fill {j}"))
            self.states[j] = BeamState(b.data_ptr() if row else None, a.data_ptr() if row else None, row)
        taken.sort()
        for (at, size, who), (nxt, _, name) in zip(taken, taken[1:]):
            if nxt < at + size:
                raise ValueError(f"{who} and {name} overlap")
        self.ws = torch.empty(256, dtype=torch.uint8, device=self.device)
        self._ws, self._beam = self.ws.data_ptr(), ctypes.byref(self.beam)


def beam_reorder_plan(beam: Beam, states, out=None) -> BeamReorderPlan:
    """The plan of moving states (tensors of B K rows; the rows' shape and type are free) to where beam_select's parents send
    them: in place (n_out = K), or into out (tensors of B n_out rows).  Its workspace orders its calls on one stream."""
    return BeamReorderPlan(beam, states, out)


def beam_reorder(plan: BeamReorderPlan, parents) -> None:
    """Row [b, i] of each of the plan's tensors becomes the state's row [b, parents[b, i]] (see gbla.h)."""
    st = _call(plan.device, lib().beam_reorder, plan._beam, plan.states, len(plan.states),
               _arg("parents", parents, (plan.B, plan.n), torch.int32, plan.device), plan._ws, 256)
    if st != GBLA_OK:
        raise GblaError(st, "beam_reorder")


def bla_core_forward_noalloc(shape: Shape, q, k, v, g, o, den=None, state=None) -> int:
    """bla_core_forward with the library's fixed 64 MiB device scratch instead
    of a workspace, for callers that cannot allocate; o (and den / state when
    given) must already exist.  Returns the status (GBLA_ERR_WORKSPACE when the
    shape needs more scratch than the fixed array holds)."""
    return lib().bla_core_forward_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o),
                                          _ptr(den), _ptr(state), _stream())


def bla_core_backward(shape: Shape, q, k, v, g, d_o, ws=None):
    """Backward of bla_core_forward for <d_o, o>: returns (dq, dk, dv, dg)."""
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty(rows(shape), shape.H, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(shape, GBLA_OP_CORE_BACKWARD, q.device)
    st = lib().bla_core_backward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(d_o), _ptr(dq),
                                 _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ws), ws.numel(), _stream())
    _check(st, "bla_core_backward")
    return dq, dk, dv, dg


def gbla_check_device_status(ws: torch.Tensor) -> int:
    return lib().gbla_check_device_status(_ptr(ws), _stream())


def bla_core_noalloc_check_device_status() -> int:
    """The error word of the last bla_core_forward_noalloc call on the current device."""
    return lib().bla_core_noalloc_check_device_status(_stream())


def gbla_diag_bounded_wait(ws: torch.Tensor, polls: int = 4096) -> int:
    """Runs the kernels' bounded mbarrier wait out on purpose (see gbla.h)."""
    return lib().gbla_diag_bounded_wait(_ptr(ws), ws.numel(), polls, _stream())


def gbla_set_kernel_policy(policy: int) -> None:
    """GBLA_POLICY_AUTO (default), GBLA_POLICY_TC or GBLA_POLICY_MMA for this thread's later calls (see gbla.h)."""
    _check(lib().gbla_set_kernel_policy(policy), "gbla_set_kernel_policy")


def gbla_profiling_enable(on: bool) -> None:
    lib().gbla_profiling_enable(1 if on else 0)


def gbla_profiling_read(cap: int = 4096) -> list[tuple[str, float]]:
    """(launch name, milliseconds) for every launch since the last read."""
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_float * cap)()
    n = lib().gbla_profiling_read(names, ms, cap)
    return [(names[i].decode(), float(ms[i])) for i in range(min(n, cap))]

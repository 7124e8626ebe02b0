"""S5 layer forward hot path on AMD MI355X (gfx950): Python binding.

Thin ctypes layer over the C ABI in include/s5.h (libs5.so, built in-tree by
``diagonal_state_space_amd.build_lib``). It only marshals arguments: checks
device, dtype, shape and contiguity of torch tensors, passes their device
pointers and the current HIP stream, and turns status codes into exceptions.
Every step of the computation runs in the library's kernels; PyTorch provides
device memory and streams. There is no fallback: if libs5.so is missing or a
GPU is not present, the calls raise.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "S5Error",
    "S5_F32",
    "S5_BF16",
    "S5_MAX_P",
    "S5_MAX_H",
    "lib",
    "lib_path",
    "discretize",
    "forward",
    "forward_timevarying",
    "forward_stateful",
    "forward_timevarying_stateful",
    "set_profiling_events",
    "status_string",
    "gated_delta",
    "gated_delta_backward",
    "gated_delta_step",
    "qk_norm_rope",
    "qk_norm_rope_backward",
    "rope_frequencies",
]

S5_F32 = 0
S5_BF16 = 1
S5_MAX_P = 256
S5_MAX_H = 512

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libs5.so")
_lib = None

EXPORTS = ("s5_discretize", "s5_forward", "s5_forward_noalloc", "s5_forward_timevarying", "s5_forward_stateful",
           "s5_forward_timevarying_stateful", "s5_forward_ex", "s5_step", "s5_glu", "s5_status_string",
           "s5_set_profiling_events", "s5_gated_delta_workspace", "s5_gated_delta", "s5_gated_delta_backward",
           "s5_gated_delta_step", "s5_qk_workspace", "s5_qk_norm_rope", "s5_qk_norm_rope_backward")

# option bits of s5_forward_ex (include/s5.h)
FLAG_HALF_SPECTRUM = 1 << 0
FLAG_BILINEAR = 1 << 1
FLAG_GELU = 1 << 2
FLAG_BIDIRECTIONAL = 1 << 3
FLAG_GELU_TANH = 1 << 4
FLAG_GLU = 1 << 5
# option bits of s5_qk_norm_rope
QK_RMS = 1 << 0
QK_L2 = 1 << 1
QK_INTERLEAVED = 1 << 2


class ForwardDesc(ctypes.Structure):
    """s5_forward_desc of include/s5.h."""
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("io", ctypes.c_int),
                ("B", ctypes.c_int64), ("L", ctypes.c_int64), ("H", ctypes.c_int64), ("P", ctypes.c_int64),
                ("u", ctypes.c_void_p), ("lam", ctypes.c_void_p), ("b_tilde", ctypes.c_void_p),
                ("c_tilde", ctypes.c_void_p), ("d", ctypes.c_void_p), ("log_delta", ctypes.c_void_p),
                ("delta", ctypes.c_void_p), ("x0", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("x_last", ctypes.c_void_p),
                ("glu_w", ctypes.c_void_p), ("glu_bias", ctypes.c_void_p), ("glu_variant", ctypes.c_int32)]


class DeltaDesc(ctypes.Structure):
    """s5_delta_desc of include/s5.h."""
    _fields_ = ([("size", ctypes.c_uint32), ("io", ctypes.c_int)] +
                [(n, ctypes.c_int64) for n in ("B", "L", "Hk", "Hv", "Dk", "Dv", "q_stride", "k_stride", "v_stride")] +
                [("scale", ctypes.c_float)] +
                [(n, ctypes.c_void_p) for n in ("q", "k", "v", "g", "beta", "s0", "lengths", "y", "s_last", "dy",
                                                "ds_last", "dq", "dk", "dv", "dg", "dbeta", "ds0", "workspace")] +
                [("workspace_bytes", ctypes.c_int64)])


class QkDesc(ctypes.Structure):
    """s5_qk_desc of include/s5.h."""
    _fields_ = ([("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("io", ctypes.c_int)] +
                [(n, ctypes.c_int64) for n in ("T", "L", "Hq", "Hk", "D", "R", "q_stride", "k_stride")] +
                [("eps", ctypes.c_float), ("rope_scale", ctypes.c_float)] +
                [(n, ctypes.c_void_p) for n in ("q", "k", "q_weight", "k_weight", "freqs", "positions", "q_out", "k_out",
                                                "dq_out", "dk_out", "dq_weight", "dk_weight", "workspace")] +
                [("workspace_bytes", ctypes.c_int64)])


class S5Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """Load libs5.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError(f"{lib_path} not found: build it with "
                              "`python -m diagonal_state_space_amd.build_lib`")
        # torch first: it carries its own HIP runtime, and libs5.so must bind
        # to that one (loaded before torch, it would bind to the system's, and
        # torch's streams would be foreign to it: every call S5_ERR_HIP)
        import torch  # noqa: F401
        L = ctypes.CDLL(lib_path)
        i64, vp, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.s5_discretize.argtypes = [i64, i64, vp, vp, vp, vp, vp, vp]
        L.s5_discretize.restype = st
        L.s5_forward.argtypes = [i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp]
        L.s5_forward.restype = st
        L.s5_forward_noalloc.argtypes = [i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp]
        L.s5_forward_noalloc.restype = st
        L.s5_forward_timevarying.argtypes = [i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp,
                                             vp, vp, vp, vp]
        L.s5_forward_timevarying.restype = st
        L.s5_forward_stateful.argtypes = [i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp]
        L.s5_forward_stateful.restype = st
        L.s5_forward_timevarying_stateful.argtypes = [i64, i64, i64, i64, ctypes.c_int, vp, vp, vp,
                                                      vp, vp, vp, vp, vp, vp, vp]
        L.s5_forward_timevarying_stateful.restype = st
        L.s5_forward_ex.argtypes = [ctypes.POINTER(ForwardDesc), vp]
        L.s5_forward_ex.restype = st
        L.s5_step.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_uint32] + [vp] * 10
        L.s5_step.restype = st
        L.s5_glu.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp]
        L.s5_glu.restype = st
        for name in ("s5_gated_delta", "s5_gated_delta_backward"):
            getattr(L, name).argtypes = [ctypes.POINTER(DeltaDesc), vp]
            getattr(L, name).restype = st
        L.s5_gated_delta_workspace.argtypes = [ctypes.POINTER(DeltaDesc), ctypes.c_int, ctypes.POINTER(i64)]
        L.s5_gated_delta_workspace.restype = st
        L.s5_gated_delta_step.argtypes = [i64] * 5 + [ctypes.c_int] + [i64] * 3 + [ctypes.c_float] + [vp] * 8
        L.s5_gated_delta_step.restype = st
        for name in ("s5_qk_norm_rope", "s5_qk_norm_rope_backward"):
            getattr(L, name).argtypes = [ctypes.POINTER(QkDesc), vp]
            getattr(L, name).restype = st
        L.s5_qk_workspace.argtypes = [ctypes.POINTER(QkDesc), ctypes.POINTER(i64)]
        L.s5_qk_workspace.restype = st
        L.s5_status_string.argtypes = [st]
        L.s5_status_string.restype = ctypes.c_char_p
        L.s5_set_profiling_events.argtypes = [vp, ctypes.c_int]
        L.s5_set_profiling_events.restype = st
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().s5_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise S5Error(status, where)


def _stream_handle(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _dev_tensor(t, name, dtype, shape):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _io_code(dtype, name="u/y") -> int:
    import torch
    if dtype == torch.float32:
        return S5_F32
    if dtype == torch.bfloat16:
        return S5_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")


def discretize(lam, b_tilde, log_delta, lam_bar=None, b_bar=None, stream=None):
    """Zero-order hold: returns (Lambda_bar [P] complex64, B_bar [P,H] complex64)."""
    import torch
    P, H = b_tilde.shape
    _dev_tensor(lam, "lam", torch.complex64, (P,))
    _dev_tensor(b_tilde, "b_tilde", torch.complex64, (P, H))
    _dev_tensor(log_delta, "log_delta", torch.float32, (P,))
    if lam_bar is None:
        lam_bar = torch.empty(P, dtype=torch.complex64, device=lam.device)
    if b_bar is None:
        b_bar = torch.empty(P, H, dtype=torch.complex64, device=lam.device)
    _dev_tensor(lam_bar, "lam_bar", torch.complex64, (P,))
    _dev_tensor(b_bar, "b_bar", torch.complex64, (P, H))
    _check(lib().s5_discretize(P, H, lam.data_ptr(), b_tilde.data_ptr(), log_delta.data_ptr(),
                               lam_bar.data_ptr(), b_bar.data_ptr(), _stream_handle(stream)),
           "s5_discretize")
    return lam_bar, b_bar


def _forward_args(u, lam, b_tilde, c_tilde, d, y):
    import torch
    if u.dim() != 3:
        raise ValueError("u must be [B, L, H]")
    B, L, H = u.shape
    P = lam.shape[0]
    io = _io_code(u.dtype)
    _dev_tensor(u, "u", u.dtype, (B, L, H))
    _dev_tensor(lam, "lam", torch.complex64, (P,))
    _dev_tensor(b_tilde, "b_tilde", torch.complex64, (P, H))
    _dev_tensor(c_tilde, "c_tilde", torch.complex64, (H, P))
    _dev_tensor(d, "d", torch.float32, (H,))
    if y is None:
        y = torch.empty_like(u)
    _dev_tensor(y, "y", u.dtype, (B, L, H))
    return B, L, H, P, io, y


def forward(u, lam, b_tilde, c_tilde, d, log_delta, y=None, stream=None):
    """Time-invariant S5 forward: y = Re(C~ x_k) + D u_k, shape of u."""
    import torch
    B, L, H, P, io, y = _forward_args(u, lam, b_tilde, c_tilde, d, y)
    _dev_tensor(log_delta, "log_delta", torch.float32, (P,))
    _check(lib().s5_forward(B, L, H, P, io, u.data_ptr(), lam.data_ptr(), b_tilde.data_ptr(),
                            c_tilde.data_ptr(), d.data_ptr(), log_delta.data_ptr(), y.data_ptr(),
                            _stream_handle(stream)), "s5_forward")
    return y


def forward_noalloc(u, lam, b_tilde, c_tilde, d, log_delta, y=None, stream=None):
    """As forward, through s5_forward_noalloc: the library's scratch is its
    fixed per-device array (nothing is allocated by the library)."""
    import torch
    B, L, H, P, io, y = _forward_args(u, lam, b_tilde, c_tilde, d, y)
    _dev_tensor(log_delta, "log_delta", torch.float32, (P,))
    _check(lib().s5_forward_noalloc(B, L, H, P, io, u.data_ptr(), lam.data_ptr(), b_tilde.data_ptr(),
                                    c_tilde.data_ptr(), d.data_ptr(), log_delta.data_ptr(), y.data_ptr(),
                                    _stream_handle(stream)), "s5_forward_noalloc")
    return y


def forward_timevarying(u, lam, b_tilde, c_tilde, d, delta, y=None, stream=None):
    """S5 forward with one interval per (batch, step, mode): delta [B, L, P]."""
    import torch
    B, L, H, P, io, y = _forward_args(u, lam, b_tilde, c_tilde, d, y)
    _dev_tensor(delta, "delta", torch.float32, (B, L, P))
    _check(lib().s5_forward_timevarying(B, L, H, P, io, u.data_ptr(), lam.data_ptr(),
                                        b_tilde.data_ptr(), c_tilde.data_ptr(), d.data_ptr(),
                                        delta.data_ptr(), y.data_ptr(), _stream_handle(stream)),
           "s5_forward_timevarying")
    return y


def _state_args(x0, x_last, B, P, device):
    import torch
    if x0 is not None:
        _dev_tensor(x0, "x0", torch.complex64, (B, P))
    if x_last is None:
        x_last = torch.empty(B, P, dtype=torch.complex64, device=device)
    _dev_tensor(x_last, "x_last", torch.complex64, (B, P))
    return (x0.data_ptr() if x0 is not None else None), x_last


def forward_stateful(u, lam, b_tilde, c_tilde, d, log_delta, x0=None, y=None, x_last=None,
                     stream=None):
    """Time-invariant forward from the state x0 ([B, P] complex64, None = zero);
    returns (y, x_last) with x_last [B, P] the state after the last step."""
    import torch
    B, L, H, P, io, y = _forward_args(u, lam, b_tilde, c_tilde, d, y)
    _dev_tensor(log_delta, "log_delta", torch.float32, (P,))
    x0p, x_last = _state_args(x0, x_last, B, P, u.device)
    _check(lib().s5_forward_stateful(B, L, H, P, io, u.data_ptr(), lam.data_ptr(), b_tilde.data_ptr(),
                                     c_tilde.data_ptr(), d.data_ptr(), log_delta.data_ptr(), x0p,
                                     y.data_ptr(), x_last.data_ptr(), _stream_handle(stream)),
           "s5_forward_stateful")
    return y, x_last


def forward_timevarying_stateful(u, lam, b_tilde, c_tilde, d, delta, x0=None, y=None, x_last=None,
                                 stream=None):
    """Time-varying forward from the state x0; returns (y, x_last)."""
    import torch
    B, L, H, P, io, y = _forward_args(u, lam, b_tilde, c_tilde, d, y)
    _dev_tensor(delta, "delta", torch.float32, (B, L, P))
    x0p, x_last = _state_args(x0, x_last, B, P, u.device)
    _check(lib().s5_forward_timevarying_stateful(B, L, H, P, io, u.data_ptr(), lam.data_ptr(),
                                                 b_tilde.data_ptr(), c_tilde.data_ptr(), d.data_ptr(),
                                                 delta.data_ptr(), x0p, y.data_ptr(),
                                                 x_last.data_ptr(), _stream_handle(stream)),
           "s5_forward_timevarying_stateful")
    return y, x_last


def forward_ex(u, lam, b_tilde, c_tilde, d, log_delta=None, delta=None, x0=None, *,
               half_spectrum=False, bilinear=False, gelu=False, bidirectional=False,
               final_state=False, gelu_tanh=False, glu_w=None, glu_bias=None, glu_variant=1,
               y=None, x_last=None, stream=None):
    """The forward pass with its options (s5_forward_ex): exactly one of
    log_delta [P] (time-invariant) and delta [B, L, P] (time-varying);
    c_tilde [H, 2P] when bidirectional; glu_w [H, H] float32 (with glu_bias
    [H] or None, glu_variant 1 or 2) applies the gated activation to y.
    Returns (y, x_last), x_last None unless final_state is set or an x_last
    buffer is given."""
    import torch
    if u.dim() != 3:
        raise ValueError("u must be [B, L, H]")
    B, L, H = u.shape
    P = lam.shape[0]
    io = _io_code(u.dtype)
    _dev_tensor(u, "u", u.dtype, (B, L, H))
    _dev_tensor(lam, "lam", torch.complex64, (P,))
    _dev_tensor(b_tilde, "b_tilde", torch.complex64, (P, H))
    _dev_tensor(c_tilde, "c_tilde", torch.complex64, (H, 2 * P if bidirectional else P))
    _dev_tensor(d, "d", torch.float32, (H,))
    if (log_delta is None) == (delta is None):
        raise ValueError("give exactly one of log_delta and delta")
    if log_delta is not None:
        _dev_tensor(log_delta, "log_delta", torch.float32, (P,))
    if delta is not None:
        _dev_tensor(delta, "delta", torch.float32, (B, L, P))
    if y is None:
        y = torch.empty_like(u)
    _dev_tensor(y, "y", u.dtype, (B, L, H))
    x0p = None
    if x0 is not None:
        x0p = _dev_tensor(x0, "x0", torch.complex64, (B, P)).data_ptr()
    if final_state and x_last is None:
        x_last = torch.empty(B, P, dtype=torch.complex64, device=u.device)
    if x_last is not None:
        _dev_tensor(x_last, "x_last", torch.complex64, (B, P))
    if glu_w is not None:
        _dev_tensor(glu_w, "glu_w", torch.float32, (H, H))
        if glu_bias is not None:
            _dev_tensor(glu_bias, "glu_bias", torch.float32, (H,))
    flags = ((FLAG_HALF_SPECTRUM if half_spectrum else 0) | (FLAG_BILINEAR if bilinear else 0) |
             (FLAG_GELU if gelu else 0) | (FLAG_BIDIRECTIONAL if bidirectional else 0) |
             (FLAG_GELU_TANH if gelu_tanh else 0) | (FLAG_GLU if glu_w is not None else 0))
    desc = ForwardDesc(ctypes.sizeof(ForwardDesc), flags, io, B, L, H, P, u.data_ptr(), lam.data_ptr(),
                       b_tilde.data_ptr(), c_tilde.data_ptr(), d.data_ptr(),
                       log_delta.data_ptr() if log_delta is not None else None,
                       delta.data_ptr() if delta is not None else None, x0p, y.data_ptr(),
                       x_last.data_ptr() if x_last is not None else None,
                       glu_w.data_ptr() if glu_w is not None else None,
                       glu_bias.data_ptr() if glu_bias is not None and glu_w is not None else None,
                       glu_variant if glu_w is not None else 0)
    _check(lib().s5_forward_ex(ctypes.byref(desc), _stream_handle(stream)), "s5_forward_ex")
    return y, x_last


def step(u, lam, b_tilde, c_tilde, d, x, log_delta=None, delta=None, *, half_spectrum=False,
         bilinear=False, gelu=False, gelu_tanh=False, y=None, stream=None):
    """One recurrent step (s5_step): u [B, H]; x [B, P] complex64 updated in
    place; exactly one of log_delta [P] and delta [B, P]. Returns y [B, H]."""
    import torch
    if u.dim() != 2:
        raise ValueError("u must be [B, H]")
    B, H = u.shape
    P = lam.shape[0]
    io = _io_code(u.dtype)
    _dev_tensor(u, "u", u.dtype, (B, H))
    _dev_tensor(lam, "lam", torch.complex64, (P,))
    _dev_tensor(b_tilde, "b_tilde", torch.complex64, (P, H))
    _dev_tensor(c_tilde, "c_tilde", torch.complex64, (H, P))
    _dev_tensor(d, "d", torch.float32, (H,))
    _dev_tensor(x, "x", torch.complex64, (B, P))
    if (log_delta is None) == (delta is None):
        raise ValueError("give exactly one of log_delta and delta")
    if log_delta is not None:
        _dev_tensor(log_delta, "log_delta", torch.float32, (P,))
    if delta is not None:
        _dev_tensor(delta, "delta", torch.float32, (B, P))
    if y is None:
        y = torch.empty_like(u)
    _dev_tensor(y, "y", u.dtype, (B, H))
    flags = ((FLAG_HALF_SPECTRUM if half_spectrum else 0) | (FLAG_BILINEAR if bilinear else 0) |
             (FLAG_GELU if gelu else 0) | (FLAG_GELU_TANH if gelu_tanh else 0))
    _check(lib().s5_step(B, H, P, io, flags, u.data_ptr(), lam.data_ptr(), b_tilde.data_ptr(),
                         c_tilde.data_ptr(), d.data_ptr(),
                         log_delta.data_ptr() if log_delta is not None else None,
                         delta.data_ptr() if delta is not None else None, x.data_ptr(), y.data_ptr(),
                         _stream_handle(stream)), "s5_step")
    return y


def glu(y, w, bias=None, variant=1, out=None, stream=None):
    """Gated activation (s5_glu): y [..., H] float32 or bfloat16 (any leading
    shape, contiguous); w [H, H] float32; bias [H] float32 or None. Returns
    (variant 1) GELU(y) * sigmoid(GELU(y) w^T + b) or (variant 2)
    y * sigmoid(GELU(y) w^T + b); out may be y (in place)."""
    import torch
    H = y.shape[-1]
    T = y.numel() // H if H else 0
    io = _io_code(y.dtype)
    _dev_tensor(y, "y", y.dtype, tuple(y.shape))
    _dev_tensor(w, "w", torch.float32, (H, H))
    if bias is not None:
        _dev_tensor(bias, "bias", torch.float32, (H,))
    if out is None:
        out = torch.empty_like(y)
    _dev_tensor(out, "out", y.dtype, tuple(y.shape))
    _check(lib().s5_glu(T, H, io, int(variant), y.data_ptr(), w.data_ptr(),
                        bias.data_ptr() if bias is not None else None, out.data_ptr(),
                        _stream_handle(stream)), "s5_glu")
    return out


def set_profiling_events(events) -> None:
    """Raw hipEvent_t handles (ints), an even number up to 12: events[2k] and
    events[2k+1] are recorded around the k-th kernel launch (0 packing, 1
    aggregate pass, 2 state and output pass; 3-5 the same for the backward
    scan of the bidirectional form) of later forward calls from this thread.
    An empty sequence (or None) turns the hook off."""
    events = list(events or [])
    arr = (ctypes.c_void_p * max(1, len(events)))(*events) if events else None
    _check(lib().s5_set_profiling_events(arr, len(events)), "s5_set_profiling_events")


# ---- gated delta rule, and the norm and rotation of its queries and keys ------


# These calls take a few microseconds on the GPU where a model decodes, so the
# checks are written for the case that they pass: one comparison of each
# property, and the words for what is wrong only after that.


def _on(t, stream, name="the first tensor"):
    """None where t's device is the current one and no stream is given; else a
    context that makes both torch's, so that outputs and workspaces are
    allocated for the stream that the kernels run on."""
    import torch
    try:
        on_gpu = t.device.type == "cuda"
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not on_gpu:
        raise ValueError(f"the tensors must be on a GPU device, got {t.device}")
    if stream is None and t.device.index == torch.cuda.current_device():
        return None
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    import contextlib
    c = contextlib.ExitStack()
    c.enter_context(torch.cuda.device(t.device))
    if stream is not None:
        c.enter_context(torch.cuda.stream(stream))
    return c


def _raw_stream(device) -> int:
    """Handle of torch's current stream on the device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _same_device(t, name, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _given(t, name, dtype, shape, device):
    """Pointer of a checked contiguous tensor, None for None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev_tensor(t, name, dtype, shape)
    _same_device(t, name, device)
    return t.data_ptr()


def _made(t, name, dtype, shape, device, zero=False):
    """A given output, checked, or a new one (filled with zeros if not every
    row of it will be written)."""
    import torch
    if t is None:
        return (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=device)
    _given(t, name, dtype, shape, device)
    return t


def _heads(t, name, dtype, lead, device):
    """Elements between the tokens of t [*lead, heads, features]: heads and
    features contiguous, one distance between all tokens."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on a GPU device, got {t.device}")
        _same_device(t, name, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    n = len(lead)
    shape = t.shape
    if len(shape) != n + 2 or shape[:n] != lead:
        raise ValueError(f"{name} must have shape {tuple(lead)} + (heads, features), got {tuple(shape)}")
    H, D = shape[n:]
    if H < 1 or D < 1:
        raise ValueError(f"{name} must have heads and features, got {tuple(shape)}")
    row = H * D
    if t.is_contiguous() or t.numel() == 0:
        return row
    st = t.stride()
    if (D > 1 and st[n + 1] != 1) or (H > 1 and st[n] != D):
        raise ValueError(f"{name}: the heads and features of a token must be contiguous, got strides {st}")
    ld, rows = None, 1   # from the innermost leading dimension outwards
    for size, stride in zip(reversed(lead), reversed(st[:n])):
        if size > 1:
            if ld is None:
                ld = stride // rows if stride % rows == 0 else -1
            elif stride != ld * rows:
                raise ValueError(f"{name}: tokens must lie at one distance, got strides {st}")
        rows *= size
    if ld is None:
        ld = row
    if ld < row:
        raise ValueError(f"{name}: tokens overlap, got strides {st}")
    return ld


def _workspace(desc, device, fn, *more):
    """Allocates what the library asks for (fn: its query) and enters it in desc."""
    import torch
    need = ctypes.c_int64()
    _check(fn(ctypes.byref(desc), *more, ctypes.byref(need)), fn.__name__)
    if need.value == 0:
        return None
    ws = torch.empty(need.value, dtype=torch.uint8, device=device)
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), need.value
    return ws


def _delta_desc(q, k, v, g, beta, s0, scale, lengths):
    import torch
    if v.dim() != 4:
        raise ValueError("v must be [B, L, Hv, Dv]")
    B, L, Hv, Dv = v.shape
    dev, io = v.device, _io_code(v.dtype, "v")
    ldv = _heads(v, "v", v.dtype, (B, L), dev)
    ldk = _heads(k, "k", v.dtype, (B, L), dev)
    ldq = _heads(q, "q", v.dtype, (B, L), dev)
    Hk, Dk = k.shape[2:]
    if q.shape != k.shape:
        raise ValueError(f"q and k must have one shape, got {tuple(q.shape)} and {tuple(k.shape)}")
    if Hv % Hk:
        raise ValueError(f"the value heads ({Hv}) must be a multiple of the key heads ({Hk})")
    f32 = torch.float32
    d = DeltaDesc(ctypes.sizeof(DeltaDesc), io, B, L, Hk, Hv, Dk, Dv, ldq, ldk, ldv,
                  Dk ** -0.5 if scale is None else float(scale), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                  _given(g, "g", f32, (B, L, Hv), dev), _given(beta, "beta", f32, (B, L, Hv), dev),
                  _given(s0, "s0", f32, (B, Hv, Dk, Dv), dev), _given(lengths, "lengths", torch.int32, (B,), dev))
    return d, dev


def gated_delta(q, k, v, g, beta, s0=None, *, scale=None, lengths=None, final_state=False, y=None, s_last=None,
                stream=None):
    """The gated delta rule (s5_gated_delta) over whole sequences:
    S_t = a_t S_{t-1} + k_t u_t^T, u_t = beta_t (v_t - a_t S_{t-1}^T k_t),
    y_t = scale S_t^T q_t, a_t = exp(g_t).

    q, k [B, L, Hk, Dk] and v [B, L, Hv, Dv], float32 or bfloat16, may be slices
    of one projection (the heads of a token contiguous, one distance between
    tokens); value head h reads key head h // (Hv // Hk). g, beta [B, L, Hv]
    float32; s0 [B, Hv, Dk, Dv] float32 or None (zero); scale None is
    Dk ** -0.5. lengths [B] int32: the valid steps of each sequence; rows of y
    behind them are zero in a y made here and left as they were in a given one.
    Returns (y, s_last), s_last None unless final_state is set or a buffer is
    given (which may be s0). Inputs that require gradients are taken, but the
    results carry no autograd graph: gated_delta_backward gives the gradients."""
    import torch
    on = _on(v, stream, "v")
    if on is not None:
        with on:
            return gated_delta(q, k, v, g, beta, s0, scale=scale, lengths=lengths, final_state=final_state, y=y, s_last=s_last)
    d, dev = _delta_desc(q, k, v, g, beta, s0, scale, lengths)
    B, L, Hv, Dv = v.shape
    y = _made(y, "y", v.dtype, (B, L, Hv, Dv), dev, zero=lengths is not None)
    if final_state or s_last is not None:
        s_last = _made(s_last, "s_last", torch.float32, (B, Hv, d.Dk, Dv), dev)
        d.s_last = s_last.data_ptr()
    d.y = y.data_ptr()
    ws = _workspace(d, dev, lib().s5_gated_delta_workspace, 0)   # noqa: F841  (held until the call is enqueued)
    _check(lib().s5_gated_delta(ctypes.byref(d), _raw_stream(dev)), "s5_gated_delta")
    return y, s_last


def gated_delta_backward(dy, q, k, v, g, beta, s0=None, ds_last=None, *, scale=None, lengths=None, dq=None, dk=None,
                         dv=None, dg=None, dbeta=None, ds0=None, stream=None):
    """Gradients of gated_delta (s5_gated_delta_backward) from dy, the gradient
    of y, and ds_last, that of the last state (None: zero); the forward pass is
    computed again, nothing is kept from it. Returns (dq, dk, dv, dg, dbeta,
    ds0), ds0 None unless s0 or a buffer for it is given. With lengths the
    rows behind are zero in gradients made here and left in given ones. It
    allocates 4.5 KB (float32: 8.8) for each step and head of 128 x 128 while it
    runs, up to 4 GiB (s5_gated_delta_workspace)."""
    import torch
    on = _on(v, stream, "v")
    if on is not None:
        with on:
            return gated_delta_backward(dy, q, k, v, g, beta, s0, ds_last, scale=scale, lengths=lengths, dq=dq, dk=dk, dv=dv,
                                        dg=dg, dbeta=dbeta, ds0=ds0)
    d, dev = _delta_desc(q, k, v, g, beta, s0, scale, lengths)
    B, L, Hv, Dv = v.shape
    f32, zero = torch.float32, lengths is not None
    d.dy = _given(dy, "dy", v.dtype, (B, L, Hv, Dv), dev)
    d.ds_last = _given(ds_last, "ds_last", f32, (B, Hv, d.Dk, Dv), dev)
    dq = _made(dq, "dq", v.dtype, tuple(q.shape), dev, zero)
    dk = _made(dk, "dk", v.dtype, tuple(k.shape), dev, zero)
    dv = _made(dv, "dv", v.dtype, (B, L, Hv, Dv), dev, zero)
    dg = _made(dg, "dg", f32, (B, L, Hv), dev, zero)
    dbeta = _made(dbeta, "dbeta", f32, (B, L, Hv), dev, zero)
    if s0 is not None or ds0 is not None:
        ds0 = _made(ds0, "ds0", f32, (B, Hv, d.Dk, Dv), dev)
        d.ds0 = ds0.data_ptr()
    d.dq, d.dk, d.dv, d.dg, d.dbeta = (t.data_ptr() for t in (dq, dk, dv, dg, dbeta))
    ws = _workspace(d, dev, lib().s5_gated_delta_workspace, 1)   # noqa: F841  (held until the call is enqueued)
    _check(lib().s5_gated_delta_backward(ctypes.byref(d), _raw_stream(dev)), "s5_gated_delta_backward")
    return dq, dk, dv, dg, dbeta, ds0


def gated_delta_step(q, k, v, g, beta, s, *, scale=None, y=None, stream=None):
    """One token of gated_delta for each of B sequences (s5_gated_delta_step):
    q, k [B, Hk, Dk], v [B, Hv, Dv], g, beta [B, Hv]; s [B, Hv, Dk, Dv] float32
    is updated in place. Returns y [B, Hv, Dv], without an autograd graph."""
    import torch
    on = _on(v, stream, "v")
    if on is not None:
        with on:
            return gated_delta_step(q, k, v, g, beta, s, scale=scale, y=y)
    if v.dim() != 3:
        raise ValueError("v must be [B, Hv, Dv]")
    B, Hv, Dv = v.shape
    dev, dtype = v.device, v.dtype
    io = _io_code(dtype, "v")
    ldv = _heads(v, "v", dtype, (B,), dev)
    ldk = _heads(k, "k", dtype, (B,), dev)
    ldq = _heads(q, "q", dtype, (B,), dev)
    Hk, Dk = k.shape[1:]
    if q.shape != k.shape:
        raise ValueError(f"q and k must have one shape, got {tuple(q.shape)} and {tuple(k.shape)}")
    if Hv % Hk:
        raise ValueError(f"the value heads ({Hv}) must be a multiple of the key heads ({Hk})")
    f32 = torch.float32
    gp = _given(g, "g", f32, (B, Hv), dev)
    bp = _given(beta, "beta", f32, (B, Hv), dev)
    sp = _given(s, "s", f32, (B, Hv, Dk, Dv), dev)
    y = _made(y, "y", dtype, (B, Hv, Dv), dev)
    _check(lib().s5_gated_delta_step(B, Hk, Hv, Dk, Dv, io, ldq, ldk, ldv, Dk ** -0.5 if scale is None else scale,
                                     q.data_ptr(), k.data_ptr(), v.data_ptr(), gp, bp, sp, y.data_ptr(), _raw_stream(dev)),
           "s5_gated_delta_step")
    return y


def _qk_desc(q, k, norm, q_weight, k_weight, eps, freqs, positions, rope_scale, interleaved):
    import torch
    if q.dim() not in (3, 4):
        raise ValueError("q must be [T, Hq, D] or [B, L, Hq, D]")
    lead, dev, io = q.shape[:-2], q.device, _io_code(q.dtype, "q")
    ldq = _heads(q, "q", q.dtype, lead, dev)
    ldk = _heads(k, "k", q.dtype, lead, dev)
    (Hq, D), Hk = q.shape[-2:], k.shape[-2]
    if k.shape[-1] != D:
        raise ValueError(f"the heads of q and k must have one size, got {D} and {k.shape[-1]}")
    flags = {"rms": QK_RMS, "l2": QK_L2, None: 0}.get(norm)
    if flags is None:
        raise ValueError(f"norm must be 'rms', 'l2' or None, got {norm!r}")
    if norm is None and (q_weight is not None or k_weight is not None):
        raise ValueError("weights need a norm")
    R = 0
    if freqs is not None:
        if not isinstance(freqs, torch.Tensor):
            raise TypeError("freqs must be a torch.Tensor")
        R = 2 * freqs.numel()
        if freqs.dim() != 1 or R > D:
            raise ValueError(f"freqs must be [R/2] with R <= {D}, got {tuple(freqs.shape)}")
    T = 1
    for n in lead:
        T *= n
    d = QkDesc(ctypes.sizeof(QkDesc), flags | (QK_INTERLEAVED if interleaved else 0), io, T, max(1, lead[-1]), Hq, Hk, D, R,
               ldq, ldk, eps, rope_scale, q.data_ptr(), k.data_ptr(),
               _given(q_weight, "q_weight", torch.float32, (D,), dev), _given(k_weight, "k_weight", torch.float32, (D,), dev),
               _given(freqs, "freqs", torch.float64, (R // 2,), dev) if R else None,
               _given(positions, "positions", torch.int32, lead, dev))
    return d, dev


def qk_norm_rope(q, k, *, norm="rms", q_weight=None, k_weight=None, eps=1e-6, freqs=None, positions=None, rope_scale=1.0,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of each query and key head and rotation of its first features by
    its token's position, in one pass (s5_qk_norm_rope): n = x w / sqrt(m + eps)
    with m the mean ("rms") or sum ("l2") of x^2 (norm None: n = x), then each
    pair (a, b) of the first R features becomes rope_scale (a cos - b sin,
    b cos + a sin) at position * freqs.

    q [B, L, Hq, D] or [T, Hq, D], k with Hk heads, float32 or bfloat16, may be
    slices of one projection; weights [D] float32 or None. freqs [R/2] float64
    radians per position (rope_frequencies), None: no rotation; pairs are
    (j, j + R/2), or (2j, 2j + 1) if interleaved. positions int32, shaped as
    the tokens; None counts 0, 1, ... along L (T). Returns contiguous
    (q_out, k_out); a contiguous input may be its own output. The results carry
    no autograd graph: qk_norm_rope_backward gives the gradients."""
    on = _on(q, stream, "q")
    if on is not None:
        with on:
            return qk_norm_rope(q, k, norm=norm, q_weight=q_weight, k_weight=k_weight, eps=eps, freqs=freqs, positions=positions,
                                rope_scale=rope_scale, interleaved=interleaved, q_out=q_out, k_out=k_out)
    d, dev = _qk_desc(q, k, norm, q_weight, k_weight, eps, freqs, positions, rope_scale, interleaved)
    q_out = _made(q_out, "q_out", q.dtype, q.shape, dev)
    k_out = _made(k_out, "k_out", q.dtype, k.shape, dev)
    d.q_out, d.k_out = q_out.data_ptr(), k_out.data_ptr()
    _check(lib().s5_qk_norm_rope(ctypes.byref(d), _raw_stream(dev)), "s5_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, *, norm="rms", q_weight=None, k_weight=None, eps=1e-6, freqs=None,
                          positions=None, rope_scale=1.0, interleaved=False, dq=None, dk=None, dq_weight=None,
                          dk_weight=None, stream=None):
    """Gradients of qk_norm_rope (s5_qk_norm_rope_backward) from dq_out and
    dk_out, those of its results, with its inputs and options. Returns
    (dq, dk, dq_weight, dk_weight), a weight's gradient None without the
    weight."""
    import torch
    on = _on(q, stream, "q")
    if on is not None:
        with on:
            return qk_norm_rope_backward(dq_out, dk_out, q, k, norm=norm, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                         freqs=freqs, positions=positions, rope_scale=rope_scale, interleaved=interleaved,
                                         dq=dq, dk=dk, dq_weight=dq_weight, dk_weight=dk_weight)
    d, dev = _qk_desc(q, k, norm, q_weight, k_weight, eps, freqs, positions, rope_scale, interleaved)
    d.dq_out = _given(dq_out, "dq_out", q.dtype, q.shape, dev)
    d.dk_out = _given(dk_out, "dk_out", q.dtype, k.shape, dev)
    dq = _made(dq, "dq", q.dtype, q.shape, dev)
    dk = _made(dk, "dk", q.dtype, k.shape, dev)
    if q_weight is not None or dq_weight is not None:
        dq_weight = _made(dq_weight, "dq_weight", torch.float32, (d.D,), dev)
        d.dq_weight = dq_weight.data_ptr()
    if k_weight is not None or dk_weight is not None:
        dk_weight = _made(dk_weight, "dk_weight", torch.float32, (d.D,), dev)
        d.dk_weight = dk_weight.data_ptr()
    d.q_out, d.k_out = dq.data_ptr(), dk.data_ptr()
    ws = _workspace(d, dev, lib().s5_qk_workspace)   # noqa: F841  (held until the call is enqueued)
    _check(lib().s5_qk_norm_rope_backward(ctypes.byref(d), _raw_stream(dev)), "s5_qk_norm_rope_backward")
    return dq, dk, dq_weight, dk_weight


def rope_frequencies(rotary_dim, base=10000.0, *, factor=1.0, scaling=None, original_length=None, fast=32.0, slow=1.0,
                     device="cuda"):
    """Radians per position of each of the rotary_dim / 2 pairs, float64:
    base ** (-2 j / rotary_dim), changed for contexts `factor` times longer than
    trained by `scaling`:
      None      as they are
      "linear"  all divided by factor (positions squeezed together)
      "base"    the base times factor ** (R / (R - 2)): the fastest pair keeps its
                frequency, the slowest is divided by factor
      "parts"   pairs that turn at least `fast` times over original_length stay,
                those with at most `slow` turns are divided by factor, those
                between in proportion to their turns
    The factor that goes with "parts" (rope_scale) is 0.1 log(factor) + 1."""
    import math

    import torch
    R = int(rotary_dim)
    if R < 2 or R % 2:
        raise ValueError(f"rotary_dim must be even and >= 2, got {rotary_dim}")
    if not (base > 0 and math.isfinite(base)) or not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("base must be > 0 and factor >= 1")
    if scaling == "base":
        if R < 4:
            raise ValueError("scaling 'base' needs two pairs")
        base = base * factor ** (R / (R - 2))
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_length is None or original_length < 1 or not fast > slow > 0:
            raise ValueError("scaling 'parts' needs original_length >= 1 and fast > slow > 0")
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    return f.to(device)

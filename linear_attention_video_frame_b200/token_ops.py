"""Python binding of the token-wise operators (include/la_token.h): the gated
delta rule with one update per token (chunked, its backward pass, one token at
a time) and the residual addition with RMSNorm and an e4m3 output (and its
backward pass).

Argument marshalling only, as in the package itself.  q, k ``[B, Hk, T, D]``
and v, o ``[B, Hv, T, D]`` (bfloat16 or float32) may be strided views as long
as the D values of a row are contiguous, for example ``[B, T, H, D]``
transposed; log_alpha, beta ``[B, Hv, T]`` and states ``[B, Hv, D, D]`` are
contiguous float32; lengths ``[B]`` is int32 or None.
"""
from __future__ import annotations

import ctypes

import torch

from . import LA_ERR_UNSUPPORTED, LaScanError, _check, _dtype_code, _ptr, _raise, _stream, lib

__all__ = [
    "LaDelta", "la_gated_delta_rule", "la_gated_delta_rule_backward", "la_gated_delta_step",
    "la_delta_workspace_size", "la_delta_plan", "delta_workspace_for", "la_add_rms_norm_fp8",
    "la_add_rms_norm_backward", "la_norm_workspace_size",
]

_Strides = ctypes.c_longlong * 3


class LaDelta(ctypes.Structure):
    """The C struct la_delta (inputs of the gated delta rule)."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", _Strides), ("k_stride", _Strides), ("v_stride", _Strides),
                ("log_alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("state_in", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("k_scale", ctypes.c_float), ("q_scale", ctypes.c_float), ("dt", ctypes.c_int),
                ("B", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int),
                ("T", ctypes.c_int), ("D", ctypes.c_int)]


def _declare():
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    LL, S, R = ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(LaDelta)
    lib.la_gated_delta_rule.argtypes = [R, P, S, P, P, Z, P]
    lib.la_gated_delta_rule.restype = I
    lib.la_gated_delta_rule_backward.argtypes = [R, P, S, P, P, P, P, P, P, P, P, Z, P]
    lib.la_gated_delta_rule_backward.restype = I
    lib.la_gated_delta_step.argtypes = [R, P, S, P, P]
    lib.la_gated_delta_step.restype = I
    lib.la_delta_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.la_delta_workspace_size.restype = Z
    lib.la_delta_plan.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(ctypes.c_int)]
    lib.la_delta_plan.restype = ctypes.c_char_p
    lib.la_add_rms_norm_fp8.argtypes = [P, P, P, P, P, P, I, LL, I, I, F, P]
    lib.la_add_rms_norm_fp8.restype = I
    lib.la_add_rms_norm_backward.argtypes = [P, P, P, P, P, P, I, LL, I, F, P, Z, P]
    lib.la_add_rms_norm_backward.restype = I
    lib.la_norm_workspace_size.argtypes = [LL, I]
    lib.la_norm_workspace_size.restype = Z


_declare()


def la_delta_workspace_size(backward: bool, dt: int, B: int, Hk: int, Hv: int, T: int,
                            D: int) -> int:
    return int(lib.la_delta_workspace_size(int(backward), dt, B, Hk, Hv, T, D))


def la_delta_plan(backward: bool, dt: int, B: int, Hk: int, Hv: int, T: int, D: int):
    """(path name, kernels per call) of a call of this shape; (None, 0) if unsupported."""
    n = ctypes.c_int(0)
    name = lib.la_delta_plan(int(backward), dt, B, Hk, Hv, T, D, ctypes.byref(n))
    return (name.decode() if name else None), int(n.value)


def delta_workspace_for(backward: bool, dt: int, B: int, Hk: int, Hv: int, T: int, D: int,
                        device=None) -> torch.Tensor:
    """A caller-owned workspace tensor of the size the library asks for."""
    n = la_delta_workspace_size(backward, dt, B, Hk, Hv, T, D)
    if n == 0:
        raise LaScanError(LA_ERR_UNSUPPORTED, "la_delta_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def la_norm_workspace_size(rows: int, N: int) -> int:
    return int(lib.la_norm_workspace_size(rows, N))


def _check_device(device: torch.device, *tensors):
    """Kernels run on the current device: every tensor must live there."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    for name, t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t: torch.Tensor, name: str, shape, dtype):
    """Checks a [B, H, T, D] tensor with contiguous rows; its strides."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    # the stride of an axis of one element is never taken; torch may report any value for it
    return _Strides(*(s if n > 1 else 0 for s, n in zip(t.stride()[:3], t.shape[:3])))


def _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths) -> LaDelta:
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v are [B, H, T, D]")
    B, Hk, T, D = q.shape
    Hv = v.shape[1]
    _dtype_code(q)
    qs = _rows(q, "q", (B, Hk, T, D), q.dtype)
    ks = _rows(k, "k", (B, Hk, T, D), q.dtype)
    vs = _rows(v, "v", (B, Hv, T, D), q.dtype)
    for t, n in ((log_alpha, "log_alpha"), (beta, "beta")):
        _check(t, n, (B, Hv, T), torch.float32)
    _check(state_in, "state_in", (B, Hv, D, D), torch.float32)
    _check(lengths, "lengths", (B,), torch.int32)
    _check_device(q.device, ("k", k), ("v", v), ("log_alpha", log_alpha), ("beta", beta),
                  ("state_in", state_in), ("lengths", lengths))
    return LaDelta(_ptr(q), _ptr(k), _ptr(v), qs, ks, vs, _ptr(log_alpha), _ptr(beta),
                   _ptr(state_in), _ptr(lengths), float(k_scale), float(q_scale),
                   _dtype_code(q), B, Hk, Hv, T, D)


def _new_rows(like: torch.Tensor, lengths) -> torch.Tensor:
    # rows behind a sequence's length are not written
    return torch.empty_like(like) if lengths is None else torch.zeros_like(like)


def la_gated_delta_rule(q, k, v, log_alpha, beta, k_scale: float = 1.0, q_scale: float = 1.0,
                        o=None, state_in=None, state_out=None, lengths=None, workspace=None,
                        stream=None):
    """Gated delta rule over T tokens: ``S_t = alpha_t (I - beta_t k k^T) S_{t-1} + beta_t k v^T``,
    ``o_t = q S_t`` with ``alpha = exp(log_alpha)`` (see include/la_token.h).  Returns o; rows
    behind a sequence's length are left as they were in a given o, 0 in a new one."""
    a = _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths)
    B, Hv, T, D = v.shape
    if o is None:
        o = _new_rows(v, lengths)
        if T and o.stride(2) == 0:                   # v was a broadcast view
            o = o.contiguous()
    os = _rows(o, "o", (B, Hv, T, D), q.dtype)
    _check(state_out, "state_out", (B, Hv, D, D), torch.float32)
    if workspace is None:
        workspace = delta_workspace_for(False, a.dt, B, a.Hk, Hv, T, D, q.device)
    _check_device(q.device, ("o", o), ("state_out", state_out), ("workspace", workspace))
    st = lib.la_gated_delta_rule(ctypes.byref(a), _ptr(o), os, _ptr(state_out), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _raise(st, "la_gated_delta_rule")
    return o


def la_gated_delta_step(q, k, v, log_alpha, beta, state_in, k_scale: float = 1.0,
                        q_scale: float = 1.0, o=None, state_out=None, lengths=None, stream=None):
    """One token of the gated delta rule for every sequence: q, k ``[B, Hk, D]``, v, o
    ``[B, Hv, D]``, log_alpha, beta ``[B, Hv]``.  state_out (default: state_in, in place) gets
    the new state.  A sequence of length 0 keeps its state and its row of o."""
    if q.dim() != 3 or v.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v of a step are [B, H, D]")
    B, Hv, D = v.shape
    _check(log_alpha, "log_alpha", (B, Hv), torch.float32)
    _check(beta, "beta", (B, Hv), torch.float32)
    if o is None:
        o = _new_rows(v, lengths)
    if state_out is None:
        state_out = state_in
    if state_out is None:
        raise ValueError("a step needs state_in or state_out")
    a = _inputs(q.unsqueeze(2), k.unsqueeze(2), v.unsqueeze(2), log_alpha.unsqueeze(2),
                beta.unsqueeze(2), k_scale, q_scale, state_in, lengths)
    os = _rows(o.unsqueeze(2), "o", (B, Hv, 1, D), q.dtype)
    _check(state_out, "state_out", (B, Hv, D, D), torch.float32)
    _check_device(q.device, ("o", o), ("state_out", state_out))
    st = lib.la_gated_delta_step(ctypes.byref(a), _ptr(o), os, _ptr(state_out), _stream(stream))
    _raise(st, "la_gated_delta_step")
    return o


def la_gated_delta_rule_backward(q, k, v, log_alpha, beta, do, k_scale: float = 1.0,
                                 q_scale: float = 1.0, state_in=None, dstate_out=None,
                                 dq=None, dk=None, dv=None, dlog_alpha=None, dbeta=None,
                                 dstate_in=None, lengths=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv, dlog_alpha, dbeta) of la_gated_delta_rule for the gradient `do` of
    its output and `dstate_out` of its final state; dstate_in (if given) gets the initial
    state's.  Gradients of rows behind a sequence's length are 0."""
    a = _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths)
    B, Hv, T, D = v.shape
    dos = _rows(do, "do", (B, Hv, T, D), q.dtype)
    for t, n in ((dstate_out, "dstate_out"), (dstate_in, "dstate_in")):
        _check(t, n, (B, Hv, D, D), torch.float32)

    def out(t, name, shape, dtype):
        if t is None:
            return torch.empty(shape, dtype=dtype, device=q.device)
        _check(t, name, shape, dtype)
        return t

    dq, dk = out(dq, "dq", q.shape, q.dtype), out(dk, "dk", k.shape, q.dtype)
    dv = out(dv, "dv", v.shape, q.dtype)
    dlog_alpha = out(dlog_alpha, "dlog_alpha", (B, Hv, T), torch.float32)
    dbeta = out(dbeta, "dbeta", (B, Hv, T), torch.float32)
    if workspace is None:
        workspace = delta_workspace_for(True, a.dt, B, a.Hk, Hv, T, D, q.device)
    _check_device(q.device, ("do", do), ("dstate_out", dstate_out), ("dstate_in", dstate_in),
                  ("dq", dq), ("dk", dk), ("dv", dv), ("dlog_alpha", dlog_alpha),
                  ("dbeta", dbeta), ("workspace", workspace))
    st = lib.la_gated_delta_rule_backward(ctypes.byref(a), _ptr(do), dos, _ptr(dstate_out),
                                          _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_alpha),
                                          _ptr(dbeta), _ptr(dstate_in), _ptr(workspace),
                                          workspace.numel(), _stream(stream))
    _raise(st, "la_gated_delta_rule_backward")
    return dq, dk, dv, dlog_alpha, dbeta


def la_add_rms_norm_fp8(x, residual, weight, eps: float = 1e-6, group: int = 128, h=None, y=None,
                        scale=None, stream=None):
    """Residual addition, RMSNorm and e4m3 output.  x, residual ``[..., N]`` (residual may be
    None), weight ``[N]`` float32.  Returns (y float8_e4m3fn ``[..., N]``, scale float32
    ``[..., ceil(N / group)]`` (group = 0: ``[..., 1]``), h = x + residual as stored, which is x
    itself without a residual).  ``y.float() * scale`` (each scale over its group) is the norm."""
    N = x.shape[-1]
    dt = _dtype_code(x)
    _check(x, "x")
    _check(residual, "residual", x.shape, x.dtype)
    _check(weight, "weight", (N,), torch.float32)
    if group not in (0, 128):
        raise ValueError(f"group must be 128 or 0 (the row), got {group}")
    rows = x.numel() // N if N else 0
    if h is None and residual is not None:
        h = torch.empty_like(x)
    if y is None:
        y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty((*x.shape[:-1], -(-N // group) if group else 1),
                            dtype=torch.float32, device=x.device)
    _check(h, "h", x.shape, x.dtype)
    _check(y, "y", x.shape, torch.float8_e4m3fn)
    _check(scale, "scale", (*x.shape[:-1], -(-N // group) if group else 1), torch.float32)
    _check_device(x.device, ("residual", residual), ("weight", weight), ("h", h), ("y", y),
                  ("scale", scale))
    st = lib.la_add_rms_norm_fp8(_ptr(x), _ptr(residual), _ptr(weight), _ptr(h), _ptr(y),
                                 _ptr(scale), dt, rows, N, group, float(eps), _stream(stream))
    _raise(st, "la_add_rms_norm_fp8")
    return y, scale, x if h is None else h


def la_add_rms_norm_backward(dy, h, weight, dh=None, eps: float = 1e-6, dx=None, dweight=None,
                             need_dweight: bool = True, workspace=None, stream=None):
    """Gradients (dx, dweight) of the norm for the gradient `dy` of its output (the 8-bit
    rounding passed straight through), h as the forward pass returned it and `dh`, the gradient
    that h gets from elsewhere.  dx is the gradient of x and of residual alike; dweight is None
    when need_dweight is False."""
    N = h.shape[-1]
    dt = _dtype_code(h)
    _check(h, "h")
    _check(dy, "dy", h.shape, h.dtype)
    _check(dh, "dh", h.shape, h.dtype)
    _check(weight, "weight", (N,), torch.float32)
    rows = h.numel() // N if N else 0
    if dx is None:
        dx = torch.empty_like(h)
    _check(dx, "dx", h.shape, h.dtype)
    if need_dweight:
        if dweight is None:
            dweight = torch.empty((N,), dtype=torch.float32, device=h.device)
        _check(dweight, "dweight", (N,), torch.float32)
        if workspace is None:
            workspace = torch.empty(la_norm_workspace_size(rows, N), dtype=torch.uint8,
                                    device=h.device)
    else:
        dweight = workspace = None
    _check_device(h.device, ("dy", dy), ("dh", dh), ("weight", weight), ("dx", dx),
                  ("dweight", dweight), ("workspace", workspace))
    st = lib.la_add_rms_norm_backward(_ptr(dy), _ptr(h), _ptr(weight), _ptr(dh), _ptr(dx),
                                      _ptr(dweight), dt, rows, N, float(eps), _ptr(workspace),
                                      0 if workspace is None else workspace.numel(),
                                      _stream(stream))
    _raise(st, "la_add_rms_norm_backward")
    return dx, dweight

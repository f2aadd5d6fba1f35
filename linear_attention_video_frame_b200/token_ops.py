"""Python binding of the token-wise operators (include/la_token.h): the gated
delta rule with one update per token (chunked, its backward pass, one token at
a time) and the residual addition with RMSNorm and an e4m3 output (and its
backward pass).

Argument marshalling only, as in the package itself.  q, k ``[B, Hk, T, D]``
and v, o ``[B, Hv, T, D]`` (bfloat16 or float32) may be strided views as long
as the D values of a row are contiguous, for example ``[B, T, H, D]``
transposed; log_alpha, beta ``[B, Hv, T]`` and states ``[B, Hv, D, D]`` are
contiguous float32; lengths ``[B]`` is int32 or None.

Autograd does not see these calls: results carry no graph, and the backward passes
are functions of their own.

``stream`` is a torch stream or the address of a CUDA stream (default: the current
one).  Inputs, and outputs that are given, have to be ready on it; a call's new
outputs are made on it and may be used on the current stream once that waits for it.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import LA_ERR_UNSUPPORTED, LA_OK, LaScanError, _check, _dtype_code, _raise, lib

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


# The struct and strides go over as packed bytes: a call of one token is bound by
# what happens before its launch.
_pack_delta = struct.Struct("3P9q4P2f6i").pack
_pack_strides = struct.Struct("3q").pack
assert struct.calcsize("3P9q4P2f6i") == ctypes.sizeof(LaDelta)


def _declare():
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    LL, S, R = ctypes.c_longlong, P, P
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


# sizes depend on nothing but their arguments
_delta_need = functools.lru_cache(maxsize=4096)(lib.la_delta_workspace_size)
_norm_need = functools.lru_cache(maxsize=4096)(lib.la_norm_workspace_size)


def _here(t: torch.Tensor, name: str) -> int:
    """Kernels run on the current device, and the first tensor must live there."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return device


def _raw_stream(device: int):
    return torch._C._cuda_getCurrentRawStream(device)


def _elsewhere(stream, call, *args, **kw):
    """`call` with `stream` as the current stream, or NotImplemented where it is that already.
    A call's new tensors so come from the stream's own memory, are filled on it, and go back
    to it when they are let go, in the order of its kernels; the stream that is current now
    is where the caller uses them, so their memory waits for it as well."""
    here = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        address = int(getattr(stream, "cuda_stream", stream))
        # 0, and CUDA's name for it, 1, are no addresses to ExternalStream
        stream = torch.cuda.ExternalStream(address, here.device) if address > 1 else \
            torch.cuda.default_stream(here.device)
    if stream.cuda_stream == here.cuda_stream:
        return NotImplemented
    with torch.cuda.stream(stream):
        result = call(*args, **kw)
    given = {id(t) for t in (*args, *kw.values())}
    for t in result if isinstance(result, tuple) else (result,):
        if t is not None and id(t) not in given:
            t.record_stream(here)
    return result


def _full(t, name: str, shape, dtype, device):
    """The address of a contiguous tensor of this shape, dtype and device; None stays None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or \
            not t.is_contiguous():
        _check(t, name, shape, dtype)
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    return t.data_ptr()


def _space(workspace, need: int, like: torch.Tensor):
    """The workspace of a call: the given one, or a new one."""
    if workspace is None:
        workspace = like.new_empty((need,), dtype=torch.uint8)
    elif workspace.device != like.device:
        raise ValueError(f"workspace is on {workspace.device}, expected {like.device}")
    elif not workspace.is_contiguous():         # its elements are counted as its bytes
        raise ValueError("workspace must be contiguous")
    return workspace


def _rows(t, name: str, shape, dtype, device):
    """The strides of [..., D] rows, which are contiguous themselves.  The stride of an axis of
    one element is never taken; torch may report any value for it."""
    if t is None:
        raise ValueError(f"{name} is required")
    s = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or \
            (s[-1] != 1 and shape[-1] != 1):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
        raise ValueError(f"the rows of {name} must be contiguous")
    if len(shape) == 3:             # one token
        return (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, 0)
    return (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0,
            s[2] if shape[2] > 1 else 0)


def _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths, device):
    """The packed la_delta; q, k, v are [B, H, T, D], or [B, H, D] with T = 1."""
    shape, vshape = q.shape, v.shape
    B, Hk, D = shape[0], shape[1], shape[-1]
    Hv = vshape[1]
    T = shape[2] if len(shape) == 4 else 1
    dtype = q.dtype
    code = _dtype_code(q)
    gates, f32 = vshape[:-1], torch.float32
    if log_alpha is None or beta is None:
        raise ValueError(f"{'beta' if beta is None else 'log_alpha'} is required")
    qs = _rows(q, "q", shape, dtype, device)
    ks = _rows(k, "k", shape, dtype, device)
    vs = _rows(v, "v", (B, Hv, T, D) if len(shape) == 4 else (B, Hv, D), dtype, device)
    return _pack_delta(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *qs, *ks, *vs,
        _full(log_alpha, "log_alpha", gates, f32, device), _full(beta, "beta", gates, f32, device),
        _full(state_in, "state_in", (B, Hv, D, D), f32, device) or 0,
        _full(lengths, "lengths", (B,), torch.int32, device) or 0,
        k_scale, q_scale, code, B, Hk, Hv, T, D), code


def _new_rows(like: torch.Tensor, lengths) -> torch.Tensor:
    # rows behind a sequence's length are not written
    o = torch.empty_like(like) if lengths is None else torch.zeros_like(like)
    s = o.stride()
    return o.contiguous() if s[-1] != 1 or 0 in s else o         # `like` was a broadcast view


def la_gated_delta_rule(q, k, v, log_alpha, beta, k_scale: float = 1.0, q_scale: float = 1.0,
                        o=None, state_in=None, state_out=None, lengths=None, workspace=None,
                        stream=None):
    """Gated delta rule over T tokens: ``S_t = alpha_t (I - beta_t k k^T) S_{t-1} + beta_t k v^T``,
    ``o_t = q S_t`` with ``alpha = exp(log_alpha)`` (see include/la_token.h).  Returns o; rows
    behind a sequence's length are left as they were in a given o, 0 in a new one."""
    if stream is not None:
        done = _elsewhere(stream, la_gated_delta_rule, q, k, v, log_alpha, beta, k_scale, q_scale,
                          o, state_in, state_out, lengths, workspace)
        if done is not NotImplemented:
            return done
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v are [B, H, T, D]")
    device = _here(q, "q")
    a, code = _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths, device)
    B, Hv, T, D = v.shape
    if o is None:
        o = _new_rows(v, lengths)
    os = _rows(o, "o", (B, Hv, T, D), q.dtype, device)
    end = _full(state_out, "state_out", (B, Hv, D, D), torch.float32, device)
    need = _delta_need(0, code, B, q.shape[1], Hv, T, D)
    if need == 0:
        raise LaScanError(LA_ERR_UNSUPPORTED, "la_gated_delta_rule")
    workspace = _space(workspace, need, q)
    st = lib.la_gated_delta_rule(a, o.data_ptr(), _pack_strides(*os), end, workspace.data_ptr(),
                                 workspace.numel(), _raw_stream(device))
    if st != LA_OK:
        _raise(st, "la_gated_delta_rule")
    return o


def la_gated_delta_step(q, k, v, log_alpha, beta, state_in, k_scale: float = 1.0,
                        q_scale: float = 1.0, o=None, state_out=None, lengths=None, stream=None):
    """One token of the gated delta rule for every sequence: q, k ``[B, Hk, D]``, v, o
    ``[B, Hv, D]``, log_alpha, beta ``[B, Hv]``.  state_out (default: state_in, in place) gets
    the new state.  A sequence of length 0 keeps its state and its row of o."""
    if stream is not None:
        done = _elsewhere(stream, la_gated_delta_step, q, k, v, log_alpha, beta, state_in, k_scale,
                          q_scale, o, state_out, lengths)
        if done is not NotImplemented:
            return done
    if q.dim() != 3 or v.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v of a step are [B, H, D]")
    if state_out is None:
        state_out = state_in
    if state_out is None:
        raise ValueError("a step needs state_in or state_out")
    device = _here(q, "q")
    a, _ = _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths, device)
    B, Hv, D = shape = v.shape
    if o is None:
        o = _new_rows(v, lengths)
    os = _rows(o, "o", shape, q.dtype, device)
    end = state_in.data_ptr() if state_out is state_in else \
        _full(state_out, "state_out", (B, Hv, D, D), torch.float32, device)
    st = lib.la_gated_delta_step(a, o.data_ptr(), _pack_strides(*os), end,
                                 _raw_stream(device))
    if st != LA_OK:
        _raise(st, "la_gated_delta_step")
    return o


def la_gated_delta_rule_backward(q, k, v, log_alpha, beta, do, k_scale: float = 1.0,
                                 q_scale: float = 1.0, state_in=None, dstate_out=None,
                                 dq=None, dk=None, dv=None, dlog_alpha=None, dbeta=None,
                                 dstate_in=None, lengths=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv, dlog_alpha, dbeta) of la_gated_delta_rule for the gradient `do` of
    its output and `dstate_out` of its final state; dstate_in (if given) gets the initial
    state's.  Gradients of rows behind a sequence's length are 0."""
    if stream is not None:
        done = _elsewhere(stream, la_gated_delta_rule_backward, q, k, v, log_alpha, beta, do,
                          k_scale, q_scale, state_in, dstate_out, dq, dk, dv, dlog_alpha, dbeta,
                          dstate_in, lengths, workspace)
        if done is not NotImplemented:
            return done
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v are [B, H, T, D]")
    device = _here(q, "q")
    a, code = _inputs(q, k, v, log_alpha, beta, k_scale, q_scale, state_in, lengths, device)
    B, Hv, T, D = vshape = v.shape
    kshape, dtype, f32 = q.shape, q.dtype, torch.float32
    dos = _rows(do, "do", vshape, dtype, device)

    def out(t, name, like):
        """The gradient of `like` and its address."""
        if t is None:
            t = torch.empty_like(like, memory_format=torch.contiguous_format)
            return t, t.data_ptr()
        return t, _full(t, name, like.shape, like.dtype, device)

    dq, pdq = out(dq, "dq", q)
    dk, pdk = out(dk, "dk", k)
    dv, pdv = out(dv, "dv", v)
    dlog_alpha, pdlog = out(dlog_alpha, "dlog_alpha", log_alpha)
    dbeta, pdbeta = out(dbeta, "dbeta", beta)
    need = _delta_need(1, code, B, kshape[1], Hv, T, D)
    if need == 0:
        raise LaScanError(LA_ERR_UNSUPPORTED, "la_gated_delta_rule_backward")
    workspace = _space(workspace, need, q)
    st = lib.la_gated_delta_rule_backward(
        a, do.data_ptr(), _pack_strides(*dos),
        _full(dstate_out, "dstate_out", (B, Hv, D, D), f32, device),
        pdq, pdk, pdv, pdlog, pdbeta, _full(dstate_in, "dstate_in", (B, Hv, D, D), f32, device),
        workspace.data_ptr(), workspace.numel(), _raw_stream(device))
    if st != LA_OK:
        _raise(st, "la_gated_delta_rule_backward")
    return dq, dk, dv, dlog_alpha, dbeta


def la_add_rms_norm_fp8(x, residual, weight, eps: float = 1e-6, group: int = 128, h=None, y=None,
                        scale=None, stream=None):
    """Residual addition, RMSNorm and e4m3 output.  x, residual ``[..., N]`` (residual may be
    None), weight ``[N]`` float32.  Returns (y float8_e4m3fn ``[..., N]``, scale float32
    ``[..., ceil(N / group)]`` (group = 0: ``[..., 1]``), h = x + residual as stored, which is x
    itself without a residual).  ``y.float() * scale`` (each scale over its group) is the norm."""
    if stream is not None:
        done = _elsewhere(stream, la_add_rms_norm_fp8, x, residual, weight, eps, group, h, y, scale)
        if done is not NotImplemented:
            return done
    if weight is None:
        raise ValueError("weight is required")
    shape, dtype = x.shape, x.dtype
    N = shape[-1]
    dt = _dtype_code(x)
    if group not in (0, 128):
        raise ValueError(f"group must be 128 or 0 (the row), got {group}")
    device = _here(x, "x")
    groups = (*shape[:-1], -(-N // group) if group else 1)
    px, pr = _full(x, "x", shape, dtype, device), _full(residual, "residual", shape, dtype, device)
    pw = _full(weight, "weight", (N,), torch.float32, device)
    if h is not None:
        ph = _full(h, "h", shape, dtype, device)
    elif residual is not None:
        h = torch.empty_like(x)
        ph = h.data_ptr()
    else:
        ph = None
    if y is None:
        y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        py = y.data_ptr()
    else:
        py = _full(y, "y", shape, torch.float8_e4m3fn, device)
    if scale is None:
        scale = weight.new_empty(groups)
        ps = scale.data_ptr()
    else:
        ps = _full(scale, "scale", groups, torch.float32, device)
    st = lib.la_add_rms_norm_fp8(px, pr, pw, ph, py, ps, dt, x.numel() // N if N else 0, N, group,
                                 eps, _raw_stream(device))
    if st != LA_OK:
        _raise(st, "la_add_rms_norm_fp8")
    return y, scale, x if h is None else h


def la_add_rms_norm_backward(dy, h, weight, dh=None, eps: float = 1e-6, dx=None, dweight=None,
                             need_dweight: bool = True, workspace=None, stream=None):
    """Gradients (dx, dweight) of the norm for the gradient `dy` of its output (the 8-bit
    rounding passed straight through), h as the forward pass returned it and `dh`, the gradient
    that h gets from elsewhere.  dx is the gradient of x and of residual alike; dweight is None
    when need_dweight is False."""
    if stream is not None:
        done = _elsewhere(stream, la_add_rms_norm_backward, dy, h, weight, dh, eps, dx, dweight,
                          need_dweight, workspace)
        if done is not NotImplemented:
            return done
    if weight is None:
        raise ValueError("weight is required")
    shape, dtype = h.shape, h.dtype
    N = shape[-1]
    dt = _dtype_code(h)
    device = _here(h, "h")
    rows = h.numel() // N if N else 0
    ph, pdy = _full(h, "h", shape, dtype, device), _full(dy, "dy", shape, dtype, device)
    pw, pdh = _full(weight, "weight", (N,), torch.float32, device), \
        _full(dh, "dh", shape, dtype, device)
    if dx is None:
        dx = torch.empty_like(h)
        pdx = dx.data_ptr()
    else:
        pdx = _full(dx, "dx", shape, dtype, device)
    pdw, space, size = None, None, 0
    if need_dweight:
        if dweight is None:
            dweight = torch.empty_like(weight)
        pdw = _full(dweight, "dweight", (N,), torch.float32, device)
        workspace = _space(workspace, _norm_need(rows, N), h)
        space, size = workspace.data_ptr(), workspace.numel()
    else:
        dweight = None
    st = lib.la_add_rms_norm_backward(pdy, ph, pw, pdh, pdx, pdw, dt, rows, N, eps, space, size,
                                      _raw_stream(device))
    if st != LA_OK:
        _raise(st, "la_add_rms_norm_backward")
    return dx, dweight

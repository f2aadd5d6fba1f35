"""The token-wise entry points on a machine without a GPU: what they export and
what they refuse before touching CUDA."""
import ctypes
import os
import re

import pytest
import torch

import linear_attention_video_frame_b200 as la

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "la_token.h")
INVALID, UNSUPPORTED = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED


def test_header_symbols_are_exported():
    names = re.findall(r"LA_API\s+[\w\s\*]+?\b(la_\w+)\s*\(", open(HEADER).read())
    assert sorted(set(names)) == sorted([
        "la_gated_delta_rule", "la_gated_delta_rule_backward", "la_gated_delta_step",
        "la_delta_workspace_size", "la_delta_plan", "la_add_rms_norm_fp8",
        "la_add_rms_norm_backward", "la_norm_workspace_size"])
    for n in names:
        assert hasattr(la.lib, n)


def _delta(**kw):
    B, Hk, Hv, T, D = (kw.pop(n, d) for n, d in zip(("B", "Hk", "Hv", "T", "D"), (2, 2, 4, 80, 64)))
    s = lambda H: la.token_ops._Strides(H * T * D, T * D, D)
    a = la.LaDelta(4096, 8192, 12288, s(Hk), s(Hk), s(Hv), 16384, 20480, None, None, 1.0, 1.0,
                   la.LA_BF16, B, Hk, Hv, T, D)
    for n, v in kw.items():
        if n.endswith("_stride"):
            v = la.token_ops._Strides(*v)
        setattr(a, n, v)
    return a


def _call(a, o=1 << 20, os=None, state=None, ws=1 << 24, bytes_=1 << 40):
    os = la.token_ops._Strides(*(os or (a.Hv * a.T * a.D, a.T * a.D, a.D)))
    return la.lib.la_gated_delta_rule(ctypes.byref(a), o, os, state, ws, bytes_, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(log_alpha=None), INVALID), (dict(beta=None), INVALID),
    (dict(Hk=3), INVALID), (dict(Hk=0), INVALID), (dict(B=0), INVALID), (dict(T=-1), INVALID),
    (dict(B=70000), INVALID), (dict(dt=7), INVALID),
    (dict(D=24), UNSUPPORTED), (dict(D=272), UNSUPPORTED), (dict(D=8), UNSUPPORTED),
    (dict(k_scale=float("nan")), INVALID), (dict(q_scale=float("inf")), INVALID),
    (dict(q_stride=(-64, 64, 64)), INVALID), (dict(k_stride=(64, 60, 64)), INVALID),
    (dict(v_stride=(64, 64, 1 << 62)), INVALID),
    (dict(T=2000000000), INVALID),
])
def test_delta_refusals(change, status):
    assert _call(_delta(**change)) == status
    a = _delta(**change)
    st = la.token_ops._Strides(0, 0, 0)
    assert la.lib.la_gated_delta_rule_backward(
        ctypes.byref(a), 1 << 20, st, None, 1 << 21, 1 << 22, 1 << 23, 1 << 24, 1 << 25, None,
        1 << 26, 1 << 40, None) == status


def test_delta_output_and_workspace_refusals():
    a = _delta()
    assert _call(a, o=None) == INVALID
    assert _call(a, os=(20480, 5120, 32)) == INVALID          # rows of o on one another
    assert _call(a, os=(20480, 0, 64)) == INVALID
    assert _call(a, os=(20480, 5120, 68)) == INVALID          # not whole 16-byte pieces
    assert _call(a, ws=None) == INVALID
    assert _call(a, ws=(1 << 24) + 16) == INVALID
    n = la.la_delta_workspace_size(False, la.LA_BF16, 2, 2, 4, 80, 64)
    assert n % 256 == 0 and _call(a, bytes_=n - 1) == INVALID
    assert la.lib.la_gated_delta_rule(None, None, None, None, None, 0, None) == INVALID


def test_step_and_backward_refusals():
    a = _delta(T=1)
    os = la.token_ops._Strides(256, 64, 64)
    assert la.lib.la_gated_delta_step(ctypes.byref(a), 1 << 20, os, None, None) == INVALID
    a = _delta(T=2)
    assert la.lib.la_gated_delta_step(ctypes.byref(a), 1 << 20, os, 1 << 21, None) == INVALID
    a = _delta(D=144)
    st = la.token_ops._Strides(0, 0, 0)
    back = lambda a, do=1 << 20, dq=1 << 21: la.lib.la_gated_delta_rule_backward(
        ctypes.byref(a), do, st, None, dq, 1 << 22, 1 << 23, 1 << 24, 1 << 25, None, 1 << 26,
        1 << 40, None)
    assert back(a) == UNSUPPORTED
    assert back(_delta(), do=None) == INVALID and back(_delta(), dq=None) == INVALID


def test_delta_sizes_and_plans():
    for dt, heads, first in ((la.LA_BF16, 1, 24), (la.LA_BF16, 64, 16), (la.LA_F32, 1, 40),
                             (la.LA_F32, 64, 24)):
        assert la.la_delta_plan(False, dt, 1, 1, heads, first - 1, 64) == ("delta_recurrent", 1)
        assert la.la_delta_plan(False, dt, 1, 1, heads, first, 64) == ("delta_chunked", 2)
    assert la.la_delta_plan(False, la.LA_F32, 1, 1, 1, 64, 144)[0] == "delta_recurrent"
    assert la.la_delta_plan(True, la.LA_BF16, 1, 1, 1, 1, 64)[0] != "delta_recurrent"
    assert la.la_delta_plan(True, la.LA_BF16, 1, 1, 1, 1, 144) == (None, 0)
    for bad in ((0, 1, 1, 4, 64), (1, 2, 3, 4, 64), (1, 1, 1, -1, 64), (1, 1, 1, 4, 40)):
        assert la.la_delta_workspace_size(False, la.LA_BF16, *bad) == 0
        with pytest.raises(la.LaScanError):
            la.delta_workspace_for(False, la.LA_BF16, *bad, device="cpu")


def test_norm_refusals():
    f = la.lib.la_add_rms_norm_fp8
    ok = dict(x=4096, res=None, w=8192, h=None, y=1 << 20, s=1 << 21, dt=1, rows=2, N=128, g=128,
              eps=1e-6)
    call = lambda **kw: f(*{**ok, **kw}.values(), None)
    assert call(x=None) == call(w=None) == call(y=None) == call(s=None) == INVALID
    assert call(g=64) == call(rows=-1) == call(dt=9) == INVALID
    assert call(eps=float("nan")) == call(eps=-1.0) == INVALID
    assert call(N=24) == call(N=16400) == call(N=0) == UNSUPPORTED
    assert call(rows=0) == la.LA_OK
    g = la.lib.la_add_rms_norm_backward
    ok2 = dict(dy=4096, h=8192, w=1 << 20, dh=None, dx=1 << 21, dw=1 << 22, dt=1, rows=2, N=128,
               eps=1e-6, ws=1 << 23, n=1 << 30)
    call = lambda **kw: g(*{**ok2, **kw}.values(), None)
    assert call(dy=None) == call(h=None) == call(dx=None) == call(ws=None) == INVALID
    assert call(ws=(1 << 23) + 4) == call(n=16) == INVALID
    assert call(N=40) == UNSUPPORTED
    assert la.la_norm_workspace_size(3, 40) == 0 and la.la_norm_workspace_size(3, 128) % 256 == 0


def test_binding_checks_tensors():
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 1, 4)
    with pytest.raises(ValueError):
        la.la_gated_delta_rule(q, q, q, g, g)                 # not on the GPU
    with pytest.raises(ValueError):
        la.la_gated_delta_step(q, q, q, g, g, None)           # four axes
    with pytest.raises((ValueError, TypeError)):
        la.la_add_rms_norm_fp8(q.half(), None, g)
    with pytest.raises(ValueError):
        la.la_add_rms_norm_fp8(q, None, torch.zeros(64))


def test_workspaces_of_a_call():
    """A given workspace counts by the bytes that lie behind its address."""
    like, space = torch.zeros(4), la.token_ops._space
    whole = torch.zeros(512, dtype=torch.uint8)
    assert space(whole, 256, like) is whole and space(None, 256, like).numel() == 256
    for view in (torch.zeros(1, dtype=torch.uint8).expand(512), whole[::2]):
        with pytest.raises(ValueError, match="workspace"):
            space(view, 256, like)


def test_missing_tensors_are_named():
    rows, gates = torch.zeros(1, 1, 4, 64), torch.zeros(1, 1, 4)
    inputs = lambda k=rows, log_alpha=gates, beta=gates: la.token_ops._inputs(
        rows, k, rows, log_alpha, beta, 1.0, 1.0, None, None, -1)
    assert inputs()[1] == la.LA_F32
    for name in ("k", "log_alpha", "beta"):
        with pytest.raises(ValueError, match=name + " is required"):
            inputs(**{name: None})
    for call in (lambda: la.la_add_rms_norm_fp8(rows, None, None),
                 lambda: la.la_add_rms_norm_backward(rows, rows, None)):
        with pytest.raises(ValueError, match="weight is required"):
            call()

"""The gated delta rule with one update per token (chunked, its backward pass,
single tokens) against its definition in float64."""
import pytest
import torch

import linear_attention_video_frame_b200 as la
from token_ref import (NAMES, U, check, check_grads, delta_bound, delta_grads_ref, delta_inputs,
                       delta_ref, to64)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.init()


def _args(x):
    return tuple(x[n] for n in ("q", "k", "v", "log_alpha", "beta"))


def _kw(x):
    return dict(k_scale=x["k_scale"], q_scale=x["q_scale"], lengths=x["lengths"])


def _forward(x, **kw):
    B, Hv, T, D = x["v"].shape
    end = torch.full((B, Hv, D, D), float("nan"), device="cuda")
    o = la.la_gated_delta_rule(*_args(x), state_in=x["state"], state_out=end, **_kw(x), **kw)
    return o, end


def _backward(x, **kw):
    B, Hv, T, D = x["v"].shape
    dstate = torch.full((B, Hv, D, D), float("nan"), device="cuda")
    g = la.la_gated_delta_rule_backward(*_args(x), x["do"], state_in=x["state"],
                                        dstate_out=x["dstate"], dstate_in=dstate, **_kw(x), **kw)
    return dict(zip(NAMES, (*g, dstate)))


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# one token to several chunks, ends inside and at a chunk's border
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 129, 320])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_lengths(T, dtype):
    x = delta_inputs(2, 2, 4, T, 64, dtype, seed=T, state=T % 2 == 0)
    o, end = _forward(x)
    ro, rs = delta_ref(**to64(x))
    check(o, ro, delta_bound(T), "o")
    check(end, rs, delta_bound(T), "state")


@pytest.mark.parametrize("D", [16, 32, 48, 80, 96, 112, 128, 144, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_head_widths(D, dtype):
    x = delta_inputs(1, 1, 2, 150, D, dtype, seed=D, token_major=True)
    o, end = _forward(x)
    ro, rs = delta_ref(**to64(x))
    check(o, ro, delta_bound(150), "o")
    check(end, rs, delta_bound(150), "state")


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 4), (3, 6), (5, 5)])
@pytest.mark.parametrize("lengths", [[0, 130, 64], [1, 63, 129]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_ragged(Hk, Hv, lengths, dtype):
    x = delta_inputs(3, Hk, Hv, 130, 48, dtype, seed=Hv, lengths=lengths)
    for b, n in enumerate(lengths):          # what lies behind a sequence does not matter
        for name in ("q", "k", "v"):
            x[name][b, :, n:] = float("nan")
        for name in ("log_alpha", "beta"):
            x[name][b, :, n:] = float("nan")
    o = torch.full_like(x["v"], 7.0)
    got, end = _forward(x, o=o)
    clean = {**x, **{n: torch.nan_to_num(x[n]) for n in ("q", "k", "v", "log_alpha", "beta")}}
    ro, rs = delta_ref(**to64(clean))
    for b, n in enumerate(lengths):
        if n < 130:
            assert (o[b, :, n:] == 7.0).all(), "rows behind a sequence were written"
        if n:
            check(o[b:b + 1, :, :n], ro[b:b + 1, :, :n], delta_bound(130), "o")
        else:
            assert torch.equal(end[b], x["state"][b])
    check(end, rs, delta_bound(130), "state")


# long sequences of few heads, whose chains are cut into segments
@pytest.mark.parametrize("T,D,lengths", [(1601, 128, None), (64 * 33 + 7, 64, None),
                                         (1500, 112, [1500, 70, 0, 741]),
                                         (64 * 24, 128, [64 * 24, 64 * 6, 64 * 6 + 1, 64])])
def test_forward_segments(T, D, lengths):
    B = 1 if lengths is None else len(lengths)
    assert la.la_delta_plan(False, la.LA_BF16, B, 1, 1, T, D)[1] > 2
    x = delta_inputs(B, 1, 1, T, D, seed=T, lengths=lengths)
    x["log_alpha"] *= 0.1                       # states that outlive a segment
    x["log_alpha"][:, :, T // 2] = -float("inf")
    x["log_alpha"][0, :, T // 2] = 0.0
    o, end = _forward(x)
    ro, rs = delta_ref(**to64(x))
    for b, n in enumerate(lengths or [T]):
        if n:
            check(o[b:b + 1, :, :n], ro[b:b + 1, :, :n], delta_bound(T), "o")
    check(end, rs, delta_bound(T), "state")


@pytest.mark.parametrize("T,D,Hv,lengths", [(1500, 64, 2, None), (1500, 128, 1, [1500, 70, 0, 741])])
def test_backward_segments(T, D, Hv, lengths):
    B = 1 if lengths is None else len(lengths)
    assert la.la_delta_plan(True, la.LA_BF16, B, 1, Hv, T, D)[1] > 5
    x = delta_inputs(B, 1, Hv, T, D, seed=T, lengths=lengths)
    x["log_alpha"] *= 0.1
    got, ref = _backward(x), delta_grads_ref(x)
    check_grads(got, ref, x, 4 * delta_bound(T))


@pytest.mark.parametrize("T,D", [(70, 64), (200, 128), (40, 32)])
def test_forgetting_tokens(T, D):
    """log_alpha of -inf, of the type's lowest value and of 0; beta of 0 and 1."""
    x = delta_inputs(1, 2, 2, T, D, seed=T)
    x["log_alpha"][:, 0, ::7] = -float("inf")
    x["log_alpha"][:, 1, 5::31] = torch.finfo(F32).min
    x["log_alpha"][:, 1, 6:20] = 0.0
    x["beta"][:, :, ::5] = 0.0
    x["beta"][:, :, 3::5] = 1.0
    o, end = _forward(x)
    ro, rs = delta_ref(**to64(x))
    check(o, ro, delta_bound(T), "o")
    check(end, rs, delta_bound(T), "state")
    got = _backward(x)
    # autograd of exp at -inf is 0 * inf; at -2000 exp is 0 in float64 as well (1e-304 at -700)
    y = {**x, "log_alpha": x["log_alpha"].clamp_min(-2000.0)}
    check_grads(got, delta_grads_ref(y), y, 4 * delta_bound(T))


def test_nothing_read_back_from_forgotten_state():
    """A state of infinities before a token that forgets it."""
    x = delta_inputs(1, 1, 1, 3, 32, seed=5)
    x["log_alpha"][:, :, 0] = 0.0
    a, _ = _forward(x)
    assert torch.isfinite(a).all()


def test_empty_call_copies_the_state():
    x = delta_inputs(2, 1, 2, 0, 32, seed=1)
    o, end = _forward(x)
    assert o.shape[2] == 0 and torch.equal(end, x["state"])
    g = _backward(x)
    assert torch.equal(g["state"], x["dstate"])
    x["state"] = x["dstate"] = None
    assert (_forward(x)[1] == 0).all() and (_backward(x)["state"] == 0).all()


@pytest.mark.parametrize("T", [64, 200])
def test_broadcast_and_strided_inputs(T):
    """Heads expanded from one, and rows cut from a wider projection."""
    x = delta_inputs(2, 4, 4, T, 64, seed=3)
    wide = torch.randn(2, T, 4 * 64 * 3, device="cuda").to(BF16)
    x["q"] = (wide[..., :256].unflatten(-1, (4, 64)) / 8).transpose(1, 2)
    x["v"] = wide[..., 512:].unflatten(-1, (4, 64)).transpose(1, 2)
    x["k"] = x["k"][:, :1].expand(-1, 4, -1, -1)
    x["do"] = x["do"][:, :, :1].expand(-1, -1, T, -1)
    o, end = _forward(x)
    ro, rs = delta_ref(**to64(x))
    # q of a wide projection is not of unit length: |q| is about 1 here too (randn / 8)
    check(o, ro, delta_bound(T), "o")
    check(end, rs, delta_bound(T), "state")
    plain = {n: t.contiguous() if torch.is_tensor(t) else t for n, t in x.items()}
    assert _same(o, _forward(plain)[0])
    a, b = _backward(x), _backward(plain)
    assert all(_same(a[n], b[n]) for n in NAMES)


@pytest.mark.parametrize("D", [64, 128])
def test_state_in_place_and_split_calls(D):
    """A prompt in two calls and then token by token is the prompt in one call."""
    T, cut = 150, 140
    x = delta_inputs(2, 2, 4, T, D, seed=9)
    o, end = _forward(x)
    state = x["state"].clone()
    part = lambda t, a, b: t[:, :, a:b].contiguous()
    o1 = la.la_gated_delta_rule(*(part(t, 0, cut) for t in _args(x)), state_in=state,
                                state_out=state, k_scale=x["k_scale"], q_scale=x["q_scale"])
    rest = []
    for t in range(cut, T):
        rest.append(la.la_gated_delta_step(*(a[:, :, t].contiguous() for a in _args(x)), state,
                                           k_scale=x["k_scale"], q_scale=x["q_scale"]))
    ro, rs = delta_ref(**to64(x))
    check(torch.cat([o1, torch.stack(rest, 2)], 2), ro, delta_bound(T), "o")
    check(state, rs, delta_bound(T) + 8 * (T - cut) * U, "state")
    check(end, rs, delta_bound(T), "state of one call")


@pytest.mark.parametrize("B,Hk,Hv,D", [(1, 1, 1, 16), (3, 2, 6, 80), (1, 20, 20, 128),
                                       (64, 2, 2, 64), (2, 1, 3, 240), (33, 4, 8, 112)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step(B, Hk, Hv, D, dtype):
    lengths = [i % 3 for i in range(B)]      # 0 leaves a sequence alone; more than 1 is taken as 1
    x = delta_inputs(B, Hk, Hv, 1, D, dtype, seed=D + B, lengths=lengths)
    a = [t[:, :, 0] for t in _args(x)]
    a[3], a[4] = a[3].contiguous(), a[4].contiguous()
    new = torch.empty_like(x["state"])
    o = torch.full((B, Hv, D), 7.0, dtype=dtype, device="cuda")
    la.la_gated_delta_step(*a, x["state"], state_out=new, o=o, **_kw(x))
    ro, rs = delta_ref(**to64(x))
    # a token: two sums of D products, in part sums of at most 8 and their join of 32
    bound = 2 * 48 * U
    for b in range(B):
        if lengths[b] == 0:
            assert (o[b] == 7.0).all() and torch.equal(new[b], x["state"][b])
        else:
            check(o[b:b + 1, :, None], ro[b:b + 1], bound, "o")
            check(new[b:b + 1], rs[b:b + 1], bound, "state")
    inplace = x["state"].clone()
    la.la_gated_delta_step(*a, inplace, o=o, **_kw(x))
    assert _same(inplace, new)


# The backward pass runs the forward's products and as many again; a gradient
# is a sum of up to six of them.
@pytest.mark.parametrize("T", [1, 63, 64, 65, 130, 200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_lengths(T, dtype):
    x = delta_inputs(1, 1, 2, T, 64, dtype, seed=T, state=T % 2 == 0)
    got, ref = _backward(x), delta_grads_ref(x)
    check_grads(got, ref, x, 4 * delta_bound(T))


@pytest.mark.parametrize("D", [16, 48, 80, 112, 128])
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 6)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_shared_heads_ragged(D, Hk, Hv, dtype):
    lengths = [100, 0, 65]
    x = delta_inputs(3, Hk, Hv, 100, D, dtype, seed=D, lengths=lengths, token_major=True)
    got, ref = _backward(x), delta_grads_ref(x)
    check_grads(got, ref, x, 4 * delta_bound(100))
    for b, m in enumerate(lengths):
        for n in NAMES[:5]:
            assert (got[n][b, :, m:] == 0).all(), f"d{n} behind a sequence"


def test_backward_against_differences():
    """Directional derivatives of the float64 forward pass."""
    x = delta_inputs(1, 2, 4, 90, 32, F32, seed=11)
    got = _backward(x)
    y = to64(x)
    do, ds = x["do"].cpu().double(), x["dstate"].cpu().double()

    def loss(z):
        o, S = delta_ref(**z)
        return float((o * do).sum() + (S * ds).sum())

    g = torch.Generator().manual_seed(1)
    for n in NAMES:
        d = torch.randn(y[n].shape, generator=g, dtype=torch.float64)
        h = 1e-4
        plus = loss({**y, n: y[n] + h * d})
        minus = loss({**y, n: y[n] - h * d})
        slope = (plus - minus) / (2 * h)
        mine = got[n].cpu().double()
        # each element is off by at most the bound of the largest; the rest of the
        # difference quotient is of order h^2 = 1e-8
        room = 4 * delta_bound(90) * float(mine.abs().max()) * float(d.abs().sum())
        assert abs(float((mine * d).sum()) - slope) <= room + 1e-5 * abs(slope), n


def test_backward_in_place_and_without_state():
    x = delta_inputs(2, 1, 1, 70, 64, seed=2)
    want = _backward(x)
    ds = x["dstate"].clone()
    la.la_gated_delta_rule_backward(*_args(x), x["do"], state_in=x["state"], dstate_out=ds,
                                    dstate_in=ds, **_kw(x))
    assert _same(ds, want["state"])
    g = la.la_gated_delta_rule_backward(*_args(x), x["do"], state_in=x["state"],
                                        dstate_out=x["dstate"], **_kw(x))
    assert all(_same(a, want[n]) for a, n in zip(g, NAMES))


def test_equal_calls_give_equal_bits():
    x = delta_inputs(2, 4, 8, 333, 128, seed=21)
    (a, s), (b, t) = _forward(x), _forward(x)
    assert _same(a, b) and _same(s, t)
    g, h = _backward(x), _backward(x)
    assert all(_same(g[n], h[n]) for n in NAMES)


def test_graphs_on_another_stream_with_their_own_workspaces():
    """Two captured calls of different shapes, replayed against each other."""
    xs = [delta_inputs(1, 2, 2, 200, 64, seed=31), delta_inputs(2, 1, 2, 90, 128, seed=32)]
    want = [(_forward(x), _backward(x)) for x in xs]
    graphs, outs = [], []
    for x in xs:
        B, Hv, T, D = x["v"].shape
        ws = [la.delta_workspace_for(bw, la.LA_BF16, B, x["q"].shape[1], Hv, T, D)
              for bw in (False, True)]
        st = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=st):
            outs.append((_forward(x, workspace=ws[0], stream=st),
                         _backward(x, workspace=ws[1], stream=st)))
        graphs.append((g, st, ws))
    for _ in range(3):
        for g, st, _ in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (f, b), (wf, wb) in zip(outs, want):
        assert _same(f[0], wf[0]) and _same(f[1], wf[1])
        assert all(_same(b[n], wb[n]) for n in NAMES)
    del graphs, g


def test_long_sequence_offsets():
    """Rows whose element offsets pass 31 bits (a long batch with wide strides)."""
    T, D = 130, 64
    stride = (1 << 31) // T // 8 * 8 + 4096
    big = torch.empty(T * stride + D, dtype=BF16, device="cuda")
    x = delta_inputs(1, 1, 1, T, D, seed=41)
    rows = big.as_strided((1, 1, T, D), (0, 0, stride, 1))
    rows.copy_(x["k"])
    want = _forward(x)
    got = _forward({**x, "k": rows})
    assert _same(got[0], want[0]) and _same(got[1], want[1])
    o = big.as_strided((1, 1, T, D), (0, 0, stride, 1), 128)
    la.la_gated_delta_rule(*_args(x), state_in=x["state"], o=o, **_kw(x))
    assert _same(o, want[0])


def test_other_stream_without_a_workspace():
    """A call on a stream of its own keeps its own workspace until it has run, whatever the
    current stream allocates and writes meanwhile."""
    x = delta_inputs(1, 2, 2, 700, 128, seed=51)
    want = _forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B, Hv, T, D = x["v"].shape
    end = torch.empty(B, Hv, D, D, device="cuda")
    o = torch.empty_like(x["v"])
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
        la.la_gated_delta_rule(*_args(x), state_in=x["state"], state_out=end, o=o, **_kw(x),
                               stream=side)
        for _ in range(4):
            torch.full((la.la_delta_workspace_size(False, la.LA_BF16, B, 2, Hv, T, D),), 255,
                       dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert _same(o, want[0]) and _same(end, want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(0, 64), (1, 64), (200, 64), (200, 128), (3, 144)])
def test_status_of_a_call(T, D, dtype):
    """Every call leaves its status in its workspace, whatever was there."""
    x = delta_inputs(1, 2, 2, T, D, dtype, seed=60 + T)
    code = la.LA_BF16 if dtype == BF16 else la.LA_F32
    for backward in (False, True)[:1 if D > 128 else 2]:
        ws = la.delta_workspace_for(backward, code, 1, 2, 2, T, D).fill_(255)
        (_backward if backward else _forward)(x, workspace=ws)
        assert la.la_query_device_status(ws) == la.LA_OK


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 64), (1, 128), (70, 48)])
def test_first_token_has_no_state_to_forget(T, D, dtype):
    """log_alpha of a first token scales a state of zeros: its gradient is 0, not the rounding
    of terms that cancel."""
    x = delta_inputs(2, 2, 4, T, D, dtype, seed=70 + T, state=False)
    assert x["state"] is None
    g = _backward(x)["log_alpha"]
    assert (g[:, :, 0] == 0).all()
    assert T == 1 or (g[:, :, 1:] != 0).any()


def _hold(stream=None):
    """Keeps a stream busy for some milliseconds."""
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        torch.cuda._sleep(30_000_000)


# one token, token by token, by chunks
@pytest.mark.parametrize("T", [1, 10, 200])
def test_new_output_is_filled_on_the_stream_of_the_call(T):
    """Rows behind a sequence are 0 in a new output: its fill must not come after the kernels,
    whatever the current stream is busy with."""
    x = delta_inputs(2, 2, 4, T, 64, seed=80 + T, lengths=[T, T // 2])
    want = torch.zeros_like(x["v"])
    _forward(x, o=want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _hold()
    o, end = _forward(x, stream=side)
    one = None
    if T == 1:
        a = [t[:, :, 0] for t in _args(x)]
        a[3], a[4] = a[3].contiguous(), a[4].contiguous()
        torch.cuda.synchronize()
        _hold()
        one = la.la_gated_delta_step(*a, x["state"], state_out=torch.empty_like(end), **_kw(x),
                                     stream=side)
    torch.cuda.synchronize()
    assert _same(o, want)
    assert one is None or _same(one, want[:, :, 0])


def test_new_tensors_of_a_call_on_another_stream():
    """What the current stream has let go but still works on is not given to the call; what the
    call's caller lets go is not given to the current stream; and what the current stream still
    reads is not given to the next call."""
    x, z = delta_inputs(1, 2, 2, 700, 128, seed=91), delta_inputs(1, 2, 2, 700, 128, seed=92)
    want, want_z = _forward(x)[0], _forward(z)[0]
    grads = _backward(x)
    side = torch.cuda.Stream()

    def call(x, **kw):
        return la.la_gated_delta_rule(*_args(x), state_in=x["state"], **_kw(x), **kw)

    def back(x, **kw):
        return la.la_gated_delta_rule_backward(*_args(x), x["do"], state_in=x["state"],
                                               dstate_out=x["dstate"], **_kw(x), **kw)

    for f, r in ((call, (want,)), (back, [grads[n] for n in NAMES[:5]])):
        junk = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in r]
        torch.cuda.synchronize()
        _hold()
        for t in junk:
            t.fill_(7.0)
        del junk, t
        got = f(x, stream=side)
        torch.cuda.synchronize()
        got = got if isinstance(got, tuple) else (got,)
        assert all(_same(a, b) for a, b in zip(got, r))
        del got

    _hold(side)
    call(x, stream=side)                        # let go at once
    after = [torch.full_like(want, 3.0) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((t == 3.0).all() for t in after)
    del after

    o = call(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _hold()
    copy = o.clone()
    del o
    others = [call(z, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    assert _same(copy, want) and all(_same(t, want_z) for t in others)


def test_streams_by_their_addresses():
    """A stream may be given as the address of its CUDA stream."""
    x = delta_inputs(1, 2, 2, 200, 64, seed=93, lengths=[150])
    want = torch.zeros_like(x["v"])
    _forward(x, o=want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _hold()
    o, _ = _forward(x, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert _same(o, want)
    o, _ = _forward(x, stream=torch.cuda.current_stream().cuda_stream)
    assert _same(o, want)


# long chains by themselves, and in segments, whose second pass starts with the status set
@pytest.mark.parametrize("Hv,T,D", [(100, 64 * 40, 64), (100, 64 * 30, 128), (1, 1601, 128)])
@pytest.mark.parametrize("backward,skip", [(False, 2), (True, 2), (True, -3)])
def test_waits_that_run_out_are_reported(monkeypatch, Hv, T, D, backward, skip):
    """An arrival that never comes: the waits for it give up, the block ends with its copies and
    products done, the call's workspace says so, and the next call works."""
    plan = la.la_delta_plan(backward, la.LA_BF16, 1, Hv, Hv, T, D)
    assert plan == ("delta_chunked", (4 if backward else 2)) if Hv > 1 else plan[1] > 3
    x = delta_inputs(1, Hv, Hv, T, D, seed=130)
    run = _backward if backward else (lambda x, **kw: dict(zip(("o", "end"), _forward(x, **kw))))
    want = run(x)
    ws = la.delta_workspace_for(backward, la.LA_BF16, 1, Hv, Hv, T, D)
    monkeypatch.setenv("LA_DELTA_TEST_SKIP_ROWS", str(skip))
    run(x, workspace=ws)
    assert la.la_query_device_status(ws) == la.LA_ERR_TIMEOUT
    monkeypatch.delenv("LA_DELTA_TEST_SKIP_ROWS")
    got = run(x, workspace=ws)
    assert la.la_query_device_status(ws) == la.LA_OK
    assert all(_same(got[n], want[n]) for n in want)


@pytest.mark.parametrize("T", [12, 70, 200])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growth_after_a_forgotten_state(T, D, dtype):
    """Positive log_alpha behind a token that forgets: nothing of the state before it comes back.
    Without writes the state stays exactly 0."""
    x = delta_inputs(1, 2, 2, T, D, dtype, seed=100 + T)
    x["log_alpha"][:, 0, 5] = -float("inf")
    x["log_alpha"][:, 1, 5] = -105.0
    x["log_alpha"][:, :, 6], x["log_alpha"][:, :, 7] = 50.0, 30.0
    x["beta"][:, :, 5:] = 0.0
    o, end = _forward(x)
    assert (o[:, :, 5:] == 0).all() and (end == 0).all()
    ro, _ = delta_ref(**to64(x))
    check(o[:, :, :5], ro[:, :, :5], delta_bound(T), "o")


@pytest.mark.parametrize("T,D", [(70, 64), (130, 128), (40, 48)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_gradient_where_the_decay_is_zero(T, D, dtype):
    """dlog_alpha is exactly 0 wherever exp(log_alpha) is 0 in float32, not only at -inf."""
    x = delta_inputs(2, 2, 4, T, D, dtype, seed=110 + T)
    at = torch.arange(3, T, 7)
    for i, value in enumerate((-104.0, -104.5, -110.0, -128.0, -1e4, -float("inf"))):
        x["log_alpha"][:, :, at[i::6]] = value
    assert (torch.exp(x["log_alpha"][:, :, at]) == 0).all()
    got = _backward(x)
    assert (got["log_alpha"][:, :, at] == 0).all()
    y = {**x, "log_alpha": x["log_alpha"].clamp(min=-2000.0)}
    y["log_alpha"] = torch.where(y["log_alpha"] <= -104.0, -2000.0, y["log_alpha"])
    check_grads(got, delta_grads_ref(y), y, 4 * delta_bound(T))


@pytest.mark.parametrize("T,D,Hv", [(1, 64, 2), (10, 64, 2), (150, 64, 2), (150, 128, 2),
                                    (10, 144, 2), (1600, 64, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forgetting_does_not_clean_a_state(T, D, Hv, dtype):
    """A forgetting token multiplies the state by 0, so what is not finite in it stays, as NaN,
    in its value column and in no other; on every path alike."""
    x = delta_inputs(1, 1, Hv, T, D, dtype, seed=120 + T)
    x["log_alpha"][:, :, 0] = -float("inf")
    clean, clean_end = _forward(x)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_end).all()
    x["state"][:, :, 2, 3] = float("inf")
    x["state"][:, :, 1, 17] = float("nan")
    runs = [_forward(x)]
    if T == 1:
        a = [t[:, :, 0] for t in _args(x)]
        a[3], a[4] = a[3].contiguous(), a[4].contiguous()
        end = torch.empty_like(clean_end)
        o = la.la_gated_delta_step(*a, x["state"], state_out=end, **_kw(x))
        runs.append((o[:, :, None], end))
    rest = [c for c in range(D) if c not in (3, 17)]
    for o, end in runs:
        for c in (3, 17):
            assert torch.isnan(o[..., c]).all() and torch.isnan(end[..., c]).all()
        assert _same(o[..., rest], clean[..., rest]) and _same(end[..., rest], clean_end[..., rest])


@pytest.mark.parametrize("address", [0, 1])
def test_the_default_stream_by_its_address(address):
    """From another current stream: the calls wait for what the default stream has to do."""
    x = delta_inputs(1, 2, 2, 200, 64, seed=94)
    want = _forward(x)[0]
    o, early = torch.full_like(x["v"], 7.0), torch.empty_like(x["v"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _hold()                                     # the default stream
    with torch.cuda.stream(side):
        la.la_gated_delta_rule(*_args(x), state_in=x["state"], o=o, **_kw(x), stream=address)
        early.copy_(o)
        p = la.la_gated_delta_rule(*_args(x), state_in=x["state"], **_kw(x), stream=address)
    torch.cuda.synchronize()
    assert (early == 7.0).all()
    assert _same(o, want) and _same(p, want)

"""Residual addition, RMSNorm and the e4m3 output with scales, and the backward
pass, against their definitions in float64."""
import pytest
import torch

import linear_attention_video_frame_b200 as la
from token_ref import U, norm_ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.init()


def _inputs(rows, N, dtype, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, N, generator=g).to(dtype).cuda()
    r = (2 * torch.randn(rows, N, generator=g)).to(dtype).cuda() if residual else None
    w = (1 + 0.2 * torch.randn(N, generator=g)).cuda()
    return x, r, w


def _sum_bound(N):
    """A float32 sum of N squares by threads of at most 32 terms, shuffles and
    warps (5 + 16 additions): 53 half steps of the sum, half of that in its
    root, and 8 roundings of the quotients and products after it."""
    return (53 / 2 + 8) * U


def _check_forward(x, r, w, group, y, scale, h):
    y64, s64, s_of, h64 = norm_ref(x, r, w, EPS, group, x.dtype)
    b = _sum_bound(x.shape[-1])
    if r is not None:
        assert torch.equal(h.double(), h64)
    assert ((scale.double() - s64).abs() <= b * s64).all()
    # the value stored is y / scale rounded to e4m3: 2^-4 of it, or half of the
    # smallest step (2^-10) below 2^-6; y / scale is known to 2 b
    t = y64 / s_of
    err = (y.float().double() - t).abs()
    allowed = torch.maximum(t.abs() * (1 + 2 * b) * 2.0 ** -4, torch.full_like(t, 2.0 ** -10))
    assert (err <= allowed + 2 * b * t.abs()).all()
    assert (y.float().abs() <= 448).all()


@pytest.mark.parametrize("rows,N", [(1, 16), (1, 2560), (3, 128), (2, 144), (5, 1008), (7, 1040),
                                    (4, 8192), (2, 8208), (1, 16384), (700, 256)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [0, 128])
def test_forward(rows, N, dtype, group):
    for residual in (True, False):
        x, r, w = _inputs(rows, N, dtype, seed=N, residual=residual)
        y, scale, h = la.la_add_rms_norm_fp8(x, r, w, eps=EPS, group=group)
        _check_forward(x, r, w, group, y, scale, h)
        assert residual or h is x


def test_rows_of_zeros_and_small_and_large_values():
    x, r, w = _inputs(4, 256, F32, seed=1)
    x[0], r[0] = 0.0, 0.0
    x[1], r[1] = x[1] * 1e-18, r[1] * 1e-18        # squares far below eps
    x[2], r[2] = x[2] * 1e15, r[2] * 1e15
    y, scale, h = la.la_add_rms_norm_fp8(x, r, w, eps=EPS)
    assert (y[0].float() == 0).all() and (scale[0] == 1).all()
    _check_forward(x[1:], r[1:], w, 128, y[1:], scale[1:], h[1:])


@pytest.mark.parametrize("group", [0, 128])
def test_nan_and_infinity_stay_in_their_row(group):
    x, r, w = _inputs(4, 384, BF16, seed=2)
    clean = la.la_add_rms_norm_fp8(x, r, w, group=group)
    x[1, 200] = float("nan")
    x[2, 5] = float("inf")
    y, scale, h = la.la_add_rms_norm_fp8(x, r, w, group=group)
    assert torch.isnan(y[1].float()).all() and torch.isnan(scale[1]).all()
    assert torch.isnan(y[2, 5].float())
    for row in (0, 3):
        assert torch.equal(y[row].view(torch.uint8), clean[0][row].view(torch.uint8))
        assert torch.equal(scale[row], clean[1][row])


def test_in_place_and_leading_axes():
    x, r, w = _inputs(6, 512, BF16, seed=3)
    y, scale, h = la.la_add_rms_norm_fp8(x, r, w)
    r2 = r.clone().view(2, 3, 512)
    y2, s2, h2 = la.la_add_rms_norm_fp8(x.view(2, 3, 512), r2, w, h=r2)
    assert h2 is r2 and torch.equal(r2.view(6, 512), h) and s2.shape == (2, 3, 4)
    assert torch.equal(y2.view(6, 512).view(torch.uint8), y.view(torch.uint8))
    y, scale, h = la.la_add_rms_norm_fp8(x[:0], None, w)
    assert y.shape == (0, 512) and scale.shape == (0, 4)


def _grads_ref(dy, h, w, dh):
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    y = h64 / (h64.square().mean(-1, keepdim=True) + EPS).sqrt() * w64
    dx, dw = torch.autograd.grad((y * dy.double()).sum(), (h64, w64))
    return (dx if dh is None else dx + dh.double()), dw


@pytest.mark.parametrize("rows,N", [(1, 16), (1, 2560), (333, 2240), (5, 144), (700, 256),
                                    (3, 8208), (2, 16384), (2000, 32)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward(rows, N, dtype):
    h, dy, w = _inputs(rows, N, dtype, seed=N + 1)
    dh, _, _ = _inputs(rows, N, dtype, seed=N + 2, residual=False)
    for extra in (dh, None):
        dx, dw = la.la_add_rms_norm_backward(dy, h, w, dh=extra, eps=EPS)
        rx, rw = _grads_ref(dy, h, w, extra)
        h64 = h.double()
        r = 1 / (h64.square().mean(-1, keepdim=True) + EPS).sqrt()
        t = (dy.double() * w.double()).abs()
        # dx is three terms, each known to the bounds of its sums and roundings
        terms = r * t + h64.abs() * r ** 3 * (t * h64.abs()).mean(-1, keepdim=True)
        if extra is not None:
            terms = terms + extra.double().abs()
        b = 4 * _sum_bound(N)
        half = torch.finfo(dtype).eps / 2 if dtype != F32 else 0.0
        assert ((dx.double() - rx).abs() <= half * rx.abs() + (1 + half) * b * terms).all()
        # a sum over the rows: blocks of rows, then at most 32 + 5 joins
        each = (dy.double() * h64 * r).abs().sum(0)
        steps = min(rows, 32 + 5 + (rows + 147) // 148 * 2) + 40
        assert ((dw.double() - rw).abs() <= (steps * U + 2 * b) * each).all()


def test_backward_against_differences():
    h, dy, w = _inputs(3, 160, F32, seed=5)
    dx, dw = la.la_add_rms_norm_backward(dy, h, w, eps=EPS)

    def loss(h64, w64):
        return float((h64 / (h64.square().mean(-1, keepdim=True) + EPS).sqrt() * w64
                      * dy.double()).sum())

    d = torch.randn_like(h64 := h.double())
    e = torch.randn_like(w64 := w.double())
    step = 1e-5
    slope = (loss(h64 + step * d, w64) - loss(h64 - step * d, w64)) / (2 * step)
    assert abs(float((dx.double() * d).sum()) - slope) <= 1e-5 * float((dx.double() * d).abs().sum())
    slope = (loss(h64, w64 + step * e) - loss(h64, w64 - step * e)) / (2 * step)
    assert abs(float((dw.double() * e).sum()) - slope) <= 1e-5 * float((dw.double() * e).abs().sum())


def test_backward_in_place_without_weight_gradient_and_no_rows():
    h, dy, w = _inputs(9, 256, BF16, seed=6)
    dx, dw = la.la_add_rms_norm_backward(dy, h, w)
    d2 = dy.clone()
    got, none = la.la_add_rms_norm_backward(d2, h, w, dx=d2, need_dweight=False)
    assert none is None and got is d2 and torch.equal(d2, dx)
    dx, dw = la.la_add_rms_norm_backward(dy[:0], h[:0], w)
    assert dx.shape == (0, 256) and (dw == 0).all()


def test_equal_calls_give_equal_bits_and_graphs_replay():
    h, dy, w = _inputs(900, 640, BF16, seed=7)
    want = la.la_add_rms_norm_backward(dy, h, w)
    wf = la.la_add_rms_norm_fp8(dy, h, w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = la.la_add_rms_norm_backward(dy, h, w, stream=st)
        gf = la.la_add_rms_norm_fp8(dy, h, w, stream=st)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(gf, wf))
    del g


def test_half_block_of_a_decoder():
    """norm -> projections -> delta rule -> norm, as a block runs them, and its
    backward pass, in float32 against float64 autograd."""
    B, T, H, D, N = 2, 100, 2, 32, 128
    g = torch.Generator().manual_seed(8)
    x, res = (torch.randn(B, T, N, generator=g).cuda() for _ in range(2))
    w1, w2 = ((1 + 0.1 * torch.randn(N, generator=g)).cuda() for _ in range(2))
    wq, wk, wv = (torch.randn(N, H * D, generator=g).cuda() / N for _ in range(3))
    wo = torch.randn(H * D, N, generator=g).cuda() / 8
    la_, be = (-0.1 * torch.rand(B, H, T, generator=g)).cuda(), torch.rand(B, H, T, generator=g).cuda()

    y8, s, h = la.la_add_rms_norm_fp8(x, res, w1, eps=EPS)
    y = y8.float() * s.repeat_interleave(128, -1)[..., :N]
    heads = lambda t: t.unflatten(-1, (H, D)).transpose(1, 2)
    q, k, v = (heads(y.double() @ m.double()).float() for m in (wq, wk, wv))
    o = la.la_gated_delta_rule(q, k, v, la_, be, q_scale=D ** -0.5)
    a = (o.transpose(1, 2).flatten(2).double() @ wo.double()).float()
    z8, s2, h2 = la.la_add_rms_norm_fp8(a, h, w2, eps=EPS)
    dz = torch.randn(B, T, N, generator=g).cuda()
    dh2, dw2 = la.la_add_rms_norm_backward(dz, h2, w2, eps=EPS)
    do = heads((dh2.double() @ wo.double().T).float())
    grads = la.la_gated_delta_rule_backward(q, k, v, la_, be, do, q_scale=D ** -0.5)
    flat = lambda t: t.transpose(1, 2).flatten(2).double()
    dy = sum(flat(t) @ m.double().T for t, m in zip(grads[:3], (wq, wk, wv))).float()
    dx, dw1 = la.la_add_rms_norm_backward(dy, h, w1, dh=dh2, eps=EPS)

    from token_ref import delta_ref
    leaves = [t.double().cpu().requires_grad_() for t in (h, w1, w2, la_, be)]
    hr, w1r, w2r, lar, ber = leaves
    n1 = hr / (hr.square().mean(-1, keepdim=True) + EPS).sqrt() * w1r
    yr = n1 + (y.double().cpu() - n1).detach()           # the 8-bit rounding passed straight through
    qr, kr, vr = (heads(yr @ m.double().cpu()) for m in (wq, wk, wv))
    orr, _ = delta_ref(qr, kr, vr, lar, ber, q_scale=float(torch.tensor(D ** -0.5)))
    h2r = hr + orr.transpose(1, 2).flatten(2) @ wo.double().cpu()
    z = h2r / (h2r.square().mean(-1, keepdim=True) + EPS).sqrt() * w2r
    ref = torch.autograd.grad((z * dz.double().cpu()).sum(), leaves)
    # four operators and six float32 roundings between them; each is known to about 1e-5
    # (delta_bound(100) = 3e-5) of its largest value
    for got, r in zip((dx, dw1, dw2, grads[3], grads[4]), ref):
        assert (got.double().cpu() - r).abs().max() <= 4e-4 * r.abs().max()


def test_new_outputs_on_another_stream():
    """New outputs of a call on a stream that is not the current one: not what the current
    stream still writes to, and not given to it before the call has run."""
    x, r, w = _inputs(300, 640, BF16, seed=17)
    want = la.la_add_rms_norm_fp8(x, r, w)
    dx, dw = la.la_add_rms_norm_backward(x, r, w)
    side = torch.cuda.Stream()
    junk = [torch.empty_like(t) for t in (*want, dx, dw)]
    torch.cuda.synchronize()
    torch.cuda._sleep(30_000_000)
    for t in junk:
        t.view(torch.uint8).fill_(7)
    del junk, t
    got = (*la.la_add_rms_norm_fp8(x, r, w, stream=side),
           *la.la_add_rms_norm_backward(x, r, w, stream=side))
    torch.cuda.synchronize()
    for a, b in zip(got, (*want, dx, dw)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    with torch.cuda.stream(side):
        torch.cuda._sleep(30_000_000)
    y, scale, _ = la.la_add_rms_norm_fp8(x, r, w, stream=side)
    del _
    after = [torch.full_like(x, 3.0) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((t == 3.0).all() for t in after)
    assert torch.equal(y.view(torch.uint8), want[0].view(torch.uint8))


@pytest.mark.parametrize("N", [256, 1040])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [0, 128])
def test_scale_that_underflows(N, dtype, group):
    """max |y| / 448 may be 0 in float32 though y is not: the scale is 1 there as well, and
    the values, far below e4m3's smallest, are 0."""
    x, r, w = _inputs(3, N, dtype, seed=N)
    x[:, ::3], r[:, ::3] = 0.0, 0.0
    y, scale, h = la.la_add_rms_norm_fp8(x, r, w * 1e-44, eps=EPS, group=group)
    assert (scale == 1).all()
    assert (y.float() == 0).all()


def _check_backward(dy, h, w, dh, eps, dx, dw=None, steps=0):
    """dx, and dw as a sum of `steps` roundings, against float64."""
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    y = h64 / (h64.square().mean(-1, keepdim=True) + eps).sqrt() * w64
    rx, rw = torch.autograd.grad((y * dy.double()).sum(), (h64, w64))
    h64 = h64.detach()
    r = 1 / (h64.square().mean(-1, keepdim=True) + eps).sqrt()
    t = (dy.double() * w.double()).abs()
    # dx is three terms, each known to the bounds of its sums and roundings
    terms = r * t + h64.abs() * r ** 3 * (t * h64.abs()).mean(-1, keepdim=True)
    if dh is not None:
        rx, terms = rx + dh.double(), terms + dh.double().abs()
    b = 4 * _sum_bound(h.shape[-1])
    half = torch.finfo(h.dtype).eps / 2 if h.dtype != F32 else 0.0
    assert ((dx.double() - rx).abs() <= half * rx.abs() + (1 + half) * b * terms).all()
    if dw is not None:
        each = (dy.double() * h64 * r).abs().sum(0)
        assert ((dw.double() - rw).abs() <= (steps * U + 2 * b) * each).all()


@pytest.mark.parametrize("N", [144, 1040, 4800, 8208])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size,eps", [(1e13, EPS), (1e15, EPS), (1e17, EPS), (1e-15, 0.0),
                                      (1e-17, 0.0)])
def test_backward_of_large_and_small_rows(N, dtype, size, eps):
    """The cube of 1 / rms leaves float32's range long before the gradient does."""
    h, dy, w = _inputs(3, N, dtype, seed=N)
    h = (h.float() * size).to(dtype)
    dx, dw = la.la_add_rms_norm_backward(dy, h, w, eps=eps)
    _check_backward(dy, h, w, None, eps, dx, dw, steps=3 + 40)


# a vector, two or four a thread; rows from the ring in shared memory or from memory; a
# warp a row and several
@pytest.mark.parametrize("rows,N,dtype", [
    (7001, 144, BF16), (6001, 1008, BF16), (6001, 1008, F32), (4003, 2240, BF16),
    (3001, 2240, F32), (2003, 4800, F32), (1501, 8192, BF16), (1501, 8192, F32),
    (1201, 8448, BF16), (1201, 8448, F32), (1000, 16384, BF16), (1000, 16384, F32)])
def test_backward_of_many_rows(rows, N, dtype):
    """Several rows a block: at most 20 blocks an SM of 148, 2960, and no more than about 640
    threads an SM from 32 a row on."""
    threads = -(-N // 8 // (1 if N <= 1024 else 2 if N <= 8192 else 4) // 32) * 32
    assert rows > 148 * max(1, 640 // threads)
    h, dy, w = _inputs(rows, N, dtype, seed=N + 3)
    dh = _inputs(rows, N, dtype, seed=N + 4, residual=False)[0]
    # a sum over the rows: those of a block (at least 148 blocks), then of the blocks' sums
    # (at most 2960) up to 93 by one of 32 threads, and 10 joins
    steps = -(-rows // 148) + 93 + 10
    for extra in (dh, None):
        dx, dw = la.la_add_rms_norm_backward(dy, h, w, dh=extra, eps=EPS)
        _check_backward(dy, h, w, extra, EPS, dx, dw, steps)

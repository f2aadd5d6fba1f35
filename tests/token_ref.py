"""float64 forms of the token-wise operators, straight from their definitions
(token by token; differentiable), and the error bounds of the tests."""
import torch

U = 2.0 ** -24                      # half a step of float32


def delta_inputs(B, Hk, Hv, T, D, dtype=torch.bfloat16, seed=0, state=True, lengths=None,
                 token_major=False, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def rows(H, unit):
        t = torch.randn(B, T, H, D, generator=g) if token_major else \
            torch.randn(B, H, T, D, generator=g)
        if unit:
            t = t / t.norm(dim=-1, keepdim=True)
        t = t.to(dtype).to(device)
        return t.transpose(1, 2) if token_major else t

    rate = torch.exp(torch.empty(B, Hv, 1).uniform_(-7.0, -1.6, generator=g))
    x = dict(q=rows(Hk, True), k=rows(Hk, True), v=rows(Hv, False),
             log_alpha=(-rate * torch.rand(B, Hv, T, generator=g) * 2).to(device),
             beta=torch.rand(B, Hv, T, generator=g).to(device),
             state=torch.randn(B, Hv, D, D, generator=g).mul(0.3).to(device) if state else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32,
                                                               device=device),
             do=rows(Hv, False),
             dstate=torch.randn(B, Hv, D, D, generator=g).mul(0.3).to(device) if state else None)
    x["k_scale"], x["q_scale"] = 0.9, D ** -0.5
    return x


def delta_ref(q, k, v, log_alpha, beta, state=None, lengths=None, k_scale=1.0, q_scale=1.0):
    """o [B, Hv, T, D] and the final state; rows behind a sequence are 0."""
    B, Hk, T, D = q.shape
    Hv = v.shape[1]
    q, k = (t.repeat_interleave(Hv // Hk, dim=1) for t in (q * q_scale, k * k_scale))
    S = q.new_zeros(B, Hv, D, D) if state is None else state
    out = []
    for t in range(T):
        a = torch.exp(log_alpha[:, :, t])[..., None, None]
        kt = k[:, :, t]
        z = v[:, :, t] - a[..., 0] * torch.einsum("bhk,bhkv->bhv", kt, S)
        new = a * S + torch.einsum("bhk,bhv->bhkv", kt, beta[:, :, t, None] * z)
        if lengths is not None:
            on = (t < lengths)[:, None, None, None]
            new = torch.where(on, new, S)
        S = new
        o = torch.einsum("bhk,bhkv->bhv", q[:, :, t], S)
        out.append(o if lengths is None else torch.where(on[..., 0], o, 0.0))
    return (torch.stack(out, 2) if out else v.new_zeros(B, Hv, 0, D)), S


NAMES = ("q", "k", "v", "log_alpha", "beta", "state")


def to64(x):
    """The inputs on the CPU in float64."""
    y = {n: x[n].detach().cpu().double() for n in NAMES if x[n] is not None}
    y["lengths"] = None if x["lengths"] is None else x["lengths"].cpu()
    y["k_scale"], y["q_scale"] = x["k_scale"], x["q_scale"]
    # float32 scales are what the kernels are given
    y["k_scale"], y["q_scale"] = (float(torch.tensor(y[n], dtype=torch.float32))
                                  for n in ("k_scale", "q_scale"))
    return y


def delta_grads_ref(x):
    y = to64(x)
    leaves = {n: y[n].requires_grad_() for n in NAMES if n in y}
    if "state" not in leaves:
        B, Hv, T, D = x["v"].shape
        leaves["state"] = y["state"] = torch.zeros(B, Hv, D, D, dtype=torch.float64,
                                                   requires_grad=True)
    Hv = x["v"].shape[1]
    z = dict(y, q=y["q"].repeat_interleave(Hv // y["q"].shape[1], 1))
    z["k"] = y["k"].repeat_interleave(Hv // y["k"].shape[1], 1)
    o, S = delta_ref(**z)
    loss = (o * x["do"].cpu().double()).sum()
    if x["dstate"] is not None:
        loss = loss + (S * x["dstate"].cpu().double()).sum()
    g = torch.autograd.grad(loss, [*leaves.values(), z["q"]])
    return dict(zip([*leaves, "q_each"], g))      # q_each: by value head


def delta_bound(T):
    """Largest error of a float32 result, relative to the largest value of its head.

    A chunk of 64 tokens is a sequence of eight products (sums of up to 128
    terms).  The tensor core adds them in groups of 16, four to eight groups a
    sum, each of which costs at most a step (2 U, it rounds towards zero), and
    the joins of part sums cost three more; a result read at its largest value
    is off by at most 8 * 11 * 2 U, the values' cancellation aside, and errors
    of one chunk's state reach the next ones undiminished where nothing decays.
    """
    chunks = (T + 63) // 64
    return 176 * U * (chunks + 1)


def check_grads(got, ref, x, bound):
    """All six gradients.  dlog_alpha is the sum, from a token to its chunk's
    end, of q . dq - v . dv, and of <dS, S> there: a difference of terms that
    may cancel (they do at a first token without a state, whose gradient is 0),
    each known to `bound` of its own size, so what it is off by is relative to
    the terms: the largest sum over 64 tokens of |q . dq| + |v . dv|, and the
    largest gradient itself for <dS, S>."""
    for n in NAMES:
        top = None
        if n == "log_alpha":
            y = to64(x)
            r = x["v"].shape[1] // x["q"].shape[1]
            qdq = (y["q"].repeat_interleave(r, 1) * ref["q_each"]).sum(-1).abs()
            terms = qdq + (y["v"] * ref["v"]).sum(-1).abs()
            pad = torch.nn.functional.pad(terms, (0, -terms.shape[-1] % 64)).unflatten(-1, (-1, 64))
            top = pad.sum(-1).amax(-1) + ref[n].abs().amax(-1)
        check(got[n], ref[n], bound, "d" + n, top)


def check(got, ref, bound, what="", top=None):
    """Elementwise: half a step of the stored type, and `bound` of the largest
    value of each [batch, head] slice (for what was summed in float32)."""
    got64, ref = got.detach().cpu().double(), ref.detach()
    assert torch.isfinite(got64).all(), f"{what}: not finite"
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    if top is None:
        top = ref.abs().flatten(2).amax(-1) if ref.dim() > 2 and ref[0, 0].numel() else ref.abs()
    top = top.reshape(top.shape + (1,) * (ref.dim() - top.dim()))
    err = (got64 - ref).abs()
    # the rounding is relative to the value before it: up to the bound away from ref
    allowed = half * (ref.abs() + bound * top) + bound * top
    over = err - allowed
    assert (over <= 0).all(), f"{what}: off by {err.flatten()[over.argmax()]:.3e}, allowed " \
        f"{allowed.expand_as(err).flatten()[over.argmax()]:.3e}"


def norm_ref(x, residual, weight, eps, group, dtype):
    h = x.double()
    if residual is not None:
        h = (h + residual.double()).float().to(dtype).double()
    y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    N = x.shape[-1]
    group = group or N
    tops = torch.stack([p.abs().amax(-1) for p in y.split(group, dim=-1)], -1)
    scale = torch.where(tops == 0, 1.0, tops / 448.0)
    return y, scale, scale[..., torch.arange(N, device=x.device) // group], h

"""Cases of the token-wise operators: the gated delta rule (chunked, its
backward pass, one token at a time) and the residual addition with RMSNorm
and an e4m3 output (and its backward pass).

``run`` computes an operator in its plain form with elementary torch
operations, or, where ``own`` is true, through this package's entry points.
``exact`` computes the same outputs in float64 from the token-by-token
definitions.
"""
import math

import torch

own = False

CHUNK = 64          # tokens the plain form takes at a time
NO_DECAY_BELOW = -128.0   # exp of it is 0 in float32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _delta(name, op, B, Hk, Hv, T, D, dtype="bf16", padded=False, state=True, token_major=False,
           resets=False):
    return dict(name=name, op=op, B=B, Hk=Hk, Hv=Hv, T=T, D=D, dtype=dtype, padded=padded,
                state=state, token_major=token_major, resets=resets)


def _norm(name, op, rows, N, dtype="bf16", group=128, residual=True):
    return dict(name=name, op=op, rows=rows, N=N, dtype=dtype, group=group, residual=residual)


def listed():
    return [
        # one long document through a layer of 20 heads of 128 (prefill)
        _delta("delta long prompt", "delta", 1, 20, 20, 16384, 128, state=False),
        # a batch of prompts of unequal lengths, projections left token-major, fewer key heads
        _delta("delta padded batch", "delta", 4, 10, 20, 2047, 128, padded=True, token_major=True),
        # one short prompt that continues a state; heads of 64
        _delta("delta short prompt", "delta", 1, 8, 8, 77, 64),
        # float32 inputs (numerics work), heads of 112, packed documents that reset the state
        _delta("delta float32", "delta", 2, 20, 20, 1000, 112, dtype="f32", resets=True),
        # a training step's sequences
        _delta("delta backward", "delta_backward", 2, 16, 16, 4096, 128, state=False),
        # training on ragged sequences with shared key heads of 64
        _delta("delta backward shared", "delta_backward", 2, 4, 16, 1023, 64, padded=True,
               token_major=True),
        # decoding one sequence: latency
        _delta("delta step single", "delta_step", 1, 20, 20, 1, 128),
        # decoding a large batch: the states' traffic
        _delta("delta step batch", "delta_step", 192, 16, 32, 1, 128),
        # the norm before a decode step's projections, one sequence
        _norm("norm single", "norm", 1, 2560),
        # the norm over four streams of eight frames of 880 tokens, width 20 x 128
        _norm("norm stream", "norm", 28160, 2560),
        # gradient over a training batch
        _norm("norm backward", "norm_backward", 8192, 2560),
        # gradient over a short ragged batch, float32, width 20 x 112
        _norm("norm backward float32", "norm_backward", 333, 2240, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_backward", "delta_step", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        N = 16 * _log_int(rng, 4, 1024)
        rows = _log_int(rng, 1, max(1, min(65536, (20_000_000 if op == "norm" else 10_000_000) // N)))
        return dict(op=op, rows=rows, N=N, dtype=dtype, group=rng.choice([0, 128]),
                    residual=rng.random() < 0.7)
    Hk, ratio = rng.choice([1, 2, 4, 5, 8, 10, 16, 20]), rng.choice([1, 1, 2, 4])
    Hv = Hk * ratio
    D = rng.choice([16, 32, 48, 64, 64, 80, 96, 112, 128, 128, 128])
    if op == "delta_step":
        B, T = _log_int(rng, 1, max(1, 4096 // Hv)), 1
    else:
        B = rng.choice([1, 1, 2, 3, 4])
        most = 200_000 if op == "delta" else 80_000
        if dtype == "f32":
            most //= 4
        T = _log_int(rng, 1, max(1, min(16384 if op == "delta" else 4096, most // (B * Hv))))
    return dict(op=op, B=B, Hk=Hk, Hv=Hv, T=T, D=D, dtype=dtype, padded=rng.random() < 0.4,
                state=rng.random() < 0.5 or op == "delta_step", token_major=rng.random() < 0.5,
                resets=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _dtype(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] in ("norm", "norm_backward"):
        rows, N = case["rows"], case["N"]
        # a residual stream has a few wide channels
        wide = 1.0 + 9.0 * (torch.rand(N, generator=g, device="cuda") < 0.01).float()
        s = dict(case=case, x=(randn(rows, N) * wide).to(dt), weight=1.0 + 0.1 * randn(N))
        s["residual"] = (2.0 * randn(rows, N) * wide).to(dt) if case["residual"] else None
        if case["op"] == "norm_backward":
            s["dy"] = randn(rows, N).to(dt)
        return s

    B, Hk, Hv, T, D = (case[n] for n in ("B", "Hk", "Hv", "T", "D"))

    def heads(H, unit):
        t = randn(B, T, H, D) if case["token_major"] else randn(B, H, T, D)
        if unit:
            t = t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)
        t = t.to(dt)
        return t.transpose(1, 2) if case["token_major"] else t

    s = dict(case=case, q=heads(Hk, True), k=heads(Hk, True), v=heads(Hv, False))
    # decays from nearly none to about 0.8 a token, one rate for each head
    rate = torch.exp(torch.empty(B, Hv, 1, device="cuda").uniform_(math.log(1e-3), math.log(0.2),
                                                                     generator=g))
    s["log_alpha"] = -rate * torch.nn.functional.softplus(randn(B, Hv, T) + 0.5)
    if case["resets"]:   # a document's first token forgets the one before
        first = torch.rand(B, 1, T, generator=g, device="cuda") < 0.01
        s["log_alpha"] = s["log_alpha"].masked_fill(first, -math.inf)
    s["beta"] = torch.sigmoid(randn(B, Hv, T))
    s["q_scale"], s["k_scale"] = D ** -0.5, 1.0
    s["state"] = 0.3 * randn(B, Hv, D, D) if case["state"] else None
    s["lengths"] = None
    if case["padded"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
        s["lengths"] = n
    if case["op"] == "delta_backward":
        s["do"] = heads(Hv, False)
        s["dstate"] = 0.3 * randn(B, Hv, D, D) if case["state"] else None
    elif case["op"] == "delta_step":
        for n in ("q", "k", "v"):
            s[n] = s[n][:, :, 0]
        s["log_alpha"], s["beta"] = s["log_alpha"][..., 0].contiguous(), s["beta"][..., 0].contiguous()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _share(t, Hv):
    """[B, Hk, ...] in float32 with each head repeated for the value heads that share it."""
    return t.float().repeat_interleave(Hv // t.shape[1], dim=1)


def _valid(lengths, T):
    return torch.arange(T, device=lengths.device)[None, None, :] < lengths[:, None, None]


class _Chunks:
    """What does not depend on the state, for all chunks at once."""

    def __init__(self, s):
        c = s["case"]
        self.T, Hv = c["T"], c["Hv"]
        pad = -self.T % CHUNK
        self.n = (self.T + pad) // CHUNK
        la, beta = s["log_alpha"], s["beta"]
        q, k, v = _share(s["q"], Hv) * s["q_scale"], _share(s["k"], Hv) * s["k_scale"], s["v"].float()
        if s["lengths"] is not None:   # rows behind a sequence leave the state alone
            ok = _valid(s["lengths"], self.T)
            la, beta = la.masked_fill(~ok, 0.0), beta.masked_fill(~ok, 0.0)
            q, k, v = (t.masked_fill(~ok[..., None], 0.0) for t in (q, k, v))
        self.q, self.k, self.v = (self.cut(t) for t in (q, k, v))
        self.beta = self.cut(beta)
        G = self.cut(la).double().clamp_min(NO_DECAY_BELOW).cumsum(-1)
        lower = torch.ones(CHUNK, CHUNK, device=G.device, dtype=torch.bool).tril()
        self.E = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf)).float()
        self.gamma = torch.exp(G).float()
        self.tail = torch.exp(G[..., -1:] - G).float()
        self.N = (self.E * (self.k @ self.k.mT)).tril(-1)
        self.P = self.E * (self.q @ self.k.mT)
        # (I + diag(beta) N)^-1 by forward substitution, a row of every chunk at a time
        A = self.beta[..., None] * self.N
        self.inv = torch.eye(CHUNK, device=A.device).expand_as(A).clone()
        for i in range(1, CHUNK):
            self.inv[..., i, :i] = -(A[..., i:i + 1, :i] @ self.inv[..., :i, :i])[..., 0, :]

    def cut(self, t):
        """[B, H, T, ...] -> [B, H, n, 64, ...], rows of zeros at the end."""
        full = t.new_zeros(t.shape[0], t.shape[1], self.n * CHUNK, *t.shape[3:])
        full[:, :, :self.T] = t
        return full.unflatten(2, (self.n, CHUNK))

    def join(self, rows):
        return torch.stack(rows, dim=2).flatten(2, 3)[:, :, :self.T]

    def forward(self, state):
        """Outputs, final state, and for each chunk its starting state and written values."""
        outs, starts, ys = [], [], []
        for c in range(self.n):
            q, k = self.q[:, :, c], self.k[:, :, c]
            gamma, tail, beta = (t[:, :, c, :, None] for t in (self.gamma, self.tail, self.beta))
            y = self.v[:, :, c] - gamma * (k @ state)
            u = self.inv[:, :, c] @ (beta * y)
            starts.append(state)
            ys.append((y, u))
            outs.append(gamma * (q @ state) + self.P[:, :, c] @ u)
            state = gamma[:, :, -1:] * state + k.mT @ (tail * u)
        return self.join(outs), state, starts, ys


def _start(s):
    c = s["case"]
    if s["state"] is not None:
        return s["state"]
    return torch.zeros(c["B"], c["Hv"], c["D"], c["D"], device="cuda")


def _plain_delta(s):
    o, state, _, _ = _Chunks(s).forward(_start(s))
    return o.to(_dtype(s["case"])), state


def _plain_delta_backward(s):
    case = s["case"]
    x = _Chunks(s)
    _, _, starts, ys = x.forward(_start(s))
    do = s["do"].float()
    if s["lengths"] is not None:
        do = do.masked_fill(~_valid(s["lengths"], x.T)[..., None], 0.0)
    do = x.cut(do)
    ds = s["dstate"] if s["dstate"] is not None else torch.zeros_like(starts[0])
    grads = []
    for c in reversed(range(x.n)):
        q, k, v, S, g = x.q[:, :, c], x.k[:, :, c], x.v[:, :, c], starts[c], do[:, :, c]
        E, N, P, inv = x.E[:, :, c], x.N[:, :, c], x.P[:, :, c], x.inv[:, :, c]
        gamma, tail, beta = (t[:, :, c, :, None] for t in (x.gamma, x.tail, x.beta))
        y, u = ys[c]
        kds = k @ ds
        du = P.mT @ g + tail * kds
        dx = inv.mT @ du
        dP, dA = (g @ u.mT).tril(), -(dx @ u.mT).tril(-1)
        dqs = g @ S.mT
        dN = beta * dA
        dxs = (beta * dx) @ S.mT
        dq = gamma * dqs + (dP * E) @ k
        dk = (-gamma * dxs + tail * (u @ ds.mT) + (dP * E).mT @ q
              + (dN * E) @ k + (dN * E).mT @ k)
        dbeta = (dx * y).sum(-1) + (dA * N).sum(-1)
        W = dP * P + dN * N
        out = tail[..., 0] * (kds * u).sum(-1)
        dG = (W.sum(-1) - W.sum(-2) + gamma[..., 0] * ((q * dqs).sum(-1) - (k * dxs).sum(-1)) - out)
        dG[..., -1] += out.sum(-1) + gamma[:, :, -1, 0] * (ds * S).sum((-1, -2))
        dla = dG.flip(-1).cumsum(-1).flip(-1)
        grads.append((dq, dk, beta * dx, dla, dbeta))
        ds = gamma[:, :, -1:] * ds + q.mT @ (gamma * g) - k.mT @ (gamma * beta * dx)
    dq, dk, dv, dla, dbeta = (x.join(list(t)[::-1]) for t in zip(*grads))
    if s["lengths"] is not None:
        ok = _valid(s["lengths"], x.T)
        dq, dk, dv = (t.masked_fill(~ok[..., None], 0.0) for t in (dq, dk, dv))
        dla, dbeta = dla.masked_fill(~ok, 0.0), dbeta.masked_fill(~ok, 0.0)
    share = (case["Hk"], case["Hv"] // case["Hk"])
    dq = dq.unflatten(1, share).sum(2) * s["q_scale"]
    dk = dk.unflatten(1, share).sum(2) * s["k_scale"]
    dt = _dtype(case)
    return dq.to(dt), dk.to(dt), dv.to(dt), dla, dbeta, ds


def _plain_step(s):
    Hv = s["case"]["Hv"]
    q, k, v = _share(s["q"], Hv) * s["q_scale"], _share(s["k"], Hv) * s["k_scale"], s["v"].float()
    alpha, beta = torch.exp(s["log_alpha"])[..., None], s["beta"][..., None]
    S = s["state"]
    u = beta * (v - alpha * (k[..., None, :] @ S)[..., 0, :])
    new = alpha[..., None] * S + k[..., :, None] * u[..., None, :]
    o = (q[..., None, :] @ new)[..., 0, :]
    if s["lengths"] is not None:
        on = (s["lengths"] > 0)[:, None, None]
        o, new = torch.where(on, o, 0.0), torch.where(on[..., None], new, S)
    S.copy_(new)
    return o.to(_dtype(s["case"])), S


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    h = (x + s["residual"].float()).to(_dtype(c)) if s["residual"] is not None else s["x"]
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
    group = c["group"] or c["N"]
    padded = torch.nn.functional.pad(y, (0, -c["N"] % group)).unflatten(-1, (-1, group))
    scale = padded.abs().amax(-1) / 448.0
    scale = torch.where(scale == 0, 1.0, scale)
    y8 = (padded / scale[..., None]).flatten(-2)[..., :c["N"]]
    return y8.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale, h


def _plain_norm_backward(s):
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)
    t = dy * s["weight"]
    dx = r * t - h * (r * r * r) * (t * h).mean(-1, keepdim=True)
    if s["residual"] is not None:      # here: the gradient that the residual stream brings
        dx = dx + s["residual"].float()
    return dx.to(_dtype(s["case"])), (dy * h * r).sum(0)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import linear_attention_video_frame_b200 as la
        if op == "norm":
            y, scale, h = la.la_add_rms_norm_fp8(s["x"], s["residual"], s["weight"], eps=1e-6,
                                                 group=s["case"]["group"])
            return y, scale, h
        if op == "norm_backward":
            dx, dw = la.la_add_rms_norm_backward(s["dy"], s["x"], s["weight"], dh=s["residual"],
                                                 eps=1e-6)
            return dx, dw
        args = (s["q"], s["k"], s["v"], s["log_alpha"], s["beta"])
        scales = dict(k_scale=s["k_scale"], q_scale=s["q_scale"], lengths=s["lengths"])
        if op == "delta_step":
            o = la.la_gated_delta_step(*args, s["state"], state_out=s["state"], **scales)
            return o, s["state"]
        c = s["case"]
        end = torch.empty(c["B"], c["Hv"], c["D"], c["D"], device="cuda")
        if op == "delta":
            o = la.la_gated_delta_rule(*args, state_in=s["state"], state_out=end, **scales)
            return o, end
        dq, dk, dv, dla, dbeta = la.la_gated_delta_rule_backward(
            *args, s["do"], state_in=s["state"], dstate_out=s["dstate"], dstate_in=end, **scales)
        return dq, dk, dv, dla, dbeta, end
    return {"delta": _plain_delta, "delta_backward": _plain_delta_backward,
            "delta_step": _plain_step, "norm": _plain_norm,
            "norm_backward": _plain_norm_backward}[op](s)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["N"]
        groups = case["rows"] * -(-case["N"] // (case["group"] or case["N"]))
        full = 3 if case["residual"] else 1        # x, residual and their sum; or x alone
        return {"bytes": n * (full * e + 1) + 4 * groups + 4 * case["N"], "flops": 8 * n}
    if case["op"] == "norm_backward":
        n = case["rows"] * case["N"]
        full = 4 if case["residual"] else 3
        return {"bytes": n * full * e + 8 * case["N"], "flops": 10 * n}
    B, Hk, Hv, T, D = (case[n] for n in ("B", "Hk", "Hv", "T", "D"))
    state = 4 * B * Hv * D * D
    tok = B * T
    if case["op"] == "delta_backward":
        rows = tok * D * e * (4 * Hk + 3 * Hv)     # q, k, dq, dk; v, do, dv
        gates = 16 * tok * Hv
        return {"bytes": rows + gates + state * (3 if case["state"] else 1),
                "flops": 18 * tok * Hv * D * D}
    rows = tok * D * e * (2 * Hk + 2 * Hv)
    return {"bytes": rows + 8 * tok * Hv + state * (2 if case["state"] else 1),
            "flops": 6 * tok * Hv * D * D}


# ---------------------------------------------------------------------------
# float64, token by token
# ---------------------------------------------------------------------------
def _tokens64(s):
    """Inputs in float64, token axis first, heads shared out, padding neutral."""
    c = s["case"]
    r = c["Hv"] // c["Hk"]
    one = c["op"] == "delta_step"

    def rows(t, share):
        t = t.double()[:, :, None] if one else t.double()
        if share:
            t = t[:, :, None].expand(-1, -1, r, -1, -1).flatten(1, 2)
        return t.permute(2, 0, 1, 3).contiguous()

    q, k, v = rows(s["q"], True) * s["q_scale"], rows(s["k"], True) * s["k_scale"], rows(s["v"], False)
    alpha, beta = torch.exp(s["log_alpha"].double()), s["beta"].double()
    if one:
        alpha, beta = alpha[..., None], beta[..., None]
    on = torch.ones(q.shape[0], c["B"], device="cuda", dtype=torch.bool)
    if s["lengths"] is not None:
        on = torch.arange(q.shape[0], device="cuda")[:, None] < s["lengths"][None, :]
    live = on[:, :, None]
    alpha = torch.where(live, alpha.permute(2, 0, 1), 1.0)
    beta = torch.where(live, beta.permute(2, 0, 1), 0.0)
    return q, k, v, alpha, beta, on


def _advance(S, k, v, a, b):
    """One token: the decayed state, what the token writes, the new state."""
    old = a[..., None, None] * S
    z = v - torch.einsum("bhk,bhkv->bhv", k, old)
    return old, z, old + torch.einsum("bhk,bhv->bhkv", k, b[..., None] * z)


def _exact_forward(s):
    q, k, v, alpha, beta, on = _tokens64(s)
    S = _start(s).double()
    o = torch.zeros_like(v)
    for t in range(q.shape[0]):
        _, _, S = _advance(S, k[t], v[t], alpha[t], beta[t])
        o[t] = torch.einsum("bhk,bhkv->bhv", q[t], S)
    o = o * on[:, :, None, None]
    return o.permute(1, 2, 0, 3), S


def _exact_backward(s):
    c = s["case"]
    q, k, v, alpha, beta, on = _tokens64(s)
    T = q.shape[0]
    do = s["do"].double().permute(2, 0, 1, 3) * on[:, :, None, None]
    step = 128
    kept, S = [], _start(s).double()
    for t in range(T):
        if t % step == 0:
            kept.append(S)
        S = _advance(S, k[t], v[t], alpha[t], beta[t])[2]
    dS = s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dla, dbeta = torch.zeros_like(alpha), torch.zeros_like(beta)
    for t0 in reversed(range(0, T, step)):
        part = [kept[t0 // step]]
        for t in range(t0, min(T, t0 + step)):
            part.append(_advance(part[-1], k[t], v[t], alpha[t], beta[t])[2])
        for t in reversed(range(t0, min(T, t0 + step))):
            old, z, new = _advance(part[t - t0], k[t], v[t], alpha[t], beta[t])
            b = beta[t][..., None]
            dS = dS + torch.einsum("bhk,bhv->bhkv", q[t], do[t])
            dq[t] = torch.einsum("bhkv,bhv->bhk", new, do[t])
            into_u = torch.einsum("bhkv,bhk->bhv", dS, k[t])
            dz = b * into_u
            dk[t] = torch.einsum("bhkv,bhv->bhk", dS, b * z) - torch.einsum("bhkv,bhv->bhk", old, dz)
            dv[t] = dz
            dbeta[t] = (into_u * z).sum(-1)
            dold = dS - torch.einsum("bhk,bhv->bhkv", k[t], dz)
            dla[t] = (dold * old).sum((-1, -2))
            dS = alpha[t][..., None, None] * dold
    live = on[:, :, None]
    dla, dbeta = dla * live, dbeta * live
    dq, dk = dq * live[..., None], dk * live[..., None]
    share = (c["Hk"], c["Hv"] // c["Hk"])
    dq = dq.permute(1, 2, 0, 3).unflatten(1, share).sum(2) * s["q_scale"]
    dk = dk.permute(1, 2, 0, 3).unflatten(1, share).sum(2) * s["k_scale"]
    return dq, dk, dv.permute(1, 2, 0, 3), dla.permute(1, 2, 0), dbeta.permute(1, 2, 0), dS


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "delta":
        return _exact_forward(s)
    if case["op"] == "delta_step":
        o, S = _exact_forward(s)
        return o[:, :, 0], S
    if case["op"] == "delta_backward":
        return _exact_backward(s)
    w = s["weight"].double()
    if case["op"] == "norm":
        # the stored sum is what is normalised, so its rounding is part of the definition
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(_dtype(case)).double()
        y = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        group = case["group"] or case["N"]
        tops = torch.stack([part.abs().amax(-1) for part in y.split(group, dim=-1)], dim=-1)
        scale = torch.where(tops == 0, 1.0, tops / 448.0)
        column = torch.arange(case["N"], device="cuda") // group
        return y / scale[:, column], scale, h
    h, dy = s["x"].double(), s["dy"].double()
    N = case["N"]
    ms = h.square().sum(-1, keepdim=True) / N + 1e-6
    dx = dy * w / ms.sqrt() - h * (dy * w * h).sum(-1, keepdim=True) / (N * ms ** 1.5)
    if s["residual"] is not None:
        dx = dx + s["residual"].double()
    return dx, (dy * h / ms.sqrt()).sum(0)

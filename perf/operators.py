"""The gated delta rule and layer norm, as measured cases: inputs, plain forms and exact values.

Operators (B batch, H heads, N positions, Dk x Dv state per head):

- ``gd_fwd``   S_t = a_t S_(t-1) + k_t u_t^T with a_t = exp(g_t) and
               u_t = beta_t (v_t - a_t S_(t-1)^T k_t);  o_t = S_t^T q_t   (whole sequences)
- ``gd_bwd``   the gradients (dq, dk, dv, dg, dbeta) of sum_t dout_t . o_t
- ``gd_step``  one position of the same recurrence, the state updated in place (decoding)
- ``ln_fwd``   y = (x - mean) rstd weight + bias over the last dimension, with mean and rstd
- ``ln_bwd``   (dx, dweight, dbias) from the saved mean and rstd

The plain forms are elementary torch operations in fp32 (the sums of log decays in fp64, rounded
once), rounded to the outputs' type at the end.  They treat a sequence in chunks of 64
positions; the loop over the chunks is the recurrence itself.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_C = 64  # chunk length of the plain forms


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest sequence call: a short prompt in fp32, state kept for decoding (latency)
        dict(name="gd_fwd_prompt_f32", op="gd_fwd", B=1, H=2, N=64, Dk=16, Dv=16, dtype="f32", s0=False, state=True,
             packed=False),
        # a training batch of short sequences
        dict(name="gd_fwd_batch_bf16", op="gd_fwd", B=4, H=8, N=1024, Dk=64, Dv=64, dtype="bf16", s0=False,
             state=False, packed=False),
        # a later piece of a long prompt: odd length, few heads, state taken in and handed on,
        # documents packed one after another (the state reset between them)
        dict(name="gd_fwd_piece_bf16", op="gd_fwd", B=1, H=8, N=8191, Dk=128, Dv=128, dtype="bf16", s0=True,
             state=True, packed=True),
        # long-context training
        dict(name="gd_fwd_long_bf16", op="gd_fwd", B=2, H=16, N=65536, Dk=128, Dv=128, dtype="bf16", s0=False,
             state=False, packed=False),
        # gradient of one sequence of odd length, few heads
        dict(name="gd_bwd_odd_bf16", op="gd_bwd", B=1, H=8, N=4095, Dk=64, Dv=64, dtype="bf16", packed=False),
        # gradient of long-context training
        dict(name="gd_bwd_long_bf16", op="gd_bwd", B=2, H=16, N=32768, Dk=128, Dv=128, dtype="bf16", packed=False),
        # one decoding step of many short streams (state in L2: latency)
        dict(name="gd_step_f32", op="gd_step", B=64, H=8, Dk=32, Dv=32, dtype="f32"),
        # one decoding step of a serving batch (state in HBM)
        dict(name="gd_step_wide_bf16", op="gd_step", B=256, H=16, Dk=128, Dv=128, dtype="bf16"),
        # the norm of one decoding step (latency)
        dict(name="ln_fwd_step_f32", op="ln_fwd", rows=64, C=256, dtype="f32", affine=True),
        # the norm over the model width in long-context training
        dict(name="ln_fwd_wide_bf16", op="ln_fwd", rows=131072, C=2048, dtype="bf16", affine=True),
        # gradient of the norm over the model width, a training batch of short sequences
        dict(name="ln_bwd_batch_bf16", op="ln_bwd", rows=4096, C=512, dtype="bf16", affine=True),
        # gradient of the norm of each head's output in long-context training
        dict(name="ln_bwd_heads_bf16", op="ln_bwd", rows=1048576, C=128, dtype="bf16", affine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gd_fwd", "gd_fwd", "gd_bwd", "gd_bwd", "gd_step", "ln_fwd", "ln_bwd"])
    if op in ("ln_fwd", "ln_bwd"):
        C = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            C = max(8, C // 8 * 8)
        rows = _log(rng, 64, max(65, min(1048576, (1 << 27) // C)))
        return dict(op=op, rows=rows, C=C, dtype=rng.choice(["f32", "bf16", "bf16"]), affine=rng.random() < 0.8)
    f32 = rng.random() < 0.3
    if f32 or rng.random() < 0.25:
        Dk, Dv = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    else:
        Dk = Dv = rng.choice([64, 128])
    H = rng.choice([1, 2, 4, 8, 16, 32])
    if op == "gd_step":
        return dict(op=op, B=_log(rng, 1, 256), H=H if H <= 16 else 16, Dk=Dk, Dv=Dv, dtype="f32" if f32 else "bf16")
    B = _log(rng, 1, 8)
    most = min(65536 if op == "gd_fwd" else 32768, (1 << 21 if op == "gd_fwd" else 1 << 20) // (B * H))
    if f32 or Dk != Dv or Dk < 64:
        most = min(most, 16384, (1 << 18) // (B * H))
    N = _log(rng, 64, max(65, most))
    c = dict(op=op, B=B, H=H, N=N, Dk=Dk, Dv=Dv, dtype="f32" if f32 else "bf16", packed=rng.random() < 0.3)
    if op == "gd_fwd":
        c["s0"] = rng.random() < 0.4
        c["state"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------- inputs
def _unit_rows(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def prepare(case, seed):
    dev, dt = torch.device("cuda"), _DT[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    s = dict(case=case)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        R, C = case["rows"], case["C"]
        x = (randn(R, C) * (0.5 + torch.rand(R, 1, generator=gen, device=dev)) + 0.3 * randn(R, 1)).to(dt)
        s["x"] = x
        s["w"] = (1 + 0.1 * randn(C)).to(dt) if case["affine"] else None
        s["b"] = (0.1 * randn(C)).to(dt) if case["affine"] else None
        if case["op"] == "ln_bwd":
            s["dout"] = randn(R, C).to(dt)
            s["mean"], s["rstd"] = _ln_stats(x.float())  # kept from the forward pass
        return s
    B, H, Dk, Dv = case["B"], case["H"], case["Dk"], case["Dv"]
    lead = (B, H) if case["op"] == "gd_step" else (B, H, case["N"])
    # unit keys and queries that share a direction, decays mostly near 1, write strengths in (0, 1)
    shared = 0.5 * randn(1, H, 1, Dk) if len(lead) == 3 else 0.5 * randn(1, H, Dk)
    s["q"] = _unit_rows(randn(*lead, Dk) + shared).to(dt)
    s["k"] = _unit_rows(randn(*lead, Dk) + shared).to(dt)
    s["v"] = randn(*lead, Dv).to(dt)
    s["g"] = (-torch.nn.functional.softplus(randn(*lead) - 3)).to(dt)
    s["beta"] = torch.sigmoid(randn(*lead)).to(dt)
    if case.get("packed"):  # a document begins: nothing of the state before it remains
        s["g"][torch.rand(lead, generator=gen, device=dev) < 0.002] = -math.inf
    if case["op"] == "gd_step":
        s["S"] = 0.5 * randn(B, H, Dk, Dv)
    elif case.get("s0"):
        s["S0"] = 0.5 * randn(B, H, Dk, Dv)
    if case["op"] == "gd_bwd":
        s["dout"] = randn(*lead, Dv).to(dt)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import causal_linear_attention_phi_gb300 as la
        if c["op"] == "gd_fwd":
            return la.gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], S0=s.get("S0"),
                                      return_state=c["state"])
        if c["op"] == "gd_bwd":
            return la.gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"])
        if c["op"] == "gd_step":
            return la.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"]), s["S"]
        if c["op"] == "ln_fwd":
            return la.layer_norm_fwd(s["x"], s["w"], s["b"], return_stats=True)
        return la.layer_norm_bwd(s["x"], s["w"], s["mean"], s["rstd"], s["dout"])
    return _PLAIN[c["op"]](s)


# ---------------------------------------------------------------------------- plain forms: gated delta rule
def _chunks(x, pad):
    """[B, H, N, ...] -> fp32 [B*H, chunks, _C, ...], the last chunk filled with `pad`."""
    B, H, N = x.shape[:3]
    M = -(-N // _C)
    y = torch.full((B * H, M * _C) + tuple(x.shape[3:]), pad, device=x.device, dtype=torch.float32)
    y[:, :N] = x.reshape(B * H, N, *x.shape[3:]).float()
    return y.reshape(B * H, M, _C, *x.shape[3:])


def _merge(x, like):
    return x.reshape(like.shape[0], like.shape[1], -1, *x.shape[3:])[:, :, :like.shape[2]].to(like.dtype).contiguous()


def _decays(g):
    """Inside each chunk: exp(sum of g over (j, i]) for i >= j, from the chunk's start to i, from j to its end.

    A decay of -inf (the state starts anew) is counted apart: sums that cross one give 0."""
    inf = g == -math.inf
    r = torch.cumsum(inf.to(torch.int32), -1)
    G = torch.cumsum(torch.where(inf, 0.0, g.double()), -1)
    low = torch.ones(_C, _C, device=g.device, dtype=torch.bool).tril()
    diff = (G[..., :, None] - G[..., None, :]).masked_fill(~low, 0.0)
    pair = torch.where(low & (r[..., :, None] == r[..., None, :]), diff.exp(), 0.0).float()
    head = torch.where(r == 0, G.exp(), 0.0).float()
    tail = torch.where(r == r[..., -1:], (G[..., -1:] - G).exp(), 0.0).float()
    return pair, head, tail


def _unit_lower_inverse(L):
    """(I + L)^-1 for strictly lower triangular L, row by row."""
    T = torch.eye(_C, device=L.device, dtype=L.dtype).expand(L.shape).clone()
    for i in range(1, _C):
        T[..., i, :i] = -(L[..., i, None, :i] @ T[..., :i, :i]).squeeze(-2)
    return T


def _gd_chunk_parts(s):
    q, k, v = (_chunks(s[n], 0.0) for n in ("q", "k", "v"))
    g, beta = _chunks(s["g"], 0.0), _chunks(s["beta"], 0.0)
    pair, head, tail = _decays(g)
    A = (k @ k.transpose(-1, -2)).mul_(pair).tril_(-1)
    T = _unit_lower_inverse(beta[..., :, None] * A)
    return q, k, v, beta, pair, head, tail, A, T


def _gd_states(k, v, beta, head, tail, A, T, S):
    """The writes X (u = beta X) of every chunk, the states that enter the chunks, and the last state."""
    X, states = torch.empty_like(v), torch.empty(*k.shape[:2], k.shape[-1], v.shape[-1], device=k.device)
    W = (tail * beta)[..., None] * k
    for m in range(k.shape[1]):
        states[:, m] = S
        R = v[:, m] - head[:, m, :, None] * (k[:, m] @ S)
        # X = R - A beta (T R'), the solution of (I + A beta) X = R
        X[:, m] = R - A[:, m] @ (T[:, m] @ (beta[:, m, :, None] * R))
        S = head[:, m, -1, None, None] * S + W[:, m].transpose(-1, -2) @ X[:, m]
    return X, states, S


def _gd_fwd(s):
    q, k, v, beta, pair, head, tail, A, T = _gd_chunk_parts(s)
    B, H = s["q"].shape[:2]
    S = s["S0"].reshape(B * H, *s["S0"].shape[2:]) if s.get("S0") is not None else \
        torch.zeros(B * H, k.shape[-1], v.shape[-1], device=k.device)
    X, states, S = _gd_states(k, v, beta, head, tail, A, T, S)
    P = (q @ k.transpose(-1, -2)).mul_(pair)
    o = _merge(head[..., None] * (q @ states) + P @ (beta[..., None] * X), s["v"])
    return (o, S.reshape(B, H, *S.shape[1:])) if s["case"]["state"] else o


def _gd_bwd(s):
    q, k, v, beta, pair, head, tail, A, T = _gd_chunk_parts(s)
    do = _chunks(s["dout"], 0.0)
    X, states, _ = _gd_states(k, v, beta, head, tail, A, T,
                              torch.zeros(k.shape[0], k.shape[-1], v.shape[-1], device=k.device))
    qk = q @ k.transpose(-1, -2)
    # the adjoint recurrence, last chunk first: d(state) after each chunk, and Y with d(v) = beta Y
    du = (qk * pair).transpose(-1, -2) @ do
    Y, after = torch.empty_like(v), torch.empty_like(states)
    dS = torch.zeros_like(states[:, 0])
    Qh, Kh = (head[..., None] * q).transpose(-1, -2), (head[..., None] * k).transpose(-1, -2)
    for m in range(k.shape[1] - 1, -1, -1):
        after[:, m] = dS
        d = du[:, m] + tail[:, m, :, None] * (k[:, m] @ dS)
        Y[:, m] = T[:, m].transpose(-1, -2) @ d
        dS = head[:, m, -1, None, None] * dS + Qh[:, m] @ do[:, m] - Kh[:, m] @ (beta[:, m, :, None] * Y[:, m])
    U, dR = beta[..., None] * X, beta[..., None] * Y
    dP = (do @ U.transpose(-1, -2)).mul_(pair)
    dA = -(dR @ U.transpose(-1, -2)).mul_(pair).tril_(-1)
    dq_in = head[..., None] * (do @ states.transpose(-1, -2))
    dk_in = -head[..., None] * (dR @ states.transpose(-1, -2))
    dk_out = tail[..., None] * (U @ after.transpose(-1, -2))
    dq = dq_in + dP @ k
    dk = dk_in + dk_out + dA @ k + dA.transpose(-1, -2) @ k + dP.transpose(-1, -2) @ q
    # d/dg: every product that a decay enters, counted at its later end less its earlier one; in
    # fp64, as these sums cancel
    pairs = ((dP * qk).tril_(-1) + dA * (k @ k.transpose(-1, -2))).double()
    into = (q * dq_in).double().sum(-1) + (k * dk_in).double().sum(-1)
    out = (k * dk_out).double().sum(-1)
    dG = pairs.sum(-1) - pairs.sum(-2) + into - out
    kept = (after * states).double().sum((-1, -2)) * head[..., -1] + out.sum(-1)
    dg = torch.flip(torch.cumsum(torch.flip(dG, [-1]), -1), [-1]) + kept[..., None]
    dg = torch.where(_chunks(s["g"], 0.0) == -math.inf, 0.0, dg)
    dbeta = (X * Y).sum(-1)
    return (_merge(dq, s["q"]), _merge(dk, s["k"]), _merge(dR, s["v"]), _merge(dg, s["g"]), _merge(dbeta, s["beta"]))


def _gd_step(s):
    q, k, v, a, beta = s["q"].float(), s["k"].float(), s["v"].float(), s["g"].float().exp(), s["beta"].float()
    S = s["S"].mul_(a[..., None, None])
    u = beta[..., None] * (v - (k[..., None, :] @ S).squeeze(-2))
    S.add_(k[..., :, None] * u[..., None, :])
    return (q[..., None, :] @ S).squeeze(-2).to(s["v"].dtype), S


# ---------------------------------------------------------------------------- plain forms: layer norm
_EPS = 1e-5


def _ln_stats(x):
    mean = x.mean(-1)
    return mean, ((x - mean[..., None]).square().mean(-1) + _EPS).rsqrt()


def _ln_fwd(s):
    x = s["x"].float()
    mean, rstd = _ln_stats(x)
    y = (x - mean[..., None]) * rstd[..., None]
    if s["w"] is not None:
        y = y * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean, rstd


def _ln_bwd(s):
    x, dy = s["x"].float(), s["dout"].float()
    xh = (x - s["mean"][..., None]) * s["rstd"][..., None]
    d = dy * s["w"].float() if s["w"] is not None else dy
    dx = s["rstd"][..., None] * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    dx = dx.to(s["x"].dtype)
    if s["w"] is None:
        return dx, None, None
    return dx, (dy * xh).sum(0).to(s["w"].dtype), dy.sum(0).to(s["b"].dtype)


_PLAIN = {"gd_fwd": _gd_fwd, "gd_bwd": _gd_bwd, "gd_step": _gd_step, "ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("ln_fwd", "ln_bwd"):
        n, aff = case["rows"] * case["C"], 2 * case["C"] * e if case["affine"] else 0
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * n * e + aff + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + aff * 3 // 2 + 8 * case["rows"], "flops": 14 * n}
    BH, Dk, Dv = case["B"] * case["H"], case["Dk"], case["Dv"]
    if case["op"] == "gd_step":
        return {"bytes": BH * (8 * Dk * Dv + e * (2 * Dk + 2 * Dv + 2)), "flops": 7 * BH * Dk * Dv}
    T = BH * case["N"]
    if case["op"] == "gd_fwd":
        states = (1 if case["s0"] else 0) + (1 if case["state"] else 0)
        return {"bytes": T * e * (2 * Dk + 2 * Dv + 2) + 4 * BH * Dk * Dv * states, "flops": 7 * T * Dk * Dv}
    return {"bytes": T * e * (4 * Dk + 3 * Dv + 4), "flops": 22 * T * Dk * Dv}


# ---------------------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        return _exact_ln(case, s)
    x = {n: t.double().flatten(0, 1) for n, t in s.items() if isinstance(t, torch.Tensor)}
    shape = s["q"].shape[:2]
    if case["op"] == "gd_bwd":
        return None if case["N"] > 40000 else _exact_gd_bwd(x, shape)
    if case["op"] == "gd_step":
        x = {n: t if n == "S" else t[:, None] for n, t in x.items()}
    S = x.get("S", x.get("S0"))
    S = x["q"].new_zeros(len(x["q"]), case["Dk"], case["Dv"]) if S is None else S
    o = torch.empty_like(x["v"])
    a = x["g"].exp()
    for t in range(o.shape[1]):
        S = a[:, t, None, None] * S
        k = x["k"][:, t, None]
        u = x["beta"][:, t, None, None] * (x["v"][:, t, None] - k @ S)
        S = torch.baddbmm(S, k.mT, u)
        o[:, t] = (x["q"][:, t, None] @ S).squeeze(1)
    S = S.unflatten(0, shape)
    if case["op"] == "gd_step":
        return o[:, 0].unflatten(0, shape), S
    return (o.unflatten(0, shape), S) if case["state"] else o.unflatten(0, shape)


def _exact_gd_bwd(x, shape):
    """The recurrence run back position by position; states kept at every 128th position and formed again."""
    q, k, v, beta, do, a = x["q"], x["k"], x["v"], x["beta"], x["dout"], x["g"].exp()
    n = q.shape[1]

    def write(Sd, t):
        return v[:, t, None] - k[:, t, None] @ Sd

    def step(S, t):
        Sd = a[:, t, None, None] * S
        return torch.baddbmm(Sd, k[:, t, :, None], beta[:, t, None, None] * write(Sd, t))

    starts, S = [], q.new_zeros(len(q), q.shape[-1], v.shape[-1])
    for t in range(n):
        if t % 128 == 0:
            starts.append(S)
        S = step(S, t)
    dq, dk, dv, dg, db = (torch.empty_like(t) for t in (q, k, v, a, beta))
    dS = torch.zeros_like(S)
    for m in range(len(starts) - 1, -1, -1):
        before, S = [], starts[m]
        for t in range(128 * m, min(n, 128 * m + 128)):
            before.append(S)
            S = step(S, t)
        for t in range(min(n, 128 * m + 128) - 1, 128 * m - 1, -1):
            kt, dot = k[:, t, :, None], do[:, t, None]
            dq[:, t] = (S @ dot.mT).squeeze(-1)
            dS = torch.baddbmm(dS, q[:, t, :, None], dot)
            Sd = a[:, t, None, None] * before[t - 128 * m]
            e, du, bt = write(Sd, t), kt.mT @ dS, beta[:, t, None, None]
            de = bt * du
            db[:, t] = (du * e).sum((-1, -2))
            dv[:, t] = de.squeeze(1)
            dk[:, t] = (dS @ (bt * e).mT - Sd @ de.mT).squeeze(-1)
            dS = torch.baddbmm(dS, kt, de, alpha=-1)
            dg[:, t] = (dS * Sd).sum((-1, -2))
            dS = a[:, t, None, None] * dS
            S = before[t - 128 * m]
    return tuple(t.unflatten(0, shape) for t in (dq, dk, dv, dg, db))


def _exact_ln(case, s):
    x = s["x"].double()
    w = s["w"].double() if case["affine"] else torch.ones(case["C"], device=x.device, dtype=torch.float64)
    if case["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, -1, correction=0)
        y = (x - mean[:, None]) / (var[:, None] + _EPS).sqrt() * w
        return (y + s["b"].double() if case["affine"] else y), mean, 1 / (var + _EPS).sqrt()
    # with the statistics that were handed in
    h = torch.sub(x, s["mean"].double()[:, None]).mul_(s["rstd"].double()[:, None])
    dy = s["dout"].double()
    dh = dy * w
    inner = torch.einsum("rc,rc->r", dh, h) / case["C"]
    dx = (dh - dh.sum(-1, keepdim=True) / case["C"] - inner[:, None] * h) * s["rstd"].double()[:, None]
    if not case["affine"]:
        return dx, None, None
    return dx, torch.einsum("rc,rc->c", dy, h), torch.einsum("rc->c", dy)

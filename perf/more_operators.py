"""Cross attention with a linear kernel and the norms around a block, as measured cases: inputs, plain forms and exact values.

Operators (B batch, H heads of queries, Hk heads of keys, N queries, M keys, phi(x) = elu(x) + 1):

- ``cross_fwd``    o_i = phi(q_i)^T S / phi(q_i)^T z with S = sum_j phi(k_j) v_j^T, z = sum_j phi(k_j) over the keys
                   j < length of the batch entry; H / Hk heads of queries share a head of keys
- ``cross_bwd``    the gradients (dq, dk, dv) of sum_i dout_i . o_i, with or without the state (S, z) kept from the forward
- ``cross_apply``  o from a kept state: single tokens (N = 1) or a few, a head's state read once
- ``gated_fwd``    y[b, n, h] = norm(o[b, h, n]) weight silu(gate[b, n, h]): the norm of each head's output with its gate,
                   heads merged
- ``gated_bwd``    (do, dgate, dweight)
- ``resid_fwd``    h = x + scale a, y = norm(h) weight + bias, with the statistics
- ``resid_bwd``    (dx, da, dscale, dweight, dbias) from dy and dh

norm is layer norm or, with ``rms``, division by the root of the mean square.  The plain forms are elementary torch
operations in fp32, rounded to the outputs' type at the end.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 1e-5


# ---------------------------------------------------------------------------- cases
def _cross(name, op, B, H, Hk, N, M, Dk, Dv, dtype, ragged, state):
    c = dict(op=op, B=B, H=H, Hk=Hk, N=N, M=M, Dk=Dk, Dv=Dv, dtype=dtype, ragged=ragged, state=state)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # the smallest call: a short prompt in fp32 attends to a short memory, the state kept for decoding (latency)
        _cross("cross_fwd_prompt_f32", "cross_fwd", 1, 2, 2, 17, 64, 16, 16, "f32", False, True),
        # a training batch of short sequences, memories padded to the longest
        _cross("cross_fwd_batch_bf16", "cross_fwd", 4, 8, 8, 1024, 777, 64, 64, "bf16", True, False),
        # long sequences attending to long memories, four heads of queries to a head of keys
        _cross("cross_fwd_long_bf16", "cross_fwd", 2, 16, 4, 65536, 131071, 128, 128, "bf16", False, True),
        # gradient of the training batch, nothing kept from the forward
        _cross("cross_bwd_batch_bf16", "cross_bwd", 4, 8, 4, 1023, 1500, 64, 64, "bf16", True, False),
        # gradient of long sequences, the state kept from the forward
        _cross("cross_bwd_long_bf16", "cross_bwd", 2, 16, 16, 32768, 32768, 128, 128, "bf16", False, True),
        # one token of many short streams (state in L2: latency)
        _cross("cross_apply_f32", "cross_apply", 64, 8, 8, 1, 0, 32, 32, "f32", False, True),
        # one token of a serving batch (state in HBM), two heads of queries to a state
        _cross("cross_apply_wide_bf16", "cross_apply", 256, 32, 16, 1, 0, 128, 128, "bf16", False, True),
        # the gated norm of every head in long-context training
        dict(name="gated_fwd_long_bf16", op="gated_fwd", B=2, H=16, N=65536, D=128, dtype="bf16", rms=True),
        # its gradient, a training batch of short sequences
        dict(name="gated_bwd_batch_bf16", op="gated_bwd", B=8, H=8, N=4095, D=64, dtype="bf16", rms=True),
        # the residual sum and norm of one decoding step (latency)
        dict(name="resid_fwd_step_f32", op="resid_fwd", rows=64, C=256, dtype="f32", rms=False, scale=True),
        # the same over the model width in long-context training
        dict(name="resid_fwd_wide_bf16", op="resid_fwd", rows=131072, C=2048, dtype="bf16", rms=True, scale=False),
        # its gradient with a scale to each channel
        dict(name="resid_bwd_wide_bf16", op="resid_bwd", rows=65536, C=2048, dtype="bf16", rms=False, scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross_fwd", "cross_fwd", "cross_bwd", "cross_bwd", "cross_apply", "gated_fwd", "gated_bwd",
                     "resid_fwd", "resid_bwd"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op.startswith("resid"):
        C = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            C = max(8, C // 8 * 8)
        rows = _log(rng, 64, max(65, min(262144, (1 << 26) // C)))
        return dict(op=op, rows=rows, C=C, dtype=dtype, rms=rng.random() < 0.5, scale=rng.random() < 0.5)
    H = rng.choice([1, 2, 4, 8, 16, 32])
    if op.startswith("gated"):
        D, B = rng.choice([16, 32, 64, 128]), _log(rng, 1, 8)
        return dict(op=op, B=B, H=H, N=_log(rng, 1, max(2, (1 << 26) // (B * H * D))), D=D, dtype=dtype,
                    rms=rng.random() < 0.5)
    Hk = max(1, H // rng.choice([1, 1, 2, 4]))
    Dk, Dv = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    if dtype == "bf16" and rng.random() < 0.6:
        Dk = Dv = rng.choice([64, 128])
    if op == "cross_apply":
        return _cross(None, op, _log(rng, 1, 256), min(H, 16), min(Hk, 16), rng.choice([1, 1, 1, 2, 5, 40]), 0, Dk, Dv,
                      dtype, False, True)
    B = _log(rng, 1, 8)
    most = (1 << 19 if dtype == "bf16" else 1 << 17) // (B * H)
    return _cross(None, op, B, H, Hk, _log(rng, 1, min(65536, most)), _log(rng, 1, min(131072, most)), Dk, Dv, dtype,
                  rng.random() < 0.5, rng.random() < 0.5)


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev, dt = torch.device("cuda"), _DT[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    s, op = dict(case=case), case["op"]
    if op.startswith("resid"):
        R, C = case["rows"], case["C"]
        x, a = randn(R, C) + 0.3 * randn(R, 1), randn(R, C)
        s["scale"] = (0.5 + 0.2 * randn(C)).to(dt) if case["scale"] else None
        s["w"] = (1 + 0.1 * randn(C)).to(dt)
        s["b"] = None if case["rms"] else (0.1 * randn(C)).to(dt)
        s["a"] = a.to(dt)
        if op == "resid_fwd":
            s["x"] = x.to(dt)
        else:
            s["h"] = (x + a).to(dt)
            s["mean"], s["rstd"] = _stats(s["h"].float(), case["rms"])  # kept from the forward pass
            s["dy"], s["dh"] = randn(R, C).to(dt), randn(R, C).to(dt)
        return s
    if op.startswith("gated"):
        B, H, N, D = (case[n] for n in "BHND")
        s["o"] = (randn(B, H, N, D) * (0.2 + torch.rand(B, H, N, 1, generator=gen, device=dev))).to(dt)
        s["gate"] = randn(B, N, H * D).to(dt)
        s["w"] = (1 + 0.1 * randn(D)).to(dt)
        if op == "gated_bwd":
            s["dout"] = randn(B, N, H * D).to(dt)
        return s
    B, H, Hk, N, M, Dk, Dv = (case[n] for n in ("B", "H", "Hk", "N", "M", "Dk", "Dv"))
    # channels with an offset to each head, as projections of normed activations have them
    s["q"] = (0.6 * randn(B, H, N, Dk) + 0.4 * randn(1, H, 1, Dk)).to(dt)
    if op == "cross_apply":
        s["S"] = 30 * randn(B, Hk, Dk, Dv)
        s["z"] = 1000 * (0.5 + torch.rand(B, Hk, Dk, generator=gen, device=dev))
        return s
    s["k"] = (0.6 * randn(B, Hk, M, Dk) + 0.4 * randn(1, Hk, 1, Dk)).to(dt)
    s["v"] = (randn(B, Hk, M, Dv) + 0.3 * randn(1, Hk, 1, Dv)).to(dt)
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, M + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        n[0] = M  # padded to the longest
        s["lengths"] = n
    if op == "cross_bwd":
        s["dout"] = randn(B, H, N, Dv).to(dt)
        s["S"], s["z"] = _sums(s["k"], s["v"], s["lengths"]) if case["state"] else (None, None)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import causal_linear_attention_phi_gb300 as la
        if c["op"] == "cross_fwd":
            return la.cross_fwd(s["q"], s["k"], s["v"], lengths=s["lengths"], return_state=c["state"])
        if c["op"] == "cross_bwd":
            return la.cross_bwd(s["q"], s["k"], s["v"], s["dout"], lengths=s["lengths"], S=s["S"], z=s["z"])
        if c["op"] == "cross_apply":
            return la.cross_apply(s["q"], s["S"], s["z"])
        if c["op"] == "gated_fwd":
            return la.gated_norm_fwd(s["o"], s["gate"], s["w"], rms=c["rms"], eps=_EPS)
        if c["op"] == "gated_bwd":
            return la.gated_norm_bwd(s["o"], s["gate"], s["w"], s["dout"], rms=c["rms"], eps=_EPS)
        if c["op"] == "resid_fwd":
            return la.residual_norm_fwd(s["x"], s["a"], s["scale"], s["w"], s["b"], rms=c["rms"], eps=_EPS,
                                        return_stats=True)
        return la.residual_norm_bwd(s["h"], s["a"], s["scale"], s["w"], s["mean"], s["rstd"], s["dy"], s["dh"],
                                    rms=c["rms"])
    return _PLAIN[c["op"]](s)


# ---------------------------------------------------------------------------- plain forms: cross attention
def _phi(x):
    return torch.where(x > 0, x + 1, torch.exp(torch.clamp(x, max=0.0)))


def _keys(k, v, lengths):
    """phi(k) and v in fp32, 0 behind the length."""
    p, v = _phi(k.float()), v.float()
    if lengths is not None:
        out = (torch.arange(k.shape[2], device=k.device) >= lengths[:, None])[:, None, :, None]
        p, v = p.masked_fill(out, 0.0), v.masked_fill(out, 0.0)
    return p, v


def _sums(k, v, lengths):
    p, v = _keys(k, v, lengths)
    return p.transpose(-1, -2) @ v, p.sum(2)


def _grouped(x, Hk):
    """[B, H, N, D] -> [B, Hk, G N, D]: the queries that share a head of keys, one after another."""
    return x.reshape(x.shape[0], Hk, -1, x.shape[-1])


def _over(den):
    return torch.where(den == 0, 0.0, 1 / den)


def _plain_apply(q, S, z):
    p = _phi(_grouped(q.float(), S.shape[1]))
    return ((p @ S) * _over((p * z[:, :, None]).sum(-1, keepdim=True))).reshape(*q.shape[:3], S.shape[-1]).to(q.dtype)


def _cross_fwd(s):
    S, z = _sums(s["k"], s["v"], s["lengths"])
    o = _plain_apply(s["q"], S, z)
    return (o, S, z) if s["case"]["state"] else o


def _cross_bwd(s):
    q, Hk = s["q"], s["k"].shape[1]
    pk, v = _keys(s["k"], s["v"], s["lengths"])
    S, z = (s["S"], s["z"]) if s["S"] is not None else (pk.transpose(-1, -2) @ v, pk.sum(2))
    pq, do = _phi(_grouped(q.float(), Hk)), _grouped(s["dout"].float(), Hk)
    inv = _over((pq * z[:, :, None]).sum(-1, keepdim=True))
    Y = (do @ S.transpose(-1, -2)).mul_(inv)
    t = (pq * Y).sum(-1, keepdim=True)
    dq = torch.addcmul(Y, -t * inv, z[:, :, None]).mul_(pq.clamp(max=1.0))
    pq.mul_(inv)
    R = pq.transpose(-1, -2) @ do
    r = -(pq * t).sum(2)
    dk = (v @ R.transpose(-1, -2)).add_(r[:, :, None]).mul_(pk.clamp(max=1.0))
    return dq.reshape(q.shape).to(q.dtype), dk.to(q.dtype), (pk @ R).to(q.dtype)


def _cross_apply(s):
    return _plain_apply(s["q"], s["S"], s["z"])


# ---------------------------------------------------------------------------- plain forms: norms
def _stats(x, rms):
    if rms:
        return None, (x.square().mean(-1) + _EPS).rsqrt()
    mean = x.mean(-1)
    return mean, ((x - mean[..., None]).square().mean(-1) + _EPS).rsqrt()


def _normed(x, mean, rstd):
    return (x if mean is None else x - mean[..., None]) * rstd[..., None]


def _norm_grad(d, n, rstd, rms):
    """The gradient of n = norm(x) for d."""
    d = d - n * (d * n).mean(-1, keepdim=True) - (0.0 if rms else d.mean(-1, keepdim=True))
    return d * rstd[..., None]


def _by_head(x, D):
    """[B, N, H D] -> fp32 [B, H, N, D]"""
    return x.float().reshape(*x.shape[:2], -1, D).transpose(1, 2)


def _merged(x, like):
    return x.transpose(1, 2).reshape(like.shape).to(like.dtype)


def _gated_fwd(s):
    o, g = s["o"].float(), _by_head(s["gate"], s["case"]["D"])
    y = _normed(o, *_stats(o, s["case"]["rms"])) * s["w"].float() * (g * torch.sigmoid(g))
    return _merged(y, s["gate"])


def _gated_bwd(s):
    rms, D, w = s["case"]["rms"], s["case"]["D"], s["w"].float()
    o, g, dy = s["o"].float(), _by_head(s["gate"], D), _by_head(s["dout"], D)
    mean, rstd = _stats(o, rms)
    n, sg = _normed(o, mean, rstd), torch.sigmoid(g)
    dgate = dy * n * w * sg * (1 + g * (1 - sg))
    d = dy * g * sg
    return (_norm_grad(d * w, n, rstd, rms).to(s["o"].dtype), _merged(dgate, s["gate"]),
            (d * n).sum((0, 1, 2)).to(s["w"].dtype))


def _resid_fwd(s):
    a = s["a"].float()
    h = s["x"].float() + (a if s["scale"] is None else s["scale"].float() * a)
    mean, rstd = _stats(h, s["case"]["rms"])
    y = _normed(h, mean, rstd) * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return h.to(s["x"].dtype), y.to(s["x"].dtype), mean, rstd


def _resid_bwd(s):
    dt, dy, w = s["h"].dtype, s["dy"].float(), s["w"].float()
    n = _normed(s["h"].float(), s["mean"], s["rstd"])
    dx = s["dh"].float() + _norm_grad(dy * w, n, s["rstd"], s["case"]["rms"])
    dw, db = (dy * n).sum(0).to(dt), dy.sum(0).to(dt)
    if s["scale"] is None:
        return dx.to(dt), dx.to(dt), None, dw, db
    return dx.to(dt), (s["scale"].float() * dx).to(dt), (s["a"].float() * dx).sum(0).to(dt), dw, db


_PLAIN = {"cross_fwd": _cross_fwd, "cross_bwd": _cross_bwd, "cross_apply": _cross_apply, "gated_fwd": _gated_fwd,
          "gated_bwd": _gated_bwd, "resid_fwd": _resid_fwd, "resid_bwd": _resid_bwd}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op.startswith("resid"):
        n, C = case["rows"] * case["C"], case["C"]
        stats = case["rows"] * (4 if case["rms"] else 8)
        if op == "resid_fwd":
            return {"bytes": 4 * n * e + stats + 3 * C * e, "flops": 9 * n}
        return {"bytes": (6 if case["scale"] else 4) * n * e + stats + 5 * C * e, "flops": 17 * n}
    if op.startswith("gated"):
        n = case["B"] * case["H"] * case["N"] * case["D"]
        return {"bytes": (3 if op == "gated_fwd" else 5) * n * e + 2 * case["D"] * e, "flops": (14 if op == "gated_fwd" else 32) * n}
    Dk, Dv = case["Dk"], case["Dv"]
    rows, keys = case["B"] * case["H"] * case["N"], case["B"] * case["Hk"] * case["M"]
    if case["ragged"]:
        keys = keys * (1 + case["B"]) // (2 * case["B"])  # the first length is whole, the others half on the average
    state = 4 * case["B"] * case["Hk"] * (Dk * Dv + Dk)
    if op == "cross_apply":
        return {"bytes": state + rows * (Dk + Dv) * e, "flops": 2 * rows * Dk * Dv}
    if op == "cross_fwd":
        return {"bytes": (rows + keys) * (Dk + Dv) * e + (state if case["state"] else 0), "flops": 2 * Dk * Dv * (rows + keys)}
    return {"bytes": (rows * (2 * Dk + Dv) + keys * 2 * (Dk + Dv)) * e + (state if case["state"] else 0),
            "flops": 2 * Dk * Dv * (2 * rows + (2 if case["state"] else 3) * keys)}


# ---------------------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    x = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    if case["op"].startswith("resid"):
        return _exact_resid(case, x)
    if case["op"].startswith("gated"):
        return _exact_gated(case, x)
    return _exact_cross(case, x)


def _exact_cross(case, x):
    """Head by head; the gradient by the weights' own chain rule, d(num) and d(den) apart."""
    B, Hk, G = case["B"], case["Hk"], case["H"] // case["Hk"]
    elu1 = lambda t: torch.nn.functional.elu(t) + 1
    out = {n: torch.zeros_like(x[n]) for n in (("q", "k", "v") if case["op"] == "cross_bwd" else ())}
    o = x["q"].new_zeros(B, case["H"], case["N"], case["Dv"])
    states, norms = [], []
    for b in range(B):
        m = int(x["lengths"][b]) if "lengths" in x else case["M"]
        for j in range(Hk):
            heads = slice(G * j, G * j + G)
            fq = elu1(x["q"][b, heads]).flatten(0, 1)
            if case["op"] == "cross_apply":
                S, z = x["S"][b, j], x["z"][b, j]
            else:
                fk, v = elu1(x["k"][b, j, :m]), x["v"][b, j, :m]
                S, z = torch.einsum("md,mv->dv", fk, v), torch.einsum("md->d", fk)
                states.append(S)
                norms.append(z)
            den = torch.mv(fq, z)[:, None]
            den = den.masked_fill(den == 0, math.inf)
            res = (fq @ S) / den
            if case["op"] != "cross_bwd":
                o[b, heads] = res.unflatten(0, (G, -1))
                continue
            dnum = x["dout"][b, heads].flatten(0, 1) / den
            dden = -(dnum * res).sum(-1)
            slope = torch.exp(x["q"][b, heads].flatten(0, 1).clamp(max=0))
            out["q"][b, heads] = ((dnum @ S.T + torch.outer(dden, z)) * slope).unflatten(0, (G, -1))
            dS, dz = torch.einsum("nd,nv->dv", fq, dnum), torch.mv(fq.T, dden)
            out["k"][b, j, :m] = (v @ dS.T + dz) * torch.exp(x["k"][b, j, :m].clamp(max=0))
            out["v"][b, j, :m] = fk @ dS
    if case["op"] == "cross_bwd":
        return out["q"], out["k"], out["v"]
    if case["op"] == "cross_fwd" and case["state"]:
        return o, torch.stack(states).unflatten(0, (B, Hk)), torch.stack(norms).unflatten(0, (B, Hk))
    return o


def _exact_gated(case, x):
    """A batch entry at a time, positions before heads throughout."""
    ys, dos, dgs, dw = [], [], [], 0.0
    for b in range(case["B"]):
        o = x["o"][b].permute(1, 0, 2)
        g = x["gate"][b].view(o.shape)
        centre = 0.0 if case["rms"] else torch.mean(o, 2, keepdim=True)
        dev = torch.sqrt(torch.mean(torch.pow(o - centre, 2), 2, keepdim=True) + _EPS)
        n, silu = (o - centre) / dev, g / (1 + torch.exp(-g))
        if case["op"] == "gated_fwd":
            ys.append((n * x["w"] * silu).flatten(1))
            continue
        dy = x["dout"][b].view(o.shape)
        dw = dw + torch.einsum("nhd,nhd->d", dy * silu, n)
        e = torch.exp(-g)
        dgs.append((dy * n * x["w"] * (1 + e + g * e) / torch.pow(1 + e, 2)).flatten(1))
        dn = dy * silu * x["w"]
        do = dn - n * (torch.einsum("nhd,nhd->nh", dn, n) / case["D"])[..., None]
        if not case["rms"]:
            do = do - torch.mean(dn, 2, keepdim=True)
        dos.append((do / dev).permute(1, 0, 2))
    return torch.stack(ys) if ys else (torch.stack(dos), torch.stack(dgs), dw)


def _exact_resid(case, x):
    C, scale = case["C"], x.get("scale", 1.0)
    if case["op"] == "resid_fwd":
        h = torch.add(x["x"], x["a"] * scale)
        if case["rms"]:
            mean, dev = None, torch.sqrt(torch.einsum("rc,rc->r", h, h) / C + _EPS)
            y = h / dev[:, None] * x["w"]
        else:
            var, mean = torch.var_mean(h, -1, correction=0)
            dev = torch.sqrt(var + _EPS)
            y = (h - mean[:, None]) / dev[:, None] * x["w"] + x["b"]
        return h, y, mean, 1 / dev
    # with the statistics that were handed in
    n = x["h"] if case["rms"] else x["h"] - x["mean"][:, None]
    n = n * x["rstd"][:, None]
    dn = x["dy"] * x["w"]
    dx = dn - n * (torch.einsum("rc,rc->r", dn, n) / C)[:, None]
    if not case["rms"]:
        dx -= (torch.einsum("rc->r", dn) / C)[:, None]
    dx = torch.addcmul(x["dh"], dx, x["rstd"][:, None])
    dscale = torch.einsum("rc,rc->c", x["a"], dx) if case["scale"] else None
    return dx, dx * scale, dscale, torch.einsum("rc,rc->c", x["dy"], n), torch.einsum("rc->c", x["dy"])

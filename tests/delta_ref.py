"""The gated delta rule and layer norm in fp64 numpy, from the definitions (no chunks).

One head at a time, position by position.  Inputs are torch tensors or arrays; bf16 values are
taken exactly.
"""
import numpy as np

from util import to_np


def _heads(*ts):
    return [to_np(t).reshape((-1,) + tuple(t.shape[2:])) for t in ts]


def delta_fwd(q, k, v, g, beta, S0=None):
    """(o, S): outputs [B,H,N,Dv] and the state after the last position [B,H,Dk,Dv]."""
    B, H, N, Dk = q.shape
    Dv = v.shape[-1]
    q, k, v, g, beta = _heads(q, k, v, g, beta)
    S = np.zeros((B * H, Dk, Dv)) if S0 is None else _heads(S0)[0].copy()
    a = np.where(g < -100, 0, np.exp(g))  # the rule's reset
    o = np.zeros((B * H, N, Dv))
    for t in range(N):
        S = a[:, t, None, None] * S
        u = beta[:, t, None] * (v[:, t] - np.einsum("hd,hde->he", k[:, t], S))
        S = S + k[:, t, :, None] * u[:, None]
        o[:, t] = np.einsum("hd,hde->he", q[:, t], S)
    return o.reshape(B, H, N, Dv), S.reshape(B, H, Dk, Dv)


def delta_bwd(q, k, v, g, beta, dout):
    """(dq, dk, dv, dg, dbeta) of sum(dout * o): the chain rule on each position's update, last first."""
    shapes = [t.shape for t in (q, k, v, g, beta)]
    q, k, v, g, beta, do = _heads(q, k, v, g, beta, dout)
    nh, N, Dk = q.shape
    a = np.where(g < -100, 0, np.exp(g))  # the rule's reset
    S = np.zeros((N + 1, nh, Dk, v.shape[-1]))
    e = np.zeros_like(v)  # v minus what the decayed state holds of the key
    for t in range(N):
        Sd = a[:, t, None, None] * S[t]
        e[:, t] = v[:, t] - np.einsum("hd,hde->he", k[:, t], Sd)
        S[t + 1] = Sd + k[:, t, :, None] * (beta[:, t, None] * e[:, t])[:, None]
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    dS = np.zeros_like(S[0])
    for t in range(N - 1, -1, -1):
        Sd = a[:, t, None, None] * S[t]
        dq[:, t] = np.einsum("hde,he->hd", S[t + 1], do[:, t])
        dS = dS + q[:, t, :, None] * do[:, t, None]
        du = np.einsum("hd,hde->he", k[:, t], dS)
        db[:, t] = np.sum(du * e[:, t], -1)
        de = beta[:, t, None] * du
        dv[:, t] = de
        dk[:, t] = np.einsum("hde,he->hd", dS, beta[:, t, None] * e[:, t]) - np.einsum("hde,he->hd", Sd, de)
        dS = dS - k[:, t, :, None] * de[:, None]
        dg[:, t] = np.sum(dS * Sd, (-1, -2))
        dS = a[:, t, None, None] * dS
    return tuple(x.reshape(s) for x, s in zip((dq, dk, dv, dg, db), shapes))


def norm_fwd(x, w=None, b=None, eps=1e-5):
    x = to_np(x)
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd
    y = y if w is None else y * to_np(w)
    return y if b is None else y + to_np(b), mean[..., 0], rstd[..., 0]


def norm_bwd(x, w, dy, eps=1e-5):
    _, mean, rstd = norm_fwd(x, eps=eps)
    x, dy = to_np(x), to_np(dy)
    h = (x - mean[..., None]) * rstd[..., None]
    d = dy if w is None else dy * to_np(w)
    dx = rstd[..., None] * (d - d.mean(-1, keepdims=True) - h * (d * h).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * h).sum(axes), dy.sum(axes)

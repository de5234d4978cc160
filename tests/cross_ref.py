"""Cross attention with phi = elu + 1 in fp64 on the CPU, and the magnitudes that rounding errors scale with.

Weights are formed as a matrix (queries by keys), so nothing here shares the kernels' algebra: o = W v with
W_ij = phi(q_i) . phi(k_j) / sum_j, and the gradient goes back through W.
"""
import numpy as np
import torch


def _np(t):
    return t.detach().cpu().double().numpy()


def phi(x):
    return np.where(x > 0, x + 1, np.exp(np.minimum(x, 0)))


def dphi(x):
    return np.where(x > 0, 1.0, np.exp(np.minimum(x, 0)))


def fwd(q, k, v, lengths=None):
    """o [B,H,N,Dv], S [B,Hk,Dk,Dv], z [B,Hk,Dk], and the magnitude of o (the same with |v|)."""
    q, k, v = _np(q), _np(k), _np(v)
    B, H, N, Dk = q.shape
    Hk, M, Dv = v.shape[1:]
    o, mag = np.zeros((B, H, N, Dv)), np.zeros((B, H, N, Dv))
    S, z = np.zeros((B, Hk, Dk, Dv)), np.zeros((B, Hk, Dk))
    for b in range(B):
        m = M if lengths is None else min(max(int(lengths[b]), 0), M)
        for j in range(Hk):
            fk, vj = phi(k[b, j, :m]), v[b, j, :m]
            S[b, j], z[b, j] = fk.T @ vj, fk.sum(0)
        for h in range(H):
            j = h // (H // Hk)
            w = phi(q[b, h]) @ phi(k[b, j, :m]).T
            den = w.sum(1, keepdims=True)
            w = np.divide(w, den, out=np.zeros_like(w), where=den != 0)
            o[b, h], mag[b, h] = w @ v[b, j, :m], w @ np.abs(v[b, j, :m])
    return o, S, z, mag


def bwd(q, k, v, dout, lengths=None):
    """(dq, dk, dv) and their magnitudes: every term of the sums by its absolute value."""
    q, k, v, do = _np(q), _np(k), _np(v), _np(dout)
    B, H, N, Dk = q.shape
    Hk, M, Dv = v.shape[1:]
    dq, dk, dv = np.zeros_like(q), np.zeros(k.shape), np.zeros(v.shape)
    mq, mk, mv = np.zeros_like(q), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        m = M if lengths is None else min(max(int(lengths[b]), 0), M)
        for h in range(H):
            j = h // (H // Hk)
            fq, fk, vj = phi(q[b, h]), phi(k[b, j, :m]), v[b, j, :m]
            s = fq @ fk.T
            den = s.sum(1, keepdims=True)
            w = np.divide(s, den, out=np.zeros_like(s), where=den != 0)
            inv = np.divide(1.0, den, out=np.zeros_like(den), where=den != 0)
            o = w @ vj
            dw = (do[b, h] @ vj.T - (do[b, h] * o).sum(1, keepdims=True)) * inv  # d(s)
            dq[b, h] = (dw @ fk) * dphi(q[b, h])
            dk[b, j, :m] += (dw.T @ fq) * dphi(k[b, j, :m])
            dv[b, j, :m] += w.T @ do[b, h]
            aw = (np.abs(do[b, h]) @ np.abs(vj).T + (np.abs(do[b, h]) * (w @ np.abs(vj))).sum(1, keepdims=True)) * inv
            mq[b, h] = (aw @ fk) * dphi(q[b, h])
            mk[b, j, :m] += (aw.T @ fq) * dphi(k[b, j, :m])
            mv[b, j, :m] += w.T @ np.abs(do[b, h])
    return (dq, dk, dv), (mq, mk, mv)


def make(B, H, Hk, N, M, Dk, Dv, dtype, seed=0, offset=0.4, lengths=None, behind=None):
    """q, k, v, dout on the CPU; rows behind the lengths filled with `behind` if given."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    q, k = 0.6 * r(B, H, N, Dk) + offset * r(1, H, 1, Dk), 0.6 * r(B, Hk, M, Dk) + offset * r(1, Hk, 1, Dk)
    v, do = r(B, Hk, M, Dv) + offset * r(1, Hk, 1, Dv), r(B, H, N, Dv)
    if behind is not None:
        for b, n in enumerate(lengths):
            n = min(max(int(n), 0), M)
            k[b, :, n:], v[b, :, n:] = behind, behind
    return tuple(t.to(dtype) for t in (q, k, v, do))

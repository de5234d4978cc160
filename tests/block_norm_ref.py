"""The gated norm of heads and the residual norm in fp64 on the CPU, with their gradients written out."""
import numpy as np
import torch


def arr(t):
    return None if t is None else t.detach().cpu().double().numpy()


def stats(x, rms, eps=1e-5):
    mean = np.zeros(x.shape[:-1]) if rms else x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    return mean, 1 / np.sqrt(var + eps)


def sigmoid(g):
    return 0.5 * (1 + np.tanh(g / 2))


def norm_back(d, n, rstd, rms):
    return rstd[..., None] * (d - n * (d * n).mean(-1, keepdims=True) - (0 if rms else d.mean(-1, keepdims=True)))


def gated(o, gate, w=None, rms=False, dy=None):
    """y [B,N,H*D]; with dy: (do, dgate, dw), and the magnitudes of dw's terms summed."""
    o, gate, w, dy = arr(o), arr(gate), arr(w), arr(dy)
    B, H, N, D = o.shape
    heads = lambda t: t.reshape(B, N, H, D).transpose(0, 2, 1, 3)
    merged = lambda t: t.transpose(0, 2, 1, 3).reshape(B, N, H * D)
    w = np.ones(D) if w is None else w
    mean, rstd = stats(o, rms)
    n, g = (o - mean[..., None]) * rstd[..., None], heads(gate)
    s = sigmoid(g)
    if dy is None:
        return merged(n * w * g * s)
    dy = heads(dy)
    do = norm_back(dy * w * g * s, n, rstd, rms)
    dgate = dy * n * w * (s + g * s * (1 - s))
    terms = dy * n * g * s
    return do, merged(dgate), terms.sum((0, 1, 2)), np.abs(terms).sum((0, 1, 2))


def resid(x, a, scale=None, w=None, b=None, rms=False):
    x, a, scale, w, b = (arr(t) for t in (x, a, scale, w, b))
    h = x + a * (1 if scale is None else scale)
    mean, rstd = stats(h, rms)
    y = (h - mean[..., None]) * rstd[..., None] * (1 if w is None else w) + (0 if b is None else b)
    return h, y, mean, rstd


def resid_back(h, a, scale, w, mean, rstd, dy, dh, rms):
    """(dx, da, dscale, dw, db) from the given statistics, and the magnitudes of the last three."""
    h, a, scale, w, mean, rstd, dy, dh = (arr(t) for t in (h, a, scale, w, mean, rstd, dy, dh))
    n = (h - (0 if rms else mean[..., None])) * rstd[..., None]
    dx = norm_back(dy * (1 if w is None else w), n, rstd, rms) + (0 if dh is None else dh)
    rows = tuple(range(h.ndim - 1))
    terms = [None if a is None else a * dx, dy * n, dy]
    sums = [None if t is None else t.sum(rows) for t in terms]
    mags = [None if t is None else np.abs(t).sum(rows) for t in terms]
    return (dx, dx * (1 if scale is None else scale), *sums), mags

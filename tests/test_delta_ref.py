"""The fp64 references of the gated delta rule and layer norm, on the CPU: the gradients against
central differences and automatic differentiation, the forward against closed forms."""
import numpy as np
import pytest
import torch

import delta_ref as R


def case(seed, B, H, N, Dk, Dv):
    r = np.random.default_rng(seed)
    q, k, v, do = (r.standard_normal(s) for s in ((B, H, N, Dk), (B, H, N, Dk), (B, H, N, Dv), (B, H, N, Dv)))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    g = -np.log1p(np.exp(r.standard_normal((B, H, N)) - 2))
    beta = 1 / (1 + np.exp(-r.standard_normal((B, H, N))))
    return q, k, v, g, beta, do


def test_forward_closed_forms():
    q, k, v, g, beta, _ = case(0, 1, 2, 9, 4, 3)
    one = np.ones_like(beta)
    # beta = 0 writes nothing
    o, S = R.delta_fwd(q, k, v, g, 0 * beta)
    assert not o.any() and not S.any()
    # beta = 1 with unit keys: the state returns exactly v for the key just written
    o, _ = R.delta_fwd(k, k, v, g, one)
    assert np.allclose(o, v, atol=1e-14)
    # orthogonal keys (here the unit vectors) do not disturb each other: the decayed sum of linear attention
    eye = np.broadcast_to(np.eye(9)[None, None], (1, 2, 9, 9))
    _, S = R.delta_fwd(eye, eye, v, g, beta)
    rest = np.exp(np.flip(np.cumsum(np.flip(g, -1), -1), -1) - g)
    assert np.allclose(S, (rest * beta)[..., None] * v, atol=1e-14)
    # a = 0 forgets everything before it
    g2 = g.copy()
    g2[..., 5] = -np.inf
    o, S = R.delta_fwd(q, k, v, g2, beta)
    o5, S5 = R.delta_fwd(q[:, :, 5:], k[:, :, 5:], v[:, :, 5:], g[:, :, 5:], beta[:, :, 5:])
    assert np.array_equal(o[:, :, 5:], o5) and np.array_equal(S, S5)


def test_split_sequences_continue():
    q, k, v, g, beta, _ = case(1, 2, 1, 11, 4, 6)
    o, S = R.delta_fwd(q, k, v, g, beta)
    _, S1 = R.delta_fwd(q[:, :, :4], k[:, :, :4], v[:, :, :4], g[:, :, :4], beta[:, :, :4])
    o2, S2 = R.delta_fwd(q[:, :, 4:], k[:, :, 4:], v[:, :, 4:], g[:, :, 4:], beta[:, :, 4:], S1)
    assert np.allclose(o[:, :, 4:], o2, atol=1e-14) and np.allclose(S, S2, atol=1e-14)


def test_gradient_against_differences():
    xs = list(case(2, 1, 1, 5, 3, 2))
    do = xs.pop()
    grads = R.delta_bwd(*xs, do)
    h = 1e-6
    for n, gr in enumerate(grads):
        for i in np.ndindex(xs[n].shape):
            f = []
            for s in (h, -h):
                ys = [x.copy() for x in xs]
                ys[n][i] += s
                f.append(np.sum(do * R.delta_fwd(*ys)[0]))
            assert abs((f[0] - f[1]) / (2 * h) - gr[i]) < 1e-7


def test_gradient_against_autograd():
    xs = [torch.from_numpy(x) for x in case(3, 2, 2, 20, 6, 5)]
    do = xs.pop()
    leaves = [x.clone().requires_grad_() for x in xs]
    q, k, v, g, beta = leaves
    S = torch.zeros(2, 2, 6, 5, dtype=torch.float64)
    loss = 0
    for t in range(20):
        S = g[:, :, t].exp()[..., None, None] * S
        u = beta[:, :, t, None] * (v[:, :, t] - torch.einsum("bhd,bhde->bhe", k[:, :, t], S))
        S = S + k[:, :, t, :, None] * u[:, :, None]
        loss = loss + (do[:, :, t] * torch.einsum("bhd,bhde->bhe", q[:, :, t], S)).sum()
    loss.backward()
    for x, gr in zip(leaves, R.delta_bwd(*xs, do)):
        assert np.allclose(x.grad.numpy(), gr, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("shape,affine", [((7, 5), True), ((2, 3, 4), True), ((3, 1), False), ((4, 6), False)])
def test_norm_gradient_against_autograd(shape, affine):
    r = np.random.default_rng(4)
    x, dy = r.standard_normal(shape), r.standard_normal(shape)
    w, b = (r.standard_normal(shape[-1]), r.standard_normal(shape[-1])) if affine else (None, None)
    xt = torch.from_numpy(x).requires_grad_()
    wt, bt = (torch.from_numpy(t).requires_grad_() if affine else None for t in (w, b))
    y = torch.nn.functional.layer_norm(xt, shape[-1:], wt, bt)
    assert np.allclose(y.detach().numpy(), R.norm_fwd(x, w, b)[0], atol=1e-13)
    y.backward(torch.from_numpy(dy))
    dx, dw, db = R.norm_bwd(x, w, dy)
    assert np.allclose(xt.grad.numpy(), dx, atol=1e-12)
    if affine:
        assert np.allclose(wt.grad.numpy(), dw, atol=1e-12) and np.allclose(bt.grad.numpy(), db, atol=1e-12)

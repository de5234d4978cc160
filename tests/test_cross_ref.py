"""The fp64 reference of cross attention against autograd of the definition and against differences."""
import numpy as np
import pytest
import torch

import cross_ref as R

F64 = torch.float64


def definition(q, k, v, lengths):
    B, H, N, _ = q.shape
    Hk, M = k.shape[1:3]
    p = lambda t: torch.nn.functional.elu(t) + 1
    kk, vv = (t.repeat_interleave(H // Hk, 1) for t in (k, v))
    s = p(q) @ p(kk).transpose(-1, -2)
    if lengths is not None:
        s = s.masked_fill(torch.arange(M)[None, None, None] >= torch.tensor(lengths)[:, None, None, None], 0.0)
    den = s.sum(-1, keepdim=True)
    return (s / den.masked_fill(den == 0, 1.0)) @ vv


@pytest.mark.parametrize("lengths", [None, [7, 0]])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (3, 1)])
def test_reference(H, Hk, lengths):
    q, k, v, do = R.make(2, H, Hk, 5, 9, 4, 6, F64, seed=H)
    for t in (q, k, v):
        t.requires_grad_(True)
    o = definition(q, k, v, lengths)
    ref = R.fwd(q, k, v, lengths)
    assert np.abs(o.detach().numpy() - ref[0]).max() < 1e-13
    grads = torch.autograd.grad((o * do).sum(), (q, k, v))
    for a, b in zip(grads, R.bwd(q, k, v, do, lengths)[0]):
        assert np.abs(a.numpy() - b).max() < 1e-12


def test_gradient_against_differences():
    q, k, v, do = R.make(1, 2, 1, 3, 4, 3, 2, F64, seed=5)
    grads, _ = R.bwd(q, k, v, do)
    f = lambda: float((torch.as_tensor(R.fwd(q, k, v)[0]) * do).sum())
    step = 1e-6  # differences: error of step^2 and of 1e-16 / step
    for t, g in zip((q, k, v), grads):
        flat, out = t.view(-1), np.zeros(t.numel())
        for i in range(t.numel()):
            was = float(flat[i])
            flat[i] = was + step
            up = f()
            flat[i] = was - step
            out[i] = (up - f()) / (2 * step)
            flat[i] = was
        assert np.abs(out - g.reshape(-1)).max() < 1e-8

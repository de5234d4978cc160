"""The norms around a block on the CPU: the fp64 reference against autograd, refusals before any device call."""
import ctypes

import numpy as np
import pytest
import torch

import block_norm_ref as R

F64 = torch.float64


@pytest.fixture(scope="module")
def la():
    from causal_linear_attention_phi_gb300 import build
    build.build_library()
    import causal_linear_attention_phi_gb300 as la
    la.library()
    return la


def normed(x, rms):
    if rms:
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5)
    return torch.nn.functional.layer_norm(x, x.shape[-1:])


@pytest.mark.parametrize("rms", [False, True])
def test_reference_against_autograd(rms):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=F64)
    o, g, w, dy = r(2, 3, 4, 16).requires_grad_(), r(2, 4, 48).requires_grad_(), r(16).requires_grad_(), r(2, 4, 48)
    y = (normed(o, rms) * w).transpose(1, 2).reshape(2, 4, 48) * torch.nn.functional.silu(g)
    assert np.abs(R.gated(o, g, w, rms) - y.detach().numpy()).max() < 1e-12
    for a, b in zip(torch.autograd.grad((y * dy).sum(), (o, g, w)), R.gated(o, g, w, rms, dy)):
        assert np.abs(a.numpy() - b).max() < 1e-12
    x, a, s, w, b = (t.requires_grad_() for t in (r(5, 7), r(5, 7), r(7), r(7), r(7)))
    dy, dh = r(5, 7), r(5, 7)
    h = x + s * a
    y = normed(h, rms) * w + b
    ref = R.resid(x, a, s, w, b, rms)
    assert max(np.abs(ref[0] - h.detach().numpy()).max(), np.abs(ref[1] - y.detach().numpy()).max()) < 1e-12
    grads = torch.autograd.grad((y * dy).sum() + (h * dh).sum(), (x, a, s, w, b))
    back, _ = R.resid_back(h, a, s, w, torch.tensor(ref[2]), torch.tensor(ref[3]), dy, dh, rms)
    for p, q in zip(grads, back):
        assert np.abs(p.numpy() - q).max() < 1e-12


def test_shapes_refused_on_the_host(la):
    lib, p = la.library(), ctypes.c_void_p(0)
    gf = lambda s, eps=1e-5: lib.la_gated_norm_fwd(*[p] * 4, la.HeadsShape(*s), 0, eps, None)
    gb = lambda s, eps=1e-5: lib.la_gated_norm_bwd(*[p] * 7, la.HeadsShape(*s), 1, eps, p, 0, None)
    for f in (gf, gb):
        assert f((-1, 1, 1, 16, 0)) == 1 and f((1, 1, 1, 16, 3)) == 1 and f((1, 1, 1, 16, 0), -1.0) == 1
        assert f((1, 1, 1, 24, 0)) == 2 and f((1, 1, 1, 256, 0)) == 2 and f((300, 300, 1, 16, 0)) == 2
        assert f((0, 1, 1, 16, 0)) == 0 and f((1, 1, 0, 16, 1)) == 0
    rf = lambda s, eps=1e-5: lib.la_residual_norm_fwd(*[p] * 9, la.NormShape(*s), 0, eps, None)
    rb = lambda s: lib.la_residual_norm_bwd(*[p] * 13, la.NormShape(*s), 0, p, 0, None)
    for f in (rf, rb):
        assert f((-1, 8, 0)) == 1 and f((1, 0, 0)) == 1 and f((1, 8, 2)) == 1 and f((1, 16385, 0)) == 2 and f((0, 8, 0)) == 0
    assert rf((4, 8, 0), -1.0) == 1 and rf((4, 8, 0), float("nan")) == 1


def test_workspace_queries(la):
    for dt in (torch.float32, torch.bfloat16):
        assert la.gated_norm_workspace_bytes(2, 4, 100, 64, dt) > 0 and la.gated_norm_workspace_bytes(2, 4, 0, 64, dt) == 0
        assert la.gated_norm_workspace_bytes(2, 4, 100, 65, dt) == 0
        assert la.residual_norm_workspace_bytes(100, 1001, dt) > 0 and la.residual_norm_workspace_bytes(0, 64, dt) == 0
    for f in (la.gated_norm_workspace_bytes, la.residual_norm_workspace_bytes):
        with pytest.raises(TypeError):
            f(*((1, 1, 1, 16) if f is la.gated_norm_workspace_bytes else (1, 16)), torch.float64)


def test_binding_refuses_host_tensors(la):
    t = torch.zeros(2, 2, 4, 16)
    for call in (lambda: la.gated_norm_fwd(t, t), lambda: la.gated_norm_bwd(t, t, None, t), lambda: la.residual_norm_fwd(t, t),
                 lambda: la.residual_norm_bwd(t, None, None, None, None, t, t, rms=True)):
        with pytest.raises(TypeError):
            call()

"""Gradients of the gated delta rule through an initial and a final state: a long sequence in pieces.

The reference is torch's autograd of the recurrence, position by position, in fp64.  Bounds as for the gradients of
whole sequences (tests/test_gpu_gated_delta.py: 4 * 320 * 2^-24 in fp32, 16 times 320 * 2^-24 for dg, 5 * 2^-8 in
bf16); the gradient of the first state passes the same recurrence, with (gam dO) as its one operand that is rounded to
bf16 alone.  Two pieces pass the bound twice.
"""
import ctypes

import numpy as np
import pytest
import torch

from util import rel_per_head, to_np

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
TOL_F32 = 320 * 2.0 ** -24


def bound(name, dtype):
    return (16 if name == "dg" else 4) * TOL_F32 if dtype == F32 else 5 * 2.0 ** -8


def make(seed, B, H, N, Dk, Dv, dtype):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q, k, v, do = unit(rn(B, H, N, Dk)), unit(rn(B, H, N, Dk)), rn(B, H, N, Dv), rn(B, H, N, Dv)
    g, beta = -torch.nn.functional.softplus(rn(B, H, N) - 3), torch.sigmoid(rn(B, H, N))
    return [t.to(dtype) for t in (q, k, v, g, beta, do)], rn(B, H, Dk, Dv), rn(B, H, Dk, Dv)


def reference(q, k, v, g, beta, do, S0, dS):
    """(dq, dk, dv, dg, dbeta, dS0) of sum(do o) + sum(dS S) in fp64."""
    leaves = [t.double().requires_grad_(True) for t in (q, k, v, g, beta, S0)]
    q, k, v, g, beta, S = leaves
    total = 0.0
    for t in range(q.shape[2]):
        a = torch.exp(g[:, :, t])[..., None, None]
        u = beta[:, :, t, None] * (v[:, :, t] - torch.einsum("bhd,bhde->bhe", k[:, :, t], a * S))
        S = a * S + k[:, :, t, :, None] * u[:, :, None]
        total = total + (torch.einsum("bhd,bhde->bhe", q[:, :, t], S) * do[:, :, t].double()).sum()
    return torch.autograd.grad(total + (S * dS.double()).sum(), leaves)


def close(name, x, ref, tol):
    x, ref = to_np(x), np.asarray(ref.detach() if isinstance(ref, torch.Tensor) else ref)
    if x.ndim == 3:
        x, ref = x[..., None], ref[..., None]
    e = rel_per_head(x, ref)
    assert e <= tol, "%s: max rel err %.3e > %.3e" % (name, e, tol)


NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def test_reference_against_differences():
    """The reference's dS0 and its use of dS against central differences of the recurrence."""
    (q, k, v, g, beta, do), S0, dS = make(1, 1, 1, 3, 2, 2, torch.float64)
    S0, dS = S0.double(), dS.double()
    grads = reference(q, k, v, g, beta, do, S0, dS)

    def value(S0, v):
        S = S0.clone()
        out = 0.0
        for t in range(3):
            a = float(torch.exp(g[0, 0, t]))
            u = float(beta[0, 0, t]) * (v[0, 0, t] - a * S[0, 0].T @ k[0, 0, t])
            S[0, 0] = a * S[0, 0] + torch.outer(k[0, 0, t], u)
            out += float((S[0, 0].T @ q[0, 0, t]) @ do[0, 0, t])
        return out + float((S * dS).sum())

    h = 1e-6
    for i in range(2):
        for j in range(2):
            e = torch.zeros_like(S0)
            e[0, 0, i, j] = h
            assert abs((value(S0 + e, v) - value(S0 - e, v)) / (2 * h) - float(grads[5][0, 0, i, j])) < 1e-7
        e = torch.zeros_like(v)
        e[0, 0, i, 1] = h
        assert abs((value(S0, v + e) - value(S0, v - e)) / (2 * h) - float(grads[2][0, 0, i, 1])) < 1e-7


@pytest.mark.parametrize("shape,want", [((-1, 1, 8, 16, 16, 0), 1), ((1, 1, 8, 16, 16, 5), 1), ((1, 1, 8, 48, 16, 0), 2),
                                        ((0, 1, 8, 16, 16, 0), 0), ((1, 1, 0, 16, 16, 0), 0)])
def test_shapes(shape, want):
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    null = ctypes.c_void_p(0)
    assert la.library().la_gated_delta_bwd_with_state(*[null] * 14, la.Shape(*shape), null, 0, None) == want


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    la.library()
    la.clear_error()
    yield la
    assert la.last_error() == 0


CASES = [(1, 2, 1, 16, 32, F32), (2, 2, 70, 64, 16, F32), (1, 3, 200, 128, 128, F32), (1, 40, 100, 32, 64, F32),
         (1, 2, 1, 64, 64, BF16), (2, 2, 65, 64, 64, BF16), (1, 3, 500, 64, 64, BF16), (1, 2, 130, 32, 128, BF16),
         (1, 2, 64, 128, 128, BF16), (1, 2, 700, 128, 128, BF16), (1, 2, 300, 128, 16, BF16)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,N,Dk,Dv,dtype", CASES)
def test_states(la, B, H, N, Dk, Dv, dtype):
    ins, S0, dS = make(N + Dk, B, H, N, Dk, Dv, dtype)
    ref = reference(*ins, S0, dS)
    dev = [t.to(DEV) for t in ins]
    got = la.gated_delta_bwd(*dev, S0=S0.to(DEV), dS=dS.to(DEV), return_dS0=True)
    assert got[5].dtype == F32 and got[5].shape == S0.shape
    for n, x, r in zip(NAMES, got, ref):
        close(n, x, r, bound(n, dtype))
    # without the final gradient, and without a state: the call for whole sequences
    ref = reference(*ins, S0, torch.zeros_like(dS))
    for n, x, r in zip(NAMES, la.gated_delta_bwd(*dev, S0=S0.to(DEV), return_dS0=True), ref):
        close(n, x, r, bound(n, dtype))
    zero = torch.zeros_like(S0, device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(la.gated_delta_bwd(*dev), la.gated_delta_bwd(*dev, S0=zero, dS=zero)))


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(32, F32), (64, BF16), (128, BF16)])
def test_two_pieces_are_the_whole(la, D, dtype):
    ins, _, dS = make(5, 1, 2, 330, D, D, dtype)
    ref = reference(*ins, torch.zeros_like(dS), torch.zeros_like(dS))
    first, second = ([t[:, :, s].contiguous().to(DEV) for t in ins] for s in (slice(0, 201), slice(201, 330)))
    _, S = la.gated_delta_fwd(*first[:5], return_state=True)
    tail = la.gated_delta_bwd(*second, S0=S, return_dS0=True)
    head = la.gated_delta_bwd(*first, dS=tail[5])
    for n, a, b, r in zip(NAMES, head, tail, ref):
        close(n, torch.cat((a, b), 2), r, 2 * bound(n, dtype))


@pytest.mark.gpu
def test_no_position_and_refusals(la):
    z = lambda *s: torch.zeros(*s, device=DEV)
    dS = torch.randn(1, 2, 16, 32, device=DEV)
    empty = (z(1, 2, 0, 16), z(1, 2, 0, 16), z(1, 2, 0, 32), z(1, 2, 0), z(1, 2, 0), z(1, 2, 0, 32))
    assert torch.equal(la.gated_delta_bwd(*empty, dS=dS, return_dS0=True)[5], dS)
    assert not la.gated_delta_bwd(*empty, return_dS0=True)[5].any()
    ins = [t.to(DEV) for t in make(6, 1, 2, 9, 16, 32, F32)[0]]
    for bad in (dict(S0=dS[:, :, :15].contiguous()), dict(dS=dS.bfloat16()), dict(S0=dS[:, :1].contiguous())):
        with pytest.raises(ValueError):
            la.gated_delta_bwd(*ins, **bad)

"""GPU parity of the gated delta rule (forward, gradient, decode step) against the fp64 recurrence.

Error of an output: per (b, h) slice, max|gpu - ref| / max|ref|.  Bounds, from the roundings on the way:
- fp32: sums of at most 64 + 2 * 128 terms in a chunk, each addition off by half a step: 320 * 2^-24; the
  gradient passes two such recurrences and three products: 4 times that (dg, a sum of differences
  of such products, 16 times).
- bf16: half a step of the output (2^-8) and as much again for the operands that are rounded to bf16; the gradient
  has four such operands on its longest path (P, the stored state and its gradient, the pair products), so
  5 * 2^-8.  Returned states are fp32 formed from operands in two bf16 parts: 2^-17 a rounding, at most
  six of them, over sums that cancel by no more than 8 here: 48 * 2^-17.
"""
import math

import numpy as np
import pytest
import torch

import delta_ref as R
from util import rel_per_head, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
TOL_F32, TOL_BF16 = 320 * 2.0 ** -24, 2 * 2.0 ** -8
TOL_STATE = {F32: TOL_F32, BF16: 48 * 2.0 ** -17}


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


def make(seed, B, H, N, Dk, Dv, dtype, gates="usual", shared=0.5):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    common = shared * rn(1, H, 1, Dk)
    q, k, v, do = unit(rn(B, H, N, Dk) + common), unit(rn(B, H, N, Dk) + common), rn(B, H, N, Dv), rn(B, H, N, Dv)
    g = -torch.nn.functional.softplus(rn(B, H, N) - 3)
    beta = torch.sigmoid(rn(B, H, N))
    if gates == "packed":
        g[torch.rand(B, H, N, generator=gen) < 0.03] = -math.inf
        g[..., N // 2] = -math.inf
    elif gates == "extreme":  # no decay, hard decay, decays past fp32's range, no write, a whole write
        g = torch.tensor([0.0, -30.0, -200.0, -1e-4, -95.0, -0.5])[torch.randint(6, (B, H, N), generator=gen)]
        beta = torch.tensor([0.0, 1.0, 0.5])[torch.randint(3, (B, H, N), generator=gen)]
    elif gates == "none":
        g, beta = torch.zeros(B, H, N), torch.ones(B, H, N)
    elif gates == "closed":
        g, beta = torch.full((B, H, N), -math.inf), beta
    return tuple(t.to(dtype) for t in (q, k, v, g, beta, do))


def dev(*ts):
    return [t.to(DEV) for t in ts]


def close(name, x, ref, tol):
    x, ref = to_np(x), np.asarray(ref)
    if x.ndim == 3:  # gates
        x, ref = x[..., None], ref[..., None]
    e = rel_per_head(x, ref)
    assert e <= tol, "%s: max rel err %.3e > %.3e" % (name, e, tol)


CASES = [
    # B, H, N, Dk, Dv, dtype, gates
    (1, 1, 1, 16, 16, F32, "usual"),
    (1, 2, 2, 16, 128, F32, "none"),
    (2, 3, 63, 32, 16, F32, "packed"),
    (1, 2, 64, 64, 64, F32, "usual"),
    (1, 3, 65, 128, 32, F32, "extreme"),
    (2, 2, 200, 128, 128, F32, "usual"),
    (1, 1, 777, 64, 16, F32, "none"),
    (1, 2, 130, 16, 64, F32, "closed"),
    (1, 3, 129, 32, 64, BF16, "usual"),
    (2, 1, 100, 128, 64, BF16, "packed"),
    (1, 1, 1, 64, 64, BF16, "usual"),
    (1, 2, 64, 64, 64, BF16, "extreme"),
    (2, 2, 65, 64, 64, BF16, "packed"),
    (1, 3, 500, 64, 64, BF16, "usual"),
    (1, 1, 1, 128, 128, BF16, "none"),
    (1, 2, 63, 128, 128, BF16, "packed"),
    (3, 1, 64, 128, 128, BF16, "usual"),
    (1, 2, 129, 128, 128, BF16, "extreme"),
    (1, 2, 1100, 128, 128, BF16, "packed"),
    (1, 1, 700, 128, 128, BF16, "none"),
    (1, 2, 192, 128, 128, BF16, "closed"),
]


@pytest.mark.parametrize("B,H,N,Dk,Dv,dtype,gates", CASES)
def test_fwd(la, B, H, N, Dk, Dv, dtype, gates):
    q, k, v, g, beta, _ = make(N + Dk, B, H, N, Dk, Dv, dtype, gates)
    o, S = la.gated_delta_fwd(*dev(q, k, v, g, beta), return_state=True)
    assert o.dtype == dtype and S.dtype == F32 and o.shape == v.shape
    ro, rS = R.delta_fwd(q, k, v, g, beta)
    close("o", o, ro, TOL_BF16 if dtype == BF16 else TOL_F32)
    close("S", S, rS, TOL_STATE[dtype])
    assert torch.equal(o, la.gated_delta_fwd(*dev(q, k, v, g, beta)))  # with and without the state


@pytest.mark.parametrize("B,H,N,Dk,Dv,dtype,gates", CASES)
def test_bwd(la, B, H, N, Dk, Dv, dtype, gates):
    q, k, v, g, beta, do = make(N + Dv, B, H, N, Dk, Dv, dtype, gates)
    ref = R.delta_bwd(q, k, v, g, beta, do)
    got = la.gated_delta_bwd(*dev(q, k, v, g, beta, do))
    for n, x, r in zip(("dq", "dk", "dv", "dg", "dbeta"), got, ref):
        assert x.dtype == dtype
        f = 16 if n == "dg" else 4
        tol = f * TOL_F32 if dtype == F32 else 5 * 2.0 ** -8
        if N == 1 and n == "dg" or gates == "closed" and n == "dg":
            assert not to_np(x).any()  # nothing decays into the only position, or into any
            continue
        close(n, x, r, tol)
    if gates in ("packed", "extreme"):
        assert not to_np(got[3])[to_np(g) < -100].any()
    again = la.gated_delta_bwd(*dev(q, k, v, g, beta, do))
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # no order of atomics in the results


@pytest.mark.parametrize("D,dtype", [(32, F32), (64, BF16), (128, BF16)])
def test_state_carries_over_pieces(la, D, dtype):
    """A sequence in pieces of 1, 64 and odd lengths, the state handed on in place, ending in decode steps."""
    B, H, N = 2, 2, 260
    q, k, v, g, beta, _ = make(9, B, H, N, D, D, dtype, "packed")
    ro, rS = R.delta_fwd(q, k, v, g, beta)
    S, outs, at = torch.zeros(B, H, D, D, device=DEV), [], 0
    for n in (1, 64, 65, 127):
        piece = [t[:, :, at:at + n].contiguous() for t in dev(q, k, v, g, beta)]
        o, S = la.gated_delta_fwd(*piece, S0=S, return_state=True)
        outs.append(o)
        at += n
    for t in range(at, N):
        step = [x[:, :, t].contiguous() for x in dev(q, k, v, g, beta)]
        outs.append(la.gated_delta_step(*step, S)[:, :, None])
    close("o", torch.cat(outs, 2), ro, TOL_BF16 if dtype == BF16 else 2 * TOL_F32)
    close("S", S, rS, 2 * TOL_STATE[dtype])


def test_state_of_no_position_and_in_place(la):
    S0 = torch.randn(1, 2, 16, 32, device=DEV)
    z = lambda *s: torch.zeros(*s, device=DEV)
    o, S = la.gated_delta_fwd(z(1, 2, 0, 16), z(1, 2, 0, 16), z(1, 2, 0, 32), z(1, 2, 0), z(1, 2, 0), S0=S0,
                              return_state=True)
    assert o.numel() == 0 and torch.equal(S, S0)
    _, S = la.gated_delta_fwd(z(1, 2, 0, 16), z(1, 2, 0, 16), z(1, 2, 0, 32), z(1, 2, 0), z(1, 2, 0),
                              return_state=True)
    assert not S.any()


STEP_CASES = [(1, 1, 16, 16, F32), (3, 5, 16, 128, F32), (2, 3, 32, 32, F32), (1, 3, 64, 16, BF16),
              (2, 2, 64, 64, BF16), (1, 5, 128, 16, F32), (1, 2, 128, 64, BF16), (2, 4, 128, 128, BF16),
              (1, 1, 128, 128, F32), (1, 3, 32, 128, BF16), (300, 16, 16, 32, F32)]


@pytest.mark.parametrize("B,H,Dk,Dv,dtype", STEP_CASES)
def test_step(la, B, H, Dk, Dv, dtype):
    T = 4 if B < 100 else 1
    q, k, v, g, beta, _ = make(B + Dk, B, H, T, Dk, Dv, dtype)
    g[0, 0, T - 1] = -math.inf
    gen = torch.Generator().manual_seed(1)
    S = torch.randn(B, H, Dk, Dv, generator=gen)
    ro, rS = R.delta_fwd(q, k, v, g, beta, S)
    S = S.to(DEV)
    outs = [la.gated_delta_step(*[x[:, :, t].contiguous() for x in dev(q, k, v, g, beta)], S) for t in range(T)]
    close("out", torch.stack(outs, 2), ro, 2.0 ** -8 + TOL_F32 if dtype == BF16 else TOL_F32)
    close("S", S, rS, TOL_F32)


def test_other_streams_and_graphs(la):
    """The forward, the gradient and the step on a side stream and replayed from a graph give the same bits."""
    q, k, v, g, beta, do = dev(*make(2, 1, 2, 300, 128, 128, BF16))
    S = torch.randn(1, 2, 128, 128, device=DEV)
    one = [x[:, :, 0].contiguous() for x in (q, k, v, g, beta)]
    o, grads = la.gated_delta_fwd(q, k, v, g, beta), la.gated_delta_bwd(q, k, v, g, beta, do)
    S1 = S.clone()
    out1 = la.gated_delta_step(*one, S1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        o2, g2 = la.gated_delta_fwd(q, k, v, g, beta), la.gated_delta_bwd(q, k, v, g, beta, do)
    st.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(grads, g2))
    ws = torch.empty(la.workspace_bytes(la.OP_GATED_DELTA_BWD, 1, 2, 300, 128, 128, BF16), dtype=torch.uint8,
                     device=DEV)
    outs = [torch.zeros_like(t) for t in (v, q, k, v, g, beta)]
    S2, out2 = S.clone(), torch.zeros_like(out1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.gated_delta_fwd(q, k, v, g, beta, out=outs[0], workspace=ws)
        la.gated_delta_bwd(q, k, v, g, beta, do, *outs[1:], workspace=ws)
        la.gated_delta_step(*one, S2, out=out2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], o) and all(torch.equal(a, b) for a, b in zip(outs[1:], grads))
    assert torch.equal(out2, out1) and torch.equal(S2, S1)


def test_refusals(la):
    q, k, v, g, beta, do = dev(*make(3, 1, 2, 70, 64, 64, BF16))
    with pytest.raises(ValueError):
        la.gated_delta_fwd(q, k, v, g[:, :, :69].contiguous(), beta)
    with pytest.raises(ValueError):
        la.gated_delta_fwd(q, k, v, g.float(), beta)
    with pytest.raises(ValueError):
        la.gated_delta_fwd(q, k, v.transpose(1, 2), g, beta)
    with pytest.raises(ValueError):
        la.gated_delta_fwd(q, k, v, g, beta, S0=torch.zeros(1, 2, 64, 32, device=DEV))
    with pytest.raises(ValueError):
        la.gated_delta_fwd(q, k, v, g, beta, out=torch.empty_like(v[:, :, :69]))
    with pytest.raises(ValueError):
        la.gated_delta_bwd(q, k, v, g, beta, do.float())
    with pytest.raises(ValueError):
        la.gated_delta_bwd(q, k, v, g, beta, do, dg=torch.empty_like(g[..., :69]))
    with pytest.raises(la.LaError) as e:
        la.gated_delta_fwd(q, k, v, g, beta, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == 3
    with pytest.raises(la.LaError) as e:
        la.gated_delta_bwd(q, k, v, g, beta, do, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == 3
    with pytest.raises(ValueError):
        la.gated_delta_step(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(),
                            g[:, :, 0].contiguous(), beta[:, :, 0].contiguous(),
                            torch.zeros(1, 2, 64, 64, device=DEV, dtype=BF16))
    # a pointer that is not 16-byte aligned: a view one element on
    flat = torch.zeros(2 * 70 * 64 + 1, device=DEV, dtype=BF16)
    with pytest.raises(la.LaError) as e:
        la.gated_delta_fwd(flat[1:].view(1, 2, 70, 64), k, v, g, beta)
    assert e.value.status == 1
    # gates need their elements' alignment only
    gf = torch.zeros(2 * 70 + 1, device=DEV, dtype=BF16)
    gf[1:] = g.flatten()
    assert torch.equal(la.gated_delta_fwd(q, k, v, gf[1:].view(1, 2, 70), beta), la.gated_delta_fwd(q, k, v, g, beta))

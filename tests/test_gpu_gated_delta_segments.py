"""The gated delta rule in bf16 over sequences that are cut into segments: both padded sizes, every width of the join's
blocks in both directions, padded heads, and states in and out.

That a case is cut is read off the size of its workspace (on the CPU), so a change of the plan that leaves one of
these ways without a case fails there.  The reference is the recurrence and its adjoint in fp64, position by position, of the
first, a middle and the last head.  Bounds as for sequences of one segment (tests/test_gpu_gated_delta.py and
tests/test_gated_delta_pieces.py): joining adds fp32 sums to what those bounds count.
"""
import math

import numpy as np
import pytest
import torch

from test_gated_delta_pieces import NAMES, bound, close, make as make_small, reference
from util import to_np

DEV = "cuda:0"
BF16 = torch.bfloat16
TOL_O, TOL_S = 2 * 2.0 ** -8, 48 * 2.0 ** -17

# H, N, Dk, Dv
CASES = [(2, 1300, 64, 64), (12, 2000, 64, 64), (25, 2000, 64, 64), (50, 2000, 64, 64), (3, 2000, 64, 32),
         (3, 1100, 16, 32), (2, 1500, 128, 128), (6, 1500, 128, 128), (12, 1500, 128, 128), (24, 1500, 128, 128),
         (2, 1500, 32, 128), (2, 1500, 128, 16)]


def padded(Dk, Dv):
    return 128 if max(Dk, Dv) > 64 else 64


def segments(la, bwd, H, N, Dk, Dv):
    """Segments of a head: what the workspace holds beside its regions for chunks, in records of a segment."""
    up = lambda n: (n + 255) // 256 * 256
    D, chunks = padded(Dk, Dv), H * ((N + 63) // 64)
    fixed = up(chunks * 9 * 64 * 4) + up((3 if bwd else 2) * chunks * 64 * 64 * 4)
    if bwd:
        fixed += 2 * up(chunks * 64 * D * 4) + 2 * up(chunks * D * D * 2)
    op = la.OP_GATED_DELTA_BWD if bwd else la.OP_GATED_DELTA_FWD
    extra = la.workspace_bytes(op, 1, H, N, Dk, Dv, BF16) - fixed
    n, rest = divmod(extra, (5 if bwd else 3) * H * D * D * 4)
    assert rest == 0 and n != 1
    return max(n, 1)


def join_columns(bwd, H, Dk, Dv):
    """Value columns of a block of the join (join in tc_gated_delta.cu)."""
    slices = H * (padded(Dk, Dv) // 16) * (2 if bwd else 1)
    return 8 if 2 * slices <= 152 else 16 if slices <= 152 else 32


def test_cases_are_cut():
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    cut = [(bwd, c) for bwd in (False, True) for c in CASES if segments(la, bwd, *c) > 1]
    joins = {(bwd, padded(*c[2:]), join_columns(bwd, c[0], *c[2:])) for bwd, c in cut}
    assert joins == {(b, D, cols) for b in (False, True) for D in (64, 128) for cols in (8, 16, 32)}
    for bwd in (False, True):
        assert {c for b, c in cut if b == bwd} >= {c for c in CASES if c[2] != c[3]}  # padded heads


def make(seed, H, N, Dk, Dv, gates):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    common = 0.5 * rn(1, H, 1, Dk)
    q, k, v, do = unit(rn(1, H, N, Dk) + common), unit(rn(1, H, N, Dk) + common), rn(1, H, N, Dv), rn(1, H, N, Dv)
    # decays slow enough that a state is felt segments later
    g = -torch.nn.functional.softplus(rn(1, H, N) - 8)
    beta = torch.sigmoid(rn(1, H, N) - 1)
    if gates == "packed":
        g[torch.rand(1, H, N, generator=gen) < 0.002] = -math.inf
        g[..., N // 2] = -math.inf
    return [t.to(BF16) for t in (q, k, v, g, beta, do)], rn(1, H, Dk, Dv), rn(1, H, Dk, Dv)


def recurrence(q, k, v, g, beta, do, S0, dS):
    """((o, S), (dq, dk, dv, dg, dbeta, dS0)) of sum(do o) + sum(dS S) in fp64; arrays [1, heads, ...]."""
    q, k, v, g, beta, do, S, D = (to_np(t)[0] for t in (q, k, v, g, beta, do, S0, dS))
    nh, N, _ = q.shape
    a = np.where(g < -100, 0, np.exp(g))  # the rule's reset
    Ss = np.zeros((N + 1,) + S.shape)
    Ss[0] = S
    e, o = np.zeros_like(v), np.zeros_like(v)
    for t in range(N):
        Sd = a[:, t, None, None] * Ss[t]
        e[:, t] = v[:, t] - np.einsum("hd,hde->he", k[:, t], Sd)
        Ss[t + 1] = Sd + k[:, t, :, None] * (beta[:, t, None] * e[:, t])[:, None]
        o[:, t] = np.einsum("hd,hde->he", q[:, t], Ss[t + 1])
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    for t in range(N - 1, -1, -1):
        Sd = a[:, t, None, None] * Ss[t]
        dq[:, t] = np.einsum("hde,he->hd", Ss[t + 1], do[:, t])
        D = D + q[:, t, :, None] * do[:, t, None]
        du = np.einsum("hd,hde->he", k[:, t], D)
        db[:, t] = np.sum(du * e[:, t], -1)
        de = beta[:, t, None] * du
        dv[:, t] = de
        dk[:, t] = np.einsum("hde,he->hd", D, beta[:, t, None] * e[:, t]) - np.einsum("hde,he->hd", Sd, de)
        D = D - k[:, t, :, None] * de[:, None]
        dg[:, t] = np.sum(D * Sd, (-1, -2))
        D = a[:, t, None, None] * D
    return (o[None], Ss[N][None]), tuple(x[None] for x in (dq, dk, dv, dg, db, D))


def test_recurrence_against_autograd():
    ins, S0, dS = make_small(3, 1, 2, 9, 3, 4, torch.float64)
    ref = reference(*ins, S0.double(), dS.double())
    for name, x, r in zip(NAMES, recurrence(*ins, S0.double(), dS.double())[1], ref):
        close(name, x, r, 1e-12)


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


@pytest.mark.gpu
@pytest.mark.parametrize("gates", ["slow", "packed"])
@pytest.mark.parametrize("H,N,Dk,Dv", CASES)
def test_segments(la, H, N, Dk, Dv, gates):
    ins, S0, dS = make(N + H + Dk, H, N, Dk, Dv, gates)
    heads = sorted({0, H // 2, H - 1})
    (ro, rS), grads = recurrence(*(t[:, heads] for t in ins), S0[:, heads], dS[:, heads])
    dev, S0d, dSd = [t.to(DEV) for t in ins], S0.to(DEV), dS.to(DEV)
    o, S = la.gated_delta_fwd(*dev[:5], S0=S0d, return_state=True)
    close("o", o[:, heads], ro, TOL_O)
    close("S", S[:, heads], rS, TOL_S)
    got = la.gated_delta_bwd(*dev, S0=S0d, dS=dSd, return_dS0=True)
    for name, x, r in zip(NAMES, got, grads):
        close(name, x[:, heads], r, bound(name, BF16))
    if gates == "packed":
        assert not to_np(got[3])[to_np(ins[3]) < -100].any()
    # a state that is zero is no state; nothing depends on an order of blocks
    zero = torch.zeros_like(S0d)
    first = la.gated_delta_fwd(*dev[:5], return_state=True) + la.gated_delta_bwd(*dev)
    again = la.gated_delta_fwd(*dev[:5], S0=zero, return_state=True) + la.gated_delta_bwd(*dev, S0=zero, dS=zero)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    assert torch.equal(o, la.gated_delta_fwd(*dev[:5], S0=S0d))

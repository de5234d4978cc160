"""A NaN among the keys that count, or in a query, shows wherever the definition has it: outputs, states and gradients are NaN
exactly where the plain form's are, and the other heads are as they were, bit for bit."""
import numpy as np
import pytest
import torch

import cross_ref as R
from util import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
NAN = float("nan")


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


def plain(q, k, v, do, lengths):
    """o, S, z, dq, dk, dv in fp64 by elementary operations, of the keys that count (0 behind them)."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    phi = lambda t: torch.where(t > 0, t + 1, torch.exp(t.clamp(max=0)))  # NaN > 0 is false, exp(NaN) is NaN
    slope = lambda t: torch.where(t > 0, torch.ones_like(t), torch.exp(t.clamp(max=0)))
    B, H = q.shape[:2]
    Hk, M = k.shape[1:3]
    G = H // Hk
    outs = [torch.zeros(B, H, q.shape[2], v.shape[3]), torch.zeros(B, Hk, q.shape[3], v.shape[3]), torch.zeros(B, Hk, q.shape[3]),
            torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    for b in range(B):
        n = lengths[b]
        for j in range(Hk):
            h = slice(G * j, G * j + G)
            pq, pk, vj, dj = phi(q[b, h]).flatten(0, 1), phi(k[b, j, :n]), v[b, j, :n], do[b, h].flatten(0, 1)
            S, z = pk.T @ vj, pk.sum(0)
            den = (pq @ z)[:, None]
            Y = dj @ S.T / den
            t = (pq * Y).sum(1, keepdim=True)
            X = pq / den
            outs[0][b, h] = ((pq @ S) / den).unflatten(0, (G, -1))
            outs[1][b, j], outs[2][b, j] = S, z
            outs[3][b, h] = ((Y - t / den * z) * slope(q[b, h]).flatten(0, 1)).unflatten(0, (G, -1))
            outs[4][b, j, :n] = (vj @ (X.T @ dj).T - (X * t).sum(0)) * slope(k[b, j, :n])
            outs[5][b, j, :n] = pk @ (X.T @ dj)
    return outs


# H, Hk, N, M, Dk, Dv, dtype: one chunk to a head, a few queries, several chunks, both paths
CASES = [(2, 2, 17, 60, 16, 32, F32), (4, 2, 100, 200, 64, 64, F32), (2, 1, 70, 150, 128, 128, F32),
         (2, 2, 100, 60, 64, 64, BF16), (4, 2, 200, 300, 128, 128, BF16), (2, 1, 130, 200, 128, 64, BF16), (2, 2, 20, 140, 16, 128, BF16)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("where", ["k", "q"])
def test_nan_stays(la, case, where):
    H, Hk, N, M, Dk, Dv, dtype = case
    lengths = [M, M - 9]
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    q, k, v, do = R.make(2, H, Hk, N, M, Dk, Dv, dtype, seed=N)

    def everything(q, k):
        x, g = [t.to(DEV) for t in (q, k, v)], do.to(DEV)
        o, S, z = la.cross_fwd(*x, lengths=n, return_state=True)
        return (o, S, z, *la.cross_bwd(*x, g, lengths=n), *la.cross_bwd(*x, g, lengths=n, S=S, z=z))

    clean = everything(q, k)
    assert all(bool(torch.isfinite(t).all()) for t in clean)
    if where == "k":
        k[1, Hk - 1, M - 20, Dk - 1] = NAN
    else:
        q[1, H - 1, N - 3, 5] = NAN
    got, want = everything(q, k), plain(q, k, v, do, lengths)
    for i, (g, c) in enumerate(zip(got, clean)):
        w = want[i if i < 6 else i - 3]
        assert np.array_equal(np.isnan(to_np(g)), torch.isnan(w).numpy()), ("o", "S", "z", "dq", "dk", "dv", "dq", "dk", "dv")[i]
        assert torch.equal(g[0], c[0]), i
        heads = g.shape[1] // Hk * (Hk - 1)
        assert torch.equal(g[1, :heads], c[1, :heads]), i


@pytest.mark.parametrize("N", [1, 2, 7, 40, 200])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_in_a_query_to_a_kept_state(la, dtype, N):
    q = torch.randn(2, 4, N, 64, device=DEV).to(dtype)
    S, z = torch.randn(2, 2, 64, 128, device=DEV), 1 + torch.rand(2, 2, 64, device=DEV)
    clean = la.cross_apply(q, S, z)
    q[1, 2, N - 1, 63] = NAN
    got = la.cross_apply(q, S, z)
    assert bool(torch.isnan(got[1, 2, N - 1]).all())
    got[1, 2, N - 1] = clean[1, 2, N - 1]
    assert torch.equal(got, clean)

"""The bf16 gradient of cross attention where the values have a large part in common: dq and dk, which it drops out of, are as near
the exact ones as the same gradient in fp32 leaves them, and their own rounding.

Bounds.  One key: the exact dq and dk are 0.  With u = 2^-24, roundings of the terms' magnitudes only: a product accumulated in
tensor memory may be cut by 2 u (S is one such sum, hi and lo parts exact), the vector c that is taken out of S is rounded once,
so what is left of S is at most 5 u of its terms, and dq, linear in it twice (Y and t), 5 u of its magnitude, which counts both.
dk = R v + r takes 5 u from each again and at most 16 accumulations of R v (2 u each) and 16 additions of R c: 58 u of its
magnitude, which is twice its terms'.  Twice these are allowed, for second-order terms and the sums inside a product.

Values around 1000: against the gradient of fp32 inputs of the same values by the CUDA-core kernels, in 2-norms.  The results'
own rounding is at most half a step, 2^-8; X = phi(q) / den, rounded once for heads above 64, adds as much of dk's terms, which
are about independent and at most three times as large in all as dk (differences of values of one spread: sqrt(2) for each of v and
o), so 4 * 2^-8 there.
"""
import numpy as np
import pytest
import torch

import cross_ref as R
from util import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
U, BU = 2.0 ** -24, 2.0 ** -8
HEADS = [(64, 64), (128, 128), (128, 64), (64, 128), (32, 16), (16, 128)]


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


def gradients(la, q, k, v, do, lengths, kept):
    x = [t.to(DEV) for t in (q, k, v)]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    S, z = la.cross_fwd(*x, lengths=n, return_state=True)[1:] if kept else (None, None)
    return [to_np(t) for t in la.cross_bwd(*x, do.to(DEV), lengths=n, S=S, z=z)]


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("Dk,Dv", HEADS)
@pytest.mark.parametrize("B,H,Hk,N,M,lengths", [(5, 2, 2, 341, 1, None), (1, 4, 2, 130, 1, None), (4, 4, 2, 70, 200, [1, 200, 0, 1])])
def test_one_key(la, B, H, Hk, N, M, lengths, Dk, Dv, kept):
    """The residue where one key counts and takes all the weight."""
    q, k, v, do = R.make(B, H, Hk, N, M, Dk, Dv, BF16, seed=Dk + Dv, lengths=lengths)
    got = gradients(la, q, k, v, do, lengths, kept)
    ref, mag = R.bwd(q, k, v, do, lengths)
    plain = gradients(la, *(t.float() for t in (q, k, v, do)), lengths, kept)
    for b in range(B):
        if lengths is not None and lengths[b] != 1:
            continue
        for what, i, part in (("dq", 0, 10 * U), ("dk", 1, 116 * U)):
            g, m = got[i][b], mag[i][b]
            assert (np.abs(ref[i][b]) <= 1e-15 * m).all()
            assert (np.abs(g) <= part * m).all(), "%s: %.1f of its bound" % (what, np.nanmax(np.abs(g) / np.maximum(part * m, 1e-300)))
            assert np.linalg.norm(g) <= 2 * np.linalg.norm(plain[i][b]), (what, np.linalg.norm(g), np.linalg.norm(plain[i][b]))


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("Dk,Dv", HEADS[:4])
@pytest.mark.parametrize("B,H,Hk,N,M,lengths", [(1, 2, 2, 200, 300, None), (2, 4, 2, 129, 700, [700, 65]), (20, 16, 16, 64, 64, None)])
def test_offset_values(la, B, H, Hk, N, M, lengths, Dk, Dv, kept):
    """Values of 1000 and a spread of some units (bf16 has steps of 4 and 8 there)."""
    q, k, v, do = R.make(B, H, Hk, N, M, Dk, Dv, BF16, seed=Dk + Dv, lengths=lengths)
    v = (1000 + 4 * v.float()).to(BF16)
    got = gradients(la, q, k, v, do, lengths, kept)
    ref = R.bwd(q, k, v, do, lengths)[0]
    plain = gradients(la, *(t.float() for t in (q, k, v, do)), lengths, kept)
    for what, i, part in (("dq", 0, BU), ("dk", 1, (4 if Dk > 64 else 1) * BU), ("dv", 2, 3 * BU)):
        own, off = np.linalg.norm(plain[i] - ref[i]), np.linalg.norm(got[i] - ref[i])
        assert off <= part * np.linalg.norm(ref[i]) + 2 * own, "%s: %.2e off, fp32 %.2e" % (what, off / np.linalg.norm(ref[i]), own / np.linalg.norm(ref[i]))


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_grow_along_the_keys(la, D):
    """Many keys whose values are in order: their mean, which is taken out of S, is that of all of them.  What is left of S is two
    bf16 parts, 2^-16 of it at most; dq is of the order of 1 / sqrt(M) of S without its mean, so 2^-16 * sqrt(131072) = 2^-7.5 in the worst case and a
    small part of that over the independent roundings of a row; half a step of dq itself bounds both."""
    q, k, v, do = R.make(1, 1, 1, 64, 131072, D, D, BF16, seed=D)
    v = v.sort(2)[0]
    ref = R.bwd(q, k, v, do)[0][0]
    for kept in (False, True):
        dq = gradients(la, q, k, v, do, None, kept)[0]
        assert np.linalg.norm(dq - ref) <= BU * np.linalg.norm(ref), np.linalg.norm(dq - ref) / np.linalg.norm(ref)

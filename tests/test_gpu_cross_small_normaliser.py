"""Cross attention where phi(q) . z is at the end of fp32's range: below the normal numbers a query counts as one that no key answers,
in outputs and gradients, and spoils nothing of its head; just above, results are those of fp64.

Bounds of the second: terms phi(q) z and phi(q) S of about 2^-121 and products of them with v are normal numbers, so roundings are relative as
anywhere: those of the parity tests, (M + G N + 2 (Dk + Dv) + 64) u, and in bf16 2^-8 for each operand and result that is rounded,
four at most.
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
SHAPES = [(F32, 5, 4, 16, 16), (F32, 70, 90, 32, 64), (BF16, 5, 4, 64, 64), (BF16, 140, 70, 128, 128), (BF16, 40, 70, 16, 128)]


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


def run(la, q, k, v, do):
    x = [t.to(DEV) for t in (q, k, v)]
    o, S, z = la.cross_fwd(*x, return_state=True)
    return [o, la.cross_apply(x[0], S, z), *la.cross_bwd(*x, do.to(DEV)), *la.cross_bwd(*x, do.to(DEV), S=S, z=z)[:1]]


@pytest.mark.parametrize("dtype,N,M,Dk,Dv", SHAPES)
@pytest.mark.parametrize("sum_of_both", [-98.0, -95.0, -93.0])
def test_subnormal_normaliser(la, dtype, N, M, Dk, Dv, sum_of_both):
    """Two queries so negative, among ordinary ones, to keys at -30."""
    q, _, v, do = R.make(1, 2, 2, N, M, Dk, Dv, dtype, seed=N)
    k = torch.full((1, 2, M, Dk), -30.0, dtype=dtype)
    low = sum_of_both + 30.0 - np.log(M * Dk / 64)  # phi(q) . z = 64 exp(sum_of_both) of both types: 1.8e-41 .. 2.6e-39
    bad = [1, N - 1]
    q[0, 1, bad] = float(low)
    den = np.exp(float(q[0, 1, 1, 0]) - 30.0) * M * Dk
    assert 1e-43 < den < 2.0 ** -128
    got = run(la, q, k, v, do)
    assert all(bool(torch.isfinite(t).all()) for t in got)
    for o in (got[0], got[1], got[2], got[5]):
        assert not o[0, 1, bad].any()
    do[0, 1, bad] = 0  # as if they were not there
    want = run(la, q, k, v, do)
    for i in (3, 4):
        assert torch.equal(got[i], want[i]) and bool(want[i].any())


@pytest.mark.parametrize("dtype,N,M,Dk,Dv", SHAPES)
def test_least_normal_normalisers(la, dtype, N, M, Dk, Dv):
    """Terms of 2^-121 and gradients of thousands: t / den is beyond fp32, dq is not."""
    q, k, v, do = R.make(1, 1, 1, N, M, Dk, Dv, dtype, seed=N)
    q, k = (-48 + q.float() / 8).to(dtype), (-36 + k.float() / 8).to(dtype)
    do = (4096 * do.float()).to(dtype)
    got = run(la, q, k, v, do)
    (ro, _, _, mo), (ref, mag) = R.fwd(q, k, v), R.bwd(q, k, v, do)
    base = (M + N + 2 * (Dk + Dv) + 64) * U + (4 * BU if dtype == BF16 else 0)
    for what, g, r, m in (("o", got[0], ro, mo), ("apply", got[1], ro, mo), ("dq", got[2], ref[0], mag[0]), ("dq", got[5], ref[0], mag[0]), ("dk", got[3], ref[1], mag[1]), ("dv", got[4], ref[2], mag[2])):
        g = to_np(g)
        assert np.isfinite(g).all(), what
        over = np.abs(g - r) / (base * m + (BU if dtype == BF16 else U) * np.abs(r) + 2.0 ** -126)
        assert over.max() <= 1, "%s: %.2f of its bound" % (what, over.max())

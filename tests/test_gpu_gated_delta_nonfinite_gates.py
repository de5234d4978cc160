"""Infinities and NaN among the gates, and anywhere in sequences of several segments: they stay in their head and do not reach
earlier chunks (a g of -inf is an ordinary value: the state starts anew)."""
import pytest
import torch

from test_gpu_gated_delta import make
from test_gpu_gated_delta_segments import segments

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
NAN, INF = float("nan"), float("inf")
# N, Dk, Dv, dtype; the bf16 ones of 1300 and 1500 are cut into segments, forward and gradient
CASES = [(300, 32, 64, F32), (200, 16, 128, BF16), (1300, 64, 64, BF16), (1500, 128, 128, BF16)]


def test_the_long_cases_are_cut():
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    for N, Dk, Dv, dtype in CASES:
        assert N < 1000 or all(segments(la, bwd, 3, N, Dk, Dv) > 2 for bwd in (False, True))


@pytest.mark.gpu
@pytest.mark.parametrize("which,bad", [(0, NAN), (1, INF), (2, NAN), (3, NAN), (3, INF), (4, NAN), (4, INF)])
@pytest.mark.parametrize("N,Dk,Dv,dtype", CASES)
def test_spread(N, Dk, Dv, dtype, which, bad):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    ins = [t.to(DEV) for t in make(4, 1, 3, N, Dk, Dv, dtype)]
    o, S = la.gated_delta_fwd(*ins[:5], return_state=True)
    grads = la.gated_delta_bwd(*ins)
    at = N // 2 + 3
    first = at // 64 * 64  # of its chunk
    ins[which][0, 1, at] = bad
    o2, S2 = la.gated_delta_fwd(*ins[:5], return_state=True)
    assert torch.equal(o2[:, ::2], o[:, ::2]) and torch.equal(S2[:, ::2], S[:, ::2])
    assert torch.equal(o2[:, 1, :first], o[:, 1, :first])
    assert not torch.isfinite(o2[:, 1, at].float()).all()
    if which:  # a query leaves the state alone
        assert not torch.isfinite(o2[:, 1, at + 1].float()).all() and not torch.isfinite(S2[:, 1]).all()
    assert all(torch.equal(a[:, ::2], b[:, ::2]) for a, b in zip(la.gated_delta_bwd(*ins), grads))
    assert la.last_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_non_finite_state(dtype):
    """A NaN in S0 or dS stays in its head and its value column."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    N, D = 1300, 64
    ins = [t.to(DEV) for t in make(5, 1, 3, N, D, D, dtype)]
    S0, dS = (torch.randn(1, 3, D, D, device=DEV) for _ in range(2))
    o, S = la.gated_delta_fwd(*ins[:5], S0=S0, return_state=True)
    grads = la.gated_delta_bwd(*ins, S0=S0, dS=dS, return_dS0=True)
    S0[0, 1, 7, 20] = NAN
    o2, S2 = la.gated_delta_fwd(*ins[:5], S0=S0, return_state=True)
    rest = [c for c in range(D) if c != 20]
    assert torch.equal(o2[:, ::2], o[:, ::2]) and torch.equal(S2[:, ::2], S[:, ::2])
    assert torch.equal(o2[..., rest], o[..., rest]) and torch.equal(S2[..., rest], S[..., rest])
    assert not torch.isfinite(o2[:, 1, 0, 20].float()).any()
    assert all(torch.equal(a[:, ::2], b[:, ::2])
               for a, b in zip(la.gated_delta_bwd(*ins, S0=S0, dS=dS, return_dS0=True), grads))
    assert la.last_error() == 0

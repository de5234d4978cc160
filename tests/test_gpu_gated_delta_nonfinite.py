"""Infinities and NaN in the gated delta rule's inputs stay in their head and do not reach earlier chunks."""
import pytest
import torch

from test_gpu_gated_delta import make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("which", [0, 1, 2, 4])
@pytest.mark.parametrize("N,Dk,Dv,dtype", [(300, 32, 64, F32), (500, 64, 64, BF16), (700, 128, 128, BF16),
                                           (200, 16, 128, BF16)])
def test_spread(N, Dk, Dv, dtype, which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    ins = [t.to(DEV) for t in make(4, 1, 3, N, Dk, Dv, dtype)]
    o, S = la.gated_delta_fwd(*ins[:5], return_state=True)
    grads = la.gated_delta_bwd(*ins)
    for bad in (float("nan"), float("inf")):
        spoilt = [t.clone() for t in ins]
        spoilt[which][0, 1, 130] = bad  # in the third chunk of the second head
        o2, S2 = la.gated_delta_fwd(*spoilt[:5], return_state=True)
        assert torch.equal(o2[:, ::2], o[:, ::2]) and torch.equal(S2[:, ::2], S[:, ::2])
        assert torch.equal(o2[:, 1, :128], o[:, 1, :128])
        assert not torch.isfinite(o2[:, 1, 130].float()).all()
        assert all(torch.equal(a[:, ::2], b[:, ::2]) for a, b in zip(la.gated_delta_bwd(*spoilt), grads))
    assert la.last_error() == 0

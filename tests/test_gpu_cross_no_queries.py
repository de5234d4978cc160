"""Cross attention without heads of queries: the keys' state is formed and their gradients are 0, as with heads of no queries."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


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


@pytest.mark.parametrize("dtype,M", [(torch.float32, 40), (torch.float32, 200), (torch.bfloat16, 200)])
def test_no_heads_of_queries(la, dtype, M):
    r = lambda *s: torch.randn(*s, device=DEV).to(dtype)
    k, v, q, do = r(2, 3, M, 64), r(2, 3, M, 32), r(2, 0, 5, 64), r(2, 0, 5, 32)
    n = torch.tensor([M, 7], dtype=torch.int32, device=DEV)
    _, wS, wz = la.cross_fwd(r(2, 3, 0, 64), k, v, lengths=n, return_state=True)
    S, z = torch.full((2, 3, 64, 32), float("nan"), device=DEV), torch.full((2, 3, 64), float("nan"), device=DEV)
    s = la.CrossShape(2, 0, 3, 5, M, 64, 32, 0 if dtype == torch.float32 else 1)
    need = la.cross_workspace_bytes(la.OP_CROSS_FWD, 2, 0, 3, 5, M, 64, 32, dtype)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    status = la.library().la_cross_fwd(None, p(k), p(v), p(n), None, p(S), p(z), s, p(ws) if need else None, need,
                                       ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0 and torch.equal(S, wS) and torch.equal(z, wz)
    o, S, z = la.cross_fwd(q, k, v, lengths=n, return_state=True)
    assert o.shape == (2, 0, 5, 32) and torch.equal(S, wS) and torch.equal(z, wz)
    assert la.cross_apply(q, S, z).shape == (2, 0, 5, 32)
    dk, dv = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    dq = la.cross_bwd(q, k, v, do, lengths=n, dk=dk, dv=dv)[0]
    assert dq.shape == q.shape and not dk.any() and not dv.any()
    no_keys = la.cross_fwd(q, k[:, :, :0].contiguous(), v[:, :, :0].contiguous(), return_state=True)
    assert not no_keys[1].any() and not no_keys[2].any()

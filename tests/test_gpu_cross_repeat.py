"""Cross attention many times over, back to back, where its kernels' warps may run furthest apart: no wait may run out, and
every call has to give the first one's bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


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


# B, H, Hk, N, M, Dk, Dv, calls: long heads (rings run ahead), heads of one chunk and of two (a group has none of many heads)
CASES = [(2, 16, 16, 32768, 32768, 64, 64, 60), (2, 16, 8, 8192, 16384, 128, 128, 60), (2, 16, 16, 8192, 8192, 128, 64, 60),
         (2, 16, 16, 8192, 8192, 64, 128, 60), (64, 32, 32, 128, 128, 64, 64, 100), (64, 32, 32, 100, 60, 128, 128, 100),
         (64, 32, 32, 200, 129, 64, 64, 100), (64, 32, 16, 64, 200, 128, 64, 100)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:7])))
def test_repeated(la, case):
    B, H, Hk, N, M, Dk, Dv, calls = case
    r = lambda *s: torch.empty(s, dtype=BF16, device=DEV).normal_()
    q, k, v, do = r(B, H, N, Dk), r(B, Hk, M, Dk), r(B, Hk, M, Dv), r(B, H, N, Dv)
    o, S, z = la.cross_fwd(q, k, v, return_state=True)
    exact = la.cross_apply(q, S, z)
    grads = la.cross_bwd(q, k, v, do, S=S, z=z)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(calls):
        got = (la.cross_fwd(q, k, v), la.cross_apply(q, S, z), *la.cross_bwd(q, k, v, do, S=S, z=z))
        for a, b in zip(got, (o, exact, *grads)):
            differ += (a.view(torch.int16) != b.view(torch.int16)).sum()
    assert int(differ) == 0 and la.last_error() == 0

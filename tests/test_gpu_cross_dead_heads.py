"""Batch entries without keys: their queries get 0 and have a gradient of 0, whatever the queries and the upstream gradient hold
there, and the other entries are as they were, bit for bit."""
import pytest
import torch

import cross_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


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


# N, M, Dk, Dv, dtype: one chunk to a head, several, few and many queries
CASES = [(17, 60, 16, 32, F32), (5, 200, 64, 64, F32), (100, 200, 128, 128, F32), (20, 60, 64, 64, BF16), (300, 300, 128, 128, BF16),
         (130, 140, 64, 128, BF16), (1, 30, 128, 64, BF16), (1, 30, 32, 16, F32)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_entries_without_keys(la, case, bad):
    N, M, Dk, Dv, dtype = case
    q, k, v, do = (t.to(DEV) for t in R.make(4, 4, 2, N, M, Dk, Dv, dtype, seed=N))
    n = torch.tensor([M, 0, -3, 9], dtype=torch.int32, device=DEV)

    def everything():
        o, S, z = la.cross_fwd(q, k, v, lengths=n, return_state=True)
        return (o, la.cross_apply(q, S, z), la.cross_apply(q[:, :, 0].contiguous(), S, z), *la.cross_bwd(q, k, v, do, lengths=n),
                *la.cross_bwd(q, k, v, do, lengths=n, S=S, z=z), S, z)

    clean = everything()
    for t in (q, k, v, do):
        t[1:3] = bad
    got = everything()
    for i, (a, b) in enumerate(zip(got, clean)):
        assert not b[1:3].any() and torch.equal(a, b), i

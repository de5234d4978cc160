"""The gated delta rule's and layer norm's C entry points called as a C program would, and with the buffers that la.h lets
be one: S with S0, dS0 with dS, and the norm's dx with dy or x.  The same bits as from separate buffers."""
import pytest
import torch

from test_gpu_gated_delta import make
from test_gpu_layer_norm import make as make_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
# one chunk; several; value columns in several slices; several segments
CASES = [(1, 2, 40, 16, 32, F32), (2, 2, 200, 64, 128, F32), (1, 40, 130, 128, 128, F32), (1, 2, 40, 64, 64, BF16),
         (2, 2, 200, 32, 128, BF16), (1, 2, 1300, 64, 64, BF16), (1, 2, 1500, 128, 128, BF16)]


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


def case(la, B, H, N, Dk, Dv, dtype):
    ins = [t.to(DEV) for t in make(N, B, H, N, Dk, Dv, dtype)]
    gen = torch.Generator().manual_seed(N)
    S0, dS = (torch.randn(B, H, Dk, Dv, generator=gen).to(DEV) for _ in range(2))
    nb = la.workspace_bytes(la.OP_GATED_DELTA_BWD, B, H, N, Dk, Dv, dtype)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN wherever it is read before it is written
    return ins, S0, dS, la.Shape(B, H, N, Dk, Dv, la.LA_F32 if dtype == F32 else la.LA_BF16), ws


def ptrs(*ts):
    return [None if t is None else t.data_ptr() for t in ts]


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("B,H,N,Dk,Dv,dtype", CASES)
def test_gradient_entry(la, B, H, N, Dk, Dv, dtype):
    """la_gated_delta_bwd: the gradient of whole sequences."""
    (q, k, v, g, beta, do), _, _, s, ws = case(la, B, H, N, Dk, Dv, dtype)
    want = la.gated_delta_bwd(q, k, v, g, beta, do)
    outs = [torch.full_like(t, float("nan")) for t in (q, k, v, g, beta)]
    st = la.library().la_gated_delta_bwd(*ptrs(q, k, v, g, beta, do, *outs), s, ws.data_ptr(), ws.numel(), stream())
    assert st == 0, la.library().la_error_detail()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("B,H,N,Dk,Dv,dtype", CASES)
def test_states_in_one_buffer(la, B, H, N, Dk, Dv, dtype):
    (q, k, v, g, beta, do), S0, dS, s, ws = case(la, B, H, N, Dk, Dv, dtype)
    o, S = la.gated_delta_fwd(q, k, v, g, beta, S0=S0, return_state=True)
    o2, both = torch.empty_like(o), S0.clone()
    st = la.library().la_gated_delta_fwd(*ptrs(q, k, v, g, beta, both, o2, both), s, ws.data_ptr(), ws.numel(), stream())
    assert st == 0, la.library().la_error_detail()
    assert torch.equal(o2, o) and torch.equal(both, S)
    want = la.gated_delta_bwd(q, k, v, g, beta, do, S0=S0, dS=dS, return_dS0=True)
    outs, both = [torch.empty_like(t) for t in (q, k, v, g, beta)], dS.clone()
    ws.fill_(0xFF)
    st = la.library().la_gated_delta_bwd_with_state(*ptrs(q, k, v, g, beta, S0, do, both, *outs, both), s, ws.data_ptr(),
                                                    ws.numel(), stream())
    assert st == 0, la.library().la_error_detail()
    assert all(torch.equal(a, b) for a, b in zip([*outs, both], want))


@pytest.mark.parametrize("shape,dtype", [((5, 7), BF16), ((1000, 33), BF16), ((700, 128), F32), ((300, 2047), BF16),
                                         ((40, 2048), BF16), ((300, 5121), F32), ((60, 8192), BF16), ((20, 16384), F32)])
def test_norm_gradient_in_place(la, shape, dtype):
    x, w, b, dy = (t.to(DEV) for t in make_norm(shape, dtype, 4))
    _, mean, rstd = la.layer_norm_fwd(x, w, b, return_stats=True)
    want = la.layer_norm_bwd(x, w, mean, rstd, dy)
    for name in ("x", "dy"):
        ins = dict(x=x.clone(), dy=dy.clone())
        got = la.layer_norm_bwd(ins["x"], w, mean, rstd, ins["dy"], dx=ins[name])
        assert all(torch.equal(a, c) for a, c in zip(got, want)), name

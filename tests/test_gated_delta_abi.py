"""The gated delta rule's and layer norm's entry points on the CPU: sizes, workspaces and what is
refused before a GPU is touched."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def la():
    from causal_linear_attention_phi_gb300 import build
    build.build_library()
    import causal_linear_attention_phi_gb300 as la
    la.library()
    return la


NULL = ctypes.c_void_p(0)


@pytest.mark.parametrize("shape,want", [((-1, 1, 8, 16, 16, 0), 1), ((1, 1, 8, 16, 16, 5), 1),
                                        ((1, 1, 8, 0, 16, 0), 1), ((1, 1, 8, 48, 16, 0), 2),
                                        ((1, 1, 8, 16, 256, 1), 2), ((256, 256, 8, 16, 16, 0), 2),
                                        ((0, 4, 8, 16, 16, 1), 0), ((1, 1, 0, 16, 16, 0), 0)])
def test_gated_delta_shapes(la, shape, want):
    lib, s = la.library(), la.Shape(*shape)
    assert lib.la_gated_delta_fwd(*[NULL] * 8, s, NULL, 0, None) == want
    assert lib.la_gated_delta_bwd(*[NULL] * 11, s, NULL, 0, None) == want
    if shape[2] == 8:  # a step ignores N
        assert lib.la_gated_delta_step(*[NULL] * 7, s, None) == want


def test_gated_delta_workspace(la):
    f, b = la.OP_GATED_DELTA_FWD, la.OP_GATED_DELTA_BWD
    for dt in (torch.float32, torch.bfloat16):
        for D in (16, 64, 128):
            one = la.workspace_bytes(f, 1, 2, 64, D, D, dt)
            assert one > 0 and one == la.workspace_bytes(f, 1, 2, 1, D, D, dt)
            # linear in the chunks of 64 positions
            grow = [la.workspace_bytes(b, 1, 2, 64 * m, D, D, dt) for m in (300, 400, 500)]
            assert grow[0] > one and 0 < grow[2] - grow[1] <= 1.1 * (grow[1] - grow[0]) + (1 << 20)
    assert la.workspace_bytes(f, 1, 2, 0, 16, 16, torch.float32) == 0
    assert la.workspace_bytes(b, 1, 2, 64, 48, 16, torch.float32) == 0


@pytest.mark.parametrize("rows,C,dtype,want", [(-1, 8, 0, 1), (4, 0, 0, 1), (4, 8, 3, 1), (4, 16385, 1, 2),
                                               (1 << 40, 8, 0, 1), (0, 8, 1, 0)])
def test_norm_shapes(la, rows, C, dtype, want):
    lib, s = la.library(), la.NormShape(rows, C, dtype)
    assert lib.la_layer_norm_fwd(*[NULL] * 6, s, 1e-5, None) == want
    assert lib.la_layer_norm_bwd(*[NULL] * 8, s, NULL, 0, None) == want
    assert lib.la_layer_norm_workspace_bytes(s) == 0


def test_norm_eps_and_workspace(la):
    lib = la.library()
    s = la.NormShape(4, 8, 0)
    for eps in (-1e-5, float("nan")):
        assert lib.la_layer_norm_fwd(*[NULL] * 6, s, eps, None) == 1
    one = la.layer_norm_workspace_bytes(1, 128, torch.float32)
    assert 0 < one <= la.layer_norm_workspace_bytes(1 << 20, 128, torch.float32) < 1 << 24
    with pytest.raises(TypeError):
        la.layer_norm_workspace_bytes(1, 128, torch.float64)


def test_python_refusals_on_host_tensors(la):
    q, v, g, S = torch.zeros(1, 1, 4, 16), torch.zeros(1, 1, 4, 16), torch.zeros(1, 1, 4), torch.zeros(1, 1, 16, 16)
    with pytest.raises(TypeError):
        la.gated_delta_fwd(q, q, v, g, g)
    with pytest.raises(TypeError):
        la.gated_delta_bwd(q, q, v, g, g, v)
    with pytest.raises(TypeError):
        la.gated_delta_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[..., 0], g[..., 0], S)
    with pytest.raises(TypeError):
        la.layer_norm_fwd(q)
    with pytest.raises(TypeError):
        la.layer_norm_bwd(q, None, g, g, q)

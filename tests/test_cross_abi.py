"""Cross attention's C entry points on the CPU: refusals before any device call, and the workspace query."""
import ctypes

import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def la():
    from causal_linear_attention_phi_gb300 import build
    build.build_library()
    import causal_linear_attention_phi_gb300 as la
    la.library()
    return la


def calls(la):
    lib, p = la.library(), ctypes.c_void_p(0)
    fwd = lambda *s: lib.la_cross_fwd(*[p] * 7, la.CrossShape(*s), p, 0, None)
    bwd = lambda *s: lib.la_cross_bwd(*[p] * 10, la.CrossShape(*s), p, 0, None)
    app = lambda *s: lib.la_cross_apply(*[p] * 4, la.CrossShape(*s), p, 0, None)
    return fwd, bwd, app


def test_shapes_refused_on_the_host(la):
    for f in calls(la):
        assert f(-1, 1, 1, 4, 4, 16, 16, 0) == 1
        assert f(1, 2, -1, 4, 4, 16, 16, 0) == 1
        assert f(1, 1, 1, 4, 4, 16, 16, 5) == 1          # dtype
        assert f(1, 1, 1, 4, 4, 48, 16, 0) == 2          # head size
        assert f(1, 1, 1, 4, 4, 16, 256, 1) == 2
        assert f(1, 4, 3, 4, 4, 16, 16, 0) == 1          # 3 heads of keys do not divide 4
        assert f(1, 4, 0, 4, 4, 16, 16, 0) == 1
        assert f(256, 256, 1, 4, 4, 16, 16, 0) == 2      # B*H
        assert f(1, 4, 1, 1 << 29, 4, 16, 16, 0) == 2    # rows of queries to a head of keys
        assert f(0, 4, 2, 4, 4, 16, 16, 0) == 0          # nothing to do
        assert f(3, 0, 0, 4, 4, 16, 16, 1) == 0
    fwd, bwd, app = calls(la)
    assert fwd(1, 2, 2, 0, 9, 16, 16, 0) == 0 and bwd(1, 2, 2, 0, 0, 16, 16, 0) == 0 and app(1, 2, 2, 0, 0, 16, 16, 0) == 0
    assert fwd(1, 1, 1, 4, -4, 16, 16, 0) == 1 and bwd(1, 1, 1, 4, -4, 16, 16, 0) == 1


def test_workspace_query(la):
    for dt in (F32, BF16):
        need = [la.cross_workspace_bytes(op, 2, 8, 4, 300, 1000, 64, 128, dt) for op in (la.OP_CROSS_FWD, la.OP_CROSS_BWD)]
        assert 0 < need[0] < need[1]
        assert la.cross_workspace_bytes(la.OP_CROSS_FWD, 2, 8, 4, 300, 0, 64, 128, dt) == 0   # no key: nothing summed
        assert la.cross_workspace_bytes(la.OP_CROSS_BWD, 2, 8, 4, 0, 1000, 64, 128, dt) == 0
        assert la.cross_workspace_bytes(la.OP_CROSS_APPLY, 2, 8, 4, 1, 0, 64, 128, dt) == 0   # single tokens need none
        assert la.cross_workspace_bytes(la.OP_CROSS_FWD, 2, 8, 3, 300, 1000, 64, 128, dt) == 0
        assert la.cross_workspace_bytes(la.OP_CAUSAL_FWD, 2, 8, 4, 300, 1000, 64, 128, dt) == 0
    assert la.workspace_bytes(la.OP_CROSS_FWD, 2, 8, 300, 64, 128, F32) == 0  # not an op of that query
    with pytest.raises(TypeError):
        la.cross_workspace_bytes(la.OP_CROSS_FWD, 1, 1, 1, 1, 1, 16, 16, torch.float16)


def test_binding_refuses_host_tensors(la):
    t = torch.zeros(1, 2, 4, 16)
    with pytest.raises(TypeError):
        la.cross_fwd(t, t, t)
    with pytest.raises(TypeError):
        la.cross_bwd(t, t, t, t)
    with pytest.raises(TypeError):
        la.cross_apply(t, torch.zeros(1, 2, 16, 16), torch.zeros(1, 2, 16))

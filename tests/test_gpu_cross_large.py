"""Cross attention and the norms around a block where offsets pass 2^31 elements: the last rows against the same rows alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
ROWS = (1 << 24) + (1 << 20) + 77  # of 128: 2.28e9 elements, 4.6 GB in bf16


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available() or torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB on the device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    la.library()
    la.clear_error()
    yield la
    assert la.last_error() == 0
    torch.cuda.empty_cache()


def rand(*s, dtype=BF16):
    return torch.empty(s, dtype=dtype, device=DEV).normal_()


def test_queries(la):
    q, k, v = rand(1, 1, ROWS, 128), rand(1, 1, 300, 128), rand(1, 1, 300, 128)
    do = rand(1, 1, ROWS, 128)
    o, S, z = la.cross_fwd(q, k, v, return_state=True)
    dq, dk, dv = la.cross_bwd(q, k, v, do, S=S, z=z)
    for rows in (slice(ROWS - 200, ROWS), slice(1 << 24, (1 << 24) + 130)):
        part, dpart = q[:, :, rows].contiguous(), do[:, :, rows].contiguous()
        assert torch.equal(la.cross_fwd(part, k, v), o[:, :, rows])
        assert torch.equal(la.cross_bwd(part, k, v, dpart, S=S, z=z)[0], dq[:, :, rows])
    assert bool(torch.isfinite(dk).all()) and bool(torch.isfinite(dv).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_keys(la, dtype):
    q, k, v, do = rand(1, 1, 300, 128, dtype=dtype), rand(1, 1, ROWS, 128, dtype=dtype), rand(1, 1, ROWS, 128, dtype=dtype), rand(1, 1, 300, 128, dtype=dtype)
    n = torch.tensor([ROWS - 40], dtype=torch.int32, device=DEV)
    o, S, z = la.cross_fwd(q, k, v, lengths=n, return_state=True)
    # the state is the sum of the halves' states: 2^25 terms of one order, partial sums in fp32 of two lengths
    half = 1 << 23
    parts = [la.cross_fwd(q, k[:, :, a:b].contiguous(), v[:, :, a:b].contiguous(), return_state=True)[1:] for a, b in ((0, half), (half, ROWS - 40))]
    # z: every term counts the same way, at most ROWS / (64 * 152) additions to a record in fp32: 1e-4 of it is 1700 roundings
    assert float(((parts[0][1].double() + parts[1][1].double()) / z.double() - 1).abs().max()) <= 1e-4
    dq, dk, dv = la.cross_bwd(q, k, v, do, lengths=n, S=S, z=z)
    assert not dk[:, :, ROWS - 40:].any() and not dv[:, :, ROWS - 40:].any()
    rows = slice(ROWS - 400, ROWS - 40)
    _, pk, pv = la.cross_bwd(q, k[:, :, rows].contiguous(), v[:, :, rows].contiguous(), do, S=S, z=z)
    assert torch.equal(pk, dk[:, :, rows]) and torch.equal(pv, dv[:, :, rows])


def test_norms(la):
    o, gate, dy = rand(1, 2, ROWS // 2, 128), rand(1, ROWS // 2, 256), rand(1, ROWS // 2, 256)
    y = la.gated_norm_fwd(o, gate, rms=True)
    do, dg, _ = la.gated_norm_bwd(o, gate, None, dy, rms=True)
    rows = slice(ROWS // 2 - 50, ROWS // 2)
    po, pg, pd = o[:, :, rows].contiguous(), gate[:, rows].contiguous(), dy[:, rows].contiguous()
    assert torch.equal(la.gated_norm_fwd(po, pg, rms=True), y[:, rows])
    ref = la.gated_norm_bwd(po, pg, None, pd, rms=True)
    assert torch.equal(ref[0], do[:, :, rows]) and torch.equal(ref[1], dg[:, rows])
    del o, gate, y, do, dg
    for C in (128, 127):
        x, a = rand(ROWS, C), rand(ROWS, C)
        h, t, mean, rstd = la.residual_norm_fwd(x, a, return_stats=True)
        dx = la.residual_norm_bwd(h, None, None, None, mean, rstd, x)[0]
        rows = slice(ROWS - 50, ROWS)
        ph, pt, pm, pr = la.residual_norm_fwd(x[rows].clone(), a[rows].clone(), return_stats=True)
        assert torch.equal(ph, h[rows]) and torch.equal(pt, t[rows]) and torch.equal(pm, mean[rows])
        assert torch.equal(la.residual_norm_bwd(ph, None, None, None, pm, pr, x[rows].clone())[0], dx[rows])
        del x, a, h, t, dx

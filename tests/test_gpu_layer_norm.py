"""GPU parity of layer norm, forward and gradient, against fp64.

Bounds (error over the largest magnitude of the row, or of the output for the sums over rows):
an fp32 row of C elements is summed in at most 16 + 10 additions along any path and passes a
handful of products: 64 * 2^-24, scaled by max|x| * rstd where the mean is taken off large values; bf16 outputs
add half a step, 2^-8.  Sums over rows: at most rows additions of half a step, relative to the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import delta_ref as R
from util import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
STEP = {F32: 64 * 2.0 ** -24, BF16: 2.0 ** -8 + 64 * 2.0 ** -24}


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    la.library()
    return la


def row_err(x, ref):
    x, ref = to_np(x), np.asarray(ref)
    top = np.abs(ref).max(-1, keepdims=True)
    return float((np.abs(x - ref) / np.where(top > 0, top, 1)).max())


CASES = [((1, 1), F32), ((5, 1), BF16), ((3, 2), F32), ((7, 7), BF16), ((33, 8), F32), ((65, 16), BF16),
         ((2, 3, 50, 64), BF16), ((1, 4, 33, 128), F32), ((1000, 128), BF16), ((9, 129), F32), ((64, 256), F32),
         ((31, 255), BF16), ((17, 513), F32), ((40, 512), BF16), ((5, 1000), BF16), ((300, 1024), F32),
         ((700, 2048), BF16), ((3, 2047), BF16), ((5, 4096), F32), ((6, 8192), BF16), ((2, 8193), BF16),
         ((3, 16384), BF16), ((2, 16383), F32), ((2, 16384), F32)]


def make(shape, dtype, seed, offset=0.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * 1.5 + offset
    w = 1 + 0.2 * torch.randn(shape[-1], generator=gen)
    b = 0.3 * torch.randn(shape[-1], generator=gen)
    return x.to(dtype), w.to(dtype), b.to(dtype), torch.randn(shape, generator=gen).to(dtype)


@pytest.mark.parametrize("shape,dtype", CASES)
def test_fwd(la, shape, dtype):
    x, w, b, _ = make(shape, dtype, shape[-1])
    y, mean, rstd = la.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), return_stats=True)
    ry, rm, rr = R.norm_fwd(x, w, b)
    assert y.dtype == dtype and mean.dtype == F32 and mean.shape == x.shape[:-1]
    assert np.abs(to_np(mean) - rm).max() <= 64 * 2.0 ** -24 * np.abs(to_np(x)).max()
    if shape[-1] > 1:  # with one element the variance is 0 and rstd is that of eps alone
        assert np.abs(to_np(rstd) / rr - 1).max() <= 64 * 2.0 ** -24 * max(1.0, (np.abs(to_np(x)).max(-1) * rr).max())
    lift = max(1.0, (np.abs(to_np(x)).max(-1) * rr).max() / 4) if shape[-1] > 1 else 1.0
    assert row_err(y, ry) <= STEP[dtype] * (lift if dtype == F32 else 1)
    plain = la.layer_norm_fwd(x.to(DEV))
    assert row_err(plain, R.norm_fwd(x)[0]) <= STEP[dtype] * (lift if dtype == F32 else 1)
    inplace = x.to(DEV)
    assert torch.equal(la.layer_norm_fwd(inplace, w.to(DEV), b.to(DEV), out=inplace), y)


@pytest.mark.parametrize("shape,dtype", CASES)
def test_bwd(la, shape, dtype):
    x, w, b, dy = make(shape, dtype, shape[-1] + 1)
    xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
    _, mean, rstd = la.layer_norm_fwd(xd, wd, b.to(DEV), return_stats=True)
    dx, dw, db = la.layer_norm_bwd(xd, wd, mean, rstd, dyd)
    rx, rw, rb = R.norm_bwd(x, w, dy)
    assert dx.dtype == dw.dtype == db.dtype == dtype
    if shape[-1] > 2:
        assert row_err(dx, rx) <= 4 * STEP[F32] * 8 + (STEP[BF16] if dtype == BF16 else 0)
    else:  # one element has no gradient; of two, it cancels to eps' share
        assert np.abs(to_np(dx) - rx).max() <= 1e-4 * max(1.0, float(rstd.max())) + (2.0 ** -8 * np.abs(rx).max())
    rows = int(np.prod(shape[:-1]))
    axes = tuple(range(len(shape) - 1))
    h = R.norm_fwd(x)[0]
    half = 2.0 ** -8 if dtype == BF16 else 0.0
    step = 2.0 ** -24 * min(rows + 64, 4096)
    big = 64 * 2.0 ** -24 * max(1.0, float((np.abs(to_np(x)).max(-1) * to_np(rstd)).max()))
    for got, ref, mag in ((dw, rw, np.abs(to_np(dy) * h).sum(axes) + big * np.abs(to_np(dy)).sum(axes) / step),
                          (db, rb, np.abs(to_np(dy)).sum(axes))):
        assert (np.abs(to_np(got) - ref) <= half * np.abs(ref) + step * mag + 1e-30).all()
    dx2, dw2, db2 = la.layer_norm_bwd(xd, None, mean, rstd, dyd)
    assert dw2 is None and db2 is None
    if shape[-1] > 2:
        assert row_err(dx2, R.norm_bwd(x, None, dy)[0]) <= 4 * STEP[F32] * 8 + (STEP[BF16] if dtype == BF16 else 0)
    again = la.layer_norm_bwd(xd, wd, mean, rstd, dyd)
    assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), again))


def test_many_rows_and_large_means(la):
    """More rows than one pass of the grid holds, and rows whose mean is 1000 times their spread."""
    x, w, b, dy = make((200003, 24), BF16, 5)
    xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
    y, mean, rstd = la.layer_norm_fwd(xd, wd, b.to(DEV), return_stats=True)
    assert row_err(y, R.norm_fwd(x, w, b)[0]) <= STEP[BF16]
    _, dw, db = la.layer_norm_bwd(xd, wd, mean, rstd, dyd)
    _, rw, rb = R.norm_bwd(x, w, dy)
    for got, ref in ((dw, rw), (db, rb)):
        # sums of 2e5 terms of size 1: walks of length sqrt(2e5), each addition off by half a step
        assert (np.abs(to_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -24 * 4096 * 450).all()
    x, w, b, _ = make((50, 640), F32, 6, offset=1500.0)
    y = la.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV))
    assert row_err(y, R.norm_fwd(x, w, b)[0]) <= 64 * 2.0 ** -24 * 1000


def test_zero_rows_graph_and_refusals(la):
    x, w, b, dy = (t.to(DEV) for t in make((12, 64), BF16, 7))
    none = x[:0]
    y, mean, rstd = la.layer_norm_fwd(none, w, b, return_stats=True)
    assert y.shape == none.shape and mean.numel() == 0
    dx, dw, db = la.layer_norm_bwd(none, w, mean, rstd, none)
    assert dx.numel() == 0 and not dw.any() and not db.any()
    # constant rows: y is the bias
    c = torch.full((3, 64), 2.5, device=DEV, dtype=BF16)
    assert torch.equal(la.layer_norm_fwd(c, w, b), b.expand(3, 64))
    y, mean, rstd = la.layer_norm_fwd(x, w, b, return_stats=True)
    ref = la.layer_norm_bwd(x, w, mean, rstd, dy)
    ws = torch.empty(la.layer_norm_workspace_bytes(12, 64, BF16), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(t) for t in (x, x, w, w)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.layer_norm_fwd(x, w, b, out=outs[0])
        la.layer_norm_bwd(x, w, mean, rstd, dy, *outs[1:], workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], y) and all(torch.equal(a, c) for a, c in zip(outs[1:], ref))
    with pytest.raises(ValueError):
        la.layer_norm_fwd(x, w[:63].contiguous(), b)
    with pytest.raises(ValueError):
        la.layer_norm_fwd(x, w.float(), b)
    with pytest.raises(ValueError):
        la.layer_norm_fwd(x.t(), None, None)
    with pytest.raises(ValueError):
        la.layer_norm_bwd(x, w, mean[:11].contiguous(), rstd, dy)
    with pytest.raises(la.LaError) as e:
        la.layer_norm_fwd(x, w, b, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(la.LaError) as e:
        la.layer_norm_fwd(torch.zeros(1, 16385, device=DEV))
    assert e.value.status == 2
    with pytest.raises(la.LaError) as e:
        la.layer_norm_bwd(x, w, mean, rstd, dy, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 3

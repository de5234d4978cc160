"""Layer norm with a bias alone or no parameters, and gradients that the caller asks for by giving their tensors.

Bounds as in tests/test_gpu_layer_norm.py: a sum over rows takes at most rows + 64 additions along any path, each off by half
a step of the sum of magnitudes, and a bf16 result is off by half its own step."""
import numpy as np
import pytest
import torch

import delta_ref as R
from test_gpu_layer_norm import STEP, make, row_err
from util import to_np

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
    return la


def close_sum(got, ref, terms, rows, dtype):
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    err = np.abs(to_np(got) - ref)
    assert (err <= half * np.abs(ref) + (rows + 64) * 2.0 ** -24 * np.abs(terms).sum(0)).all()


@pytest.mark.parametrize("shape,dtype", [((33, 64), F32), ((70, 512), BF16), ((9, 2047), BF16), ((12, 6000), F32)])
def test_bias_alone(la, shape, dtype):
    x, _, b, dy = make(shape, dtype, 21)
    xd, bd, dyd = (t.to(DEV) for t in (x, b, dy))
    y, mean, rstd = la.layer_norm_fwd(xd, None, bd, return_stats=True)
    assert row_err(y, R.norm_fwd(x, None, b)[0]) <= 2 * STEP[dtype]
    nan = lambda: torch.full_like(bd, float("nan"))
    db = nan()
    dx, none, got = la.layer_norm_bwd(xd, None, mean, rstd, dyd, dbias=db)
    assert none is None and got is db
    close_sum(db, to_np(dy).sum(0), to_np(dy), shape[0], dtype)
    assert torch.equal(dx, la.layer_norm_bwd(xd, None, mean, rstd, dyd)[0])
    # the weight's gradient too, at the weight 1: what a weight of ones gives
    dw, db2 = nan(), nan()
    dx2, got, got2 = la.layer_norm_bwd(xd, None, mean, rstd, dyd, dweight=dw, dbias=db2)
    assert got is dw and got2 is db2 and torch.equal(db, db2) and torch.equal(dx, dx2)
    ones = la.layer_norm_bwd(xd, torch.ones_like(bd), mean, rstd, dyd)
    assert torch.equal(dw, ones[1]) and torch.equal(db, ones[2]) and torch.equal(dx, ones[0])
    only = nan()
    assert la.layer_norm_bwd(xd, None, mean, rstd, dyd, dweight=only)[1:] == (only, None) and torch.equal(only, dw)


def test_nothing_asked_for_and_refusals(la):
    x, w, b, dy = (t.to(DEV) for t in make((12, 64), BF16, 22))
    _, mean, rstd = la.layer_norm_fwd(x, None, None, return_stats=True)
    assert la.layer_norm_bwd(x, None, mean, rstd, dy)[1:] == (None, None)
    for bad in (dict(dbias=b[:63].contiguous()), dict(dweight=w.float()), dict(dbias=b[None]), dict(dweight=w.repeat(2)[::2])):
        with pytest.raises(ValueError):
            la.layer_norm_bwd(x, None, mean, rstd, dy, **bad)
    with pytest.raises(TypeError):
        la.layer_norm_bwd(x, None, mean, rstd, dy, dbias=b.cpu())
    with pytest.raises(la.LaError) as e:
        la.layer_norm_bwd(x, None, mean, rstd, dy, dbias=b, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 3
    none = x[:0]
    db = torch.full_like(b, 7)
    la.layer_norm_bwd(none, None, mean[:0], rstd[:0], none, dbias=db)
    assert not db.any()

"""GPU parity of the gated norm of heads and of the residual norm, forward and gradient, against fp64.

Bounds.  u = 2^-24, b = 2^-8 (half a step of fp32 and of bf16, relative).  A row of C elements is summed along paths of at
most 32 + 10 additions and passes a few tens of products, exponentials (2 u) and reciprocals: 64 u of the row's largest value for
an output, twice that for a gradient, whose rows hold two such sums; `lift` scales it where the mean is taken off large values.
A bf16 output adds half a step of itself.  Sums over rows: paths of at most rows additions, u of the terms' magnitudes each.
"""
import numpy as np
import pytest
import torch

import block_norm_ref as R
from util import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
U, BU = 2.0 ** -24, 2.0 ** -8


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


def step(dtype):
    return BU if dtype == BF16 else U


def rows_ok(what, got, ref, dtype, part=64 * U):
    got = to_np(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    top = np.abs(ref).max(-1, keepdims=True)
    over = np.abs(got - ref) / (part * top + step(dtype) * np.abs(ref) + 1e-37)
    assert over.max(initial=0.0) <= 1, "%s: %.2f of its bound" % (what, over.max())


def sums_ok(what, got, ref, mag, dtype, rows):
    got = to_np(got)
    over = np.abs(got - ref) / ((rows + 128) * U * mag + step(dtype) * np.abs(ref) + 1e-37)
    assert got.shape == ref.shape and over.max() <= 1, "%s: %.2f of its bound" % (what, over.max())


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


GATED = [(1, 1, 1, 16, F32), (1, 1, 1, 16, BF16), (2, 3, 5, 32, F32), (1, 8, 130, 64, F32), (3, 2, 33, 128, F32), (2, 3, 7, 16, BF16),
         (1, 4, 200, 32, BF16), (2, 5, 67, 64, BF16), (1, 16, 150, 128, BF16), (200, 1, 1, 64, BF16), (70, 3, 1, 128, BF16),
         (1, 1, 3000, 16, BF16), (1, 1500, 3, 16, BF16), (2, 2, 2000, 128, BF16)]


def gated_inputs(B, H, N, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    return (r(B, H, N, D) * (0.2 + torch.rand(B, H, N, 1, generator=gen))).to(dtype), (2 * r(B, N, H * D)).to(dtype), \
        (1 + 0.2 * r(D)).to(dtype), r(B, N, H * D).to(dtype)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("case", GATED, ids=lambda c: "-".join(str(x) for x in c))
def test_gated(la, case, rms):
    *shape, dtype = case
    B, H, N, D = shape
    o, g, w, dy = gated_inputs(*shape, dtype, sum(shape))
    do_, gd, wd, dyd = dev(o, g, w, dy)
    heads = lambda t: to_np(t).reshape(B, N, H, D)
    for weight, wdev in ((w, wd), (None, None)):
        y = la.gated_norm_fwd(do_, gd, wdev, rms=rms)
        ref = R.gated(o, g, weight, rms)
        assert y.dtype == dtype and y.shape == g.shape
        # relative to the row before its gate: an output is n w silu, each factor within its bound of itself or of the row
        silu = np.abs(heads(g)) * R.sigmoid(heads(g))
        norm_top = np.abs(R.gated(o, torch.full_like(g, 40.0), weight, rms).reshape(B, N, H, D) / 40).max(-1, keepdims=True)
        over = np.abs(heads(y) - ref.reshape(B, N, H, D)) / (64 * U * norm_top * silu + step(dtype) * np.abs(ref.reshape(B, N, H, D)) + 1e-37)
        assert over.max() <= 1, over.max()
        got = la.gated_norm_bwd(do_, gd, wdev, dyd, rms=rms, dweight=None if weight is not None else torch.empty_like(wd))
        rdo, rdg, rdw, mag = R.gated(o, g, weight, rms, dy)
        rows_ok("do", got[0], rdo, dtype, 128 * U)
        rows_ok("dgate", got[1].view(B, N, H, D), rdg.reshape(B, N, H, D), dtype, 128 * U)
        sums_ok("dweight", got[2], rdw, mag, dtype, B * N * H)
    assert la.gated_norm_bwd(do_, gd, None, dyd, rms=rms)[2] is None
    # in place, and with the heads as a dimension
    y = la.gated_norm_fwd(do_, gd, wd, rms=rms)
    assert torch.equal(la.gated_norm_fwd(do_, gd.view(B, N, H, D), wd, rms=rms), y.view(B, N, H, D))
    want = la.gated_norm_bwd(do_, gd, wd, dyd, rms=rms)
    o2, g2 = do_.clone(), gd.clone()
    got = la.gated_norm_bwd(o2, g2, wd, dyd, rms=rms, dx=o2, dgate=g2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g2 = gd.clone()
    assert torch.equal(la.gated_norm_fwd(do_, g2, wd, rms=rms, out=g2), y)


RESID = [((1, 1), F32), ((5, 1), BF16), ((3, 2), F32), ((7, 7), BF16), ((33, 8), F32), ((65, 16), BF16), ((2, 3, 50, 64), BF16),
         ((129, 128), F32), ((1000, 128), BF16), ((9, 129), F32), ((64, 256), F32), ((31, 255), BF16), ((17, 513), F32),
         ((40, 512), BF16), ((5, 1000), BF16), ((300, 1024), F32), ((1400, 2048), BF16), ((3, 2047), BF16), ((700, 1001), BF16),
         ((5, 4096), F32), ((6, 8192), BF16), ((2, 8193), BF16), ((330, 8200), BF16), ((3, 16384), BF16), ((2, 16383), F32),
         ((2, 16384), F32), ((2000, 40), BF16)]


def resid_inputs(shape, dtype, seed, offset=0.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)
    C = shape[-1]
    return [t.to(dtype) for t in (r(*shape) + offset, r(*shape), 0.5 + 0.3 * r(C), 1 + 0.2 * r(C), 0.3 * r(C), r(*shape), r(*shape))]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shape,dtype", RESID)
def test_residual(la, shape, dtype, rms):
    x, a, sc, w, b, dy, dh = resid_inputs(shape, dtype, shape[-1])
    xd, ad, scd, wd, bd, dyd, dhd = dev(x, a, sc, w, b, dy, dh)
    rows = int(np.prod(shape[:-1]))
    h, y, mean, rstd = la.residual_norm_fwd(xd, ad, scd, wd, bd, rms=rms, return_stats=True)
    rh, ry, rm, rr = R.resid(x, a, sc, w, b, rms)
    rows_ok("h", h, rh, dtype, 2 * U)
    # with one element the layer norm is of a difference of 0: y is the bias alone, rstd that of eps
    n_top = np.abs((rh - rm[..., None]) * rr[..., None]).max(-1, keepdims=True) if shape[-1] > 1 or rms else np.ones(rh.shape[:-1] + (1,))
    lift = np.maximum(1.0, np.abs(rh).max(-1, keepdims=True) * rr[..., None] / 4) if shape[-1] > 1 or rms else 1.0
    wt = np.abs(to_np(w)).max()
    over = np.abs(to_np(y) - ry) / (64 * U * lift * n_top * wt + step(dtype) * np.abs(ry) + 4 * U * np.abs(to_np(b)).max())
    assert over.max() <= 1, over.max()
    assert (mean is None) == rms and rstd.shape == shape[:-1]
    if not rms:
        assert np.abs(to_np(mean) - rm).max() <= 64 * U * np.abs(rh).max()
    if shape[-1] > 1 or rms:
        assert (np.abs(to_np(rstd) / rr - 1) <= 64 * U * np.maximum(1, (np.abs(rh).max(-1) * rr))).all()
    h2, y2 = la.residual_norm_fwd(xd, ad, rms=rms)
    rh2, ry2 = R.resid(x, a, rms=rms)[:2]
    rows_ok("h plain", h2, rh2, dtype, 2 * U)
    x3, a3 = xd.clone(), ad.clone()
    h3, y3 = la.residual_norm_fwd(x3, a3, scd, wd, bd, rms=rms, h=x3, out=a3)
    assert torch.equal(h3, h) and torch.equal(y3, y)
    # the gradient from the kept sum and statistics
    for full in (True, False):
        args = (h, ad, scd, wd, mean, rstd, dyd, dhd) if full else (h, None, None, None, mean, rstd, dyd, None)
        got = la.residual_norm_bwd(*args, rms=rms)
        ref, mags = R.resid_back(h, a if full else None, sc if full else None, w if full else None, mean, rstd, dy, dh if full else None, rms)
        n = np.abs((to_np(h) - (0 if rms else to_np(mean)[..., None])) * to_np(rstd)[..., None])
        d = np.abs(to_np(dy) * (to_np(w) if full else 1))
        top = to_np(rstd)[..., None] * (d.max(-1, keepdims=True) + n.max(-1, keepdims=True) * (d * n).mean(-1, keepdims=True)) + \
            (np.abs(to_np(dh)).max(-1, keepdims=True) if full else 0)
        near = 128 * U * top * np.maximum(1.0, np.abs(to_np(h)).max(-1, keepdims=True) * to_np(rstd)[..., None] / 4)
        for what, g, r, k in (("dx", got[0], ref[0], 1.0), ("da", got[1], ref[1], np.abs(to_np(sc)) if full else 1.0)):
            over = np.abs(to_np(g) - r) / (near * k + step(dtype) * np.abs(r) + 1e-37)
            assert over.max() <= 1, (what, over.max())
        if not full:
            assert got[1] is got[0] and got[2] is None and got[3] is None and got[4] is None
            continue
        flat = lambda t: np.abs(to_np(t)).reshape(rows, -1)
        off = (flat(a) * near.reshape(rows, -1)).sum(0)  # what dx's own bound adds to dscale
        over = np.abs(to_np(got[2]) - ref[2]) / ((rows + 128) * U * mags[0] + off + step(dtype) * np.abs(ref[2]) + 1e-37)
        assert over.max() <= 1, ("dscale", over.max())
        off = (flat(dy) * 4 * U * np.broadcast_to(np.abs(to_np(h)) + (0 if rms else np.abs(to_np(mean)[..., None])), h.shape).reshape(rows, -1) *
               to_np(rstd).reshape(rows, 1)).sum(0)  # n's own roundings
        over = np.abs(to_np(got[3]) - ref[3]) / ((rows + 128) * U * mags[1] + off + step(dtype) * np.abs(ref[3]) + 1e-37)
        assert over.max() <= 1, ("dweight", over.max())
        sums_ok("dbias", got[4], ref[4], mags[2], dtype, rows)
        dh4, a4 = dhd.clone(), ad.clone()
        again = la.residual_norm_bwd(h, a4, scd, wd, mean, rstd, dyd, dh4, rms=rms, dx=dh4, da=a4)
        assert all(torch.equal(p, q) for p, q in zip(again, got))


def test_parts_of_the_sums(la):
    """Single sums, a scale without dh, a weight's gradients into given tensors."""
    x, a, sc, w, b, dy, dh = dev(*resid_inputs((70, 96), BF16, 4))
    h, y, mean, rstd = la.residual_norm_fwd(x, a, sc, w, b, return_stats=True)
    full = la.residual_norm_bwd(h, a, sc, w, mean, rstd, dy)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    none = la.residual_norm_bwd(h, a, sc, None, mean, rstd, dy)
    given = la.residual_norm_bwd(h, a, sc, None, mean, rstd, dy, dweight=dw, dbias=db)
    assert none[3] is None and given[3] is dw and torch.equal(given[0], none[0]) and torch.equal(dw, full[3]) and torch.equal(db, full[4])
    only = la.residual_norm_bwd(h, None, None, w, mean, rstd, dy)
    assert torch.equal(only[0], full[0]) and torch.equal(only[3], full[3]) and only[2] is None


def test_no_rows(la):
    for dtype in (F32, BF16):
        e = torch.empty(0, 48, dtype=dtype, device=DEV)
        p = torch.ones(48, dtype=dtype, device=DEV)
        h, y, mean, rstd = la.residual_norm_fwd(e, e, p, p, p, return_stats=True)
        assert h.shape == y.shape == (0, 48) and mean.shape == rstd.shape == (0,)
        dx, da, ds, dw, db = la.residual_norm_bwd(e, e, p, p, mean, rstd, e, e)
        assert dx.shape == (0, 48) and not ds.any() and not dw.any() and not db.any()
        o, g = torch.empty(2, 3, 0, 16, dtype=dtype, device=DEV), torch.empty(2, 0, 48, dtype=dtype, device=DEV)
        assert la.gated_norm_fwd(o, g, p[:16]).shape == (2, 0, 48)
        assert not la.gated_norm_bwd(o, g, p[:16], g)[2].any()


def test_refusals(la):
    r = lambda *s: torch.randn(*s, device=DEV)
    o, g = r(2, 3, 5, 16), r(2, 5, 48)
    for call in (lambda: la.gated_norm_fwd(o, r(2, 3, 5, 16)), lambda: la.gated_norm_fwd(o, g.bfloat16()),
                 lambda: la.gated_norm_fwd(o, g, r(48)), lambda: la.gated_norm_fwd(o.transpose(1, 2), g),
                 lambda: la.gated_norm_bwd(o, g, None, o), lambda: la.gated_norm_fwd(o, g, out=o)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(la.LaError) as e:
        la.gated_norm_fwd(r(2, 3, 5, 24), r(2, 5, 72))
    assert e.value.status == 2
    x, a, p, st = r(6, 20), r(6, 20), r(20), r(6)
    for call in (lambda: la.residual_norm_fwd(x, r(6, 21)), lambda: la.residual_norm_fwd(x, a, r(21)),
                 lambda: la.residual_norm_bwd(x, None, p, p, st, st, a), lambda: la.residual_norm_bwd(x, a, None, p, None, st, a),
                 lambda: la.residual_norm_bwd(x, a, None, p, st, r(7), a), lambda: la.residual_norm_bwd(x, a, None, p, st, st, a, da=a)):
        with pytest.raises((ValueError, TypeError)):
            call()
    same = torch.empty_like(x)
    for call in (lambda: la.residual_norm_fwd(x, a, h=same, out=same),
                 lambda: la.residual_norm_bwd(x, a, p, p, st, st, a, dx=same, da=same), lambda: la.residual_norm_fwd(x, a, eps=-1.0)):
        with pytest.raises(la.LaError) as e:
            call()
        assert e.value.status == 1
    with pytest.raises(la.LaError) as e:
        la.residual_norm_bwd(x, a, p, p, st, st, a, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 3


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_on_another_stream(la, dtype):
    def make(seed):
        o, g, w, dy = gated_inputs(2, 4, 100, 64, dtype, seed)
        return dev(o, g, w, dy, *resid_inputs((200, 256), dtype, seed))
    def run(o, g, w, dy, x, a, sc, w2, b, dy2, dh):
        h, y, mean, rstd = la.residual_norm_fwd(x, a, sc, w2, b, return_stats=True)
        return (la.gated_norm_fwd(o, g, w, rms=True), *la.gated_norm_bwd(o, g, w, dy, rms=True), h, y, mean, rstd,
                *la.residual_norm_bwd(h, a, sc, w2, mean, rstd, dy2, dh))
    slots, side = make(0), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(*slots)
    for seed in (1, 2):
        fresh = make(seed)
        for s, f in zip(slots, fresh):
            s.copy_(f)
        graph.replay()
        eager = run(*fresh)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, eager))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            other = run(*fresh)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(other, eager))


def test_rows_stay_apart(la):
    """NaN and infinities in a row or a head reach no other row's outputs."""
    x, a, sc, w, b, dy, dh = dev(*resid_inputs((50, 200), BF16, 8))
    want = la.residual_norm_fwd(x, a, sc, w, b)
    x2 = x.clone()
    x2[17, 3] = float("nan")
    got = la.residual_norm_fwd(x2, a, sc, w, b)
    keep = torch.arange(50, device=DEV) != 17
    assert all(torch.equal(p[keep], q[keep]) for p, q in zip(got, want)) and got[1][17].isnan().all()
    o, g, w, dy = dev(*gated_inputs(2, 3, 40, 32, F32, 9))
    y = la.gated_norm_fwd(o, g, w)
    o2 = o.clone()
    o2[1, 2, 5, 0] = float("inf")
    y2 = la.gated_norm_fwd(o2, g, w)
    bad = torch.zeros(2, 40, 3, 32, dtype=torch.bool, device=DEV)
    bad[1, 5, 2] = True
    assert torch.equal(y2.view(2, 40, 3, 32)[~bad], y.view(2, 40, 3, 32)[~bad])

"""GPU parity of cross attention, forward, gradient and apply, against fp64.

Bounds, elementwise, in magnitudes (the reference's sums with every term by its absolute value) and results.  u = 2^-24
for a rounding to fp32; a sum of n terms in any order adds at most n u of its magnitude, so with the sums over M keys,
over G N queries and over the head sizes in turn fp32 costs (M + G N + 2 (Dk + Dv) + 64) u, phi's exponential (a few u)
and the divisions among the 64.  b = 2^-8 for a rounding to bf16, which a bf16 call adds where it says so: o takes phi(q)
(in num and den), phi(k) and S rounded once: 4 b at most; dq takes S in two parts, phi(k) too, all else fp32: 4 b^2;
dk takes phi(q) / den rounded once: b + 4 b^2; dv that and phi(k): 2 b + 4 b^2; all round their result, b of it.
"""
import numpy as np
import pytest
import torch

import cross_ref as R
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


def base(q, k, v):
    return (k.shape[2] + q.shape[1] // k.shape[1] * q.shape[2] + 2 * (q.shape[3] + v.shape[3]) + 64) * U


def within(what, got, ref, mag, part, rounding):
    got = to_np(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    bound = part * mag + rounding * (np.abs(ref) + part * mag) + 1e-37
    over = np.abs(got - ref) / bound
    assert over.max(initial=0.0) <= 1.0, "%s: %.2f of its bound" % (what, over.max())


def check_fwd(got, q, k, v, lengths):
    o, S, z = got
    ro, rS, rz, mag = R.fwd(q, k, v, lengths)
    b, bf = base(q, k, v), q.dtype == BF16
    within("o", o, ro, mag, b + (4 * BU if bf else 0), BU if bf else U)
    aS = R.fwd(q, k, v.abs(), lengths)[1]
    within("S", S, rS, aS, b + (BU * BU if bf else 0), U)
    within("z", z, rz, rz, b + (BU * BU if bf else 0), U)


def check_bwd(got, q, k, v, do, lengths):
    ref, mag = R.bwd(q, k, v, do, lengths)
    b, bf = base(q, k, v), q.dtype == BF16
    for what, g, r, m, part in zip(("dq", "dk", "dv"), got, ref, mag, (4 * BU * BU, BU + 4 * BU * BU, 2 * BU + 4 * BU * BU)):
        within(what, g, r, m, b + (part if bf else 0), BU if bf else U)


def dev(*ts):
    return [t.to(DEV) for t in ts]


# B, H, Hk, N, M, Dk, Dv, dtype, lengths
CASES = [
    (1, 1, 1, 1, 1, 16, 16, F32, None), (1, 2, 2, 17, 64, 16, 16, F32, None), (2, 4, 2, 65, 63, 32, 16, F32, [63, 5]),
    (1, 2, 1, 130, 129, 16, 128, F32, None), (3, 2, 2, 70, 200, 64, 64, F32, [0, 200, 131]),
    (2, 2, 2, 64, 300, 128, 128, F32, [300, 1]), (1, 8, 2, 33, 1000, 128, 32, F32, None), (40, 2, 1, 3, 70, 32, 64, F32, None),
    (2, 8, 2, 16, 64, 128, 128, F32, [64, 0]), (3, 4, 4, 64, 33, 32, 128, F32, [1, 33, -2]), (2, 4, 2, 33, 64, 64, 32, F32, [64, 63]),
    (300, 2, 1, 5, 7, 16, 64, F32, None),
    (1, 1, 1, 1, 1, 64, 64, BF16, None), (1, 1, 1, 128, 128, 128, 128, BF16, None), (2, 2, 2, 127, 129, 128, 128, BF16, [129, 64]),
    (2, 4, 2, 200, 63, 64, 64, BF16, [63, 62]), (3, 4, 1, 100, 257, 128, 64, BF16, [0, 257, 128]),
    (1, 2, 2, 300, 700, 64, 128, BF16, None), (2, 2, 1, 77, 190, 32, 16, BF16, [65, 190]), (1, 3, 3, 140, 65, 16, 128, BF16, None),
    (1, 2, 2, 129, 400, 128, 16, BF16, None), (1, 1, 1, 40, 2000, 128, 128, BF16, None), (1, 1, 1, 2500, 40, 64, 64, BF16, None),
    (40, 2, 2, 5, 100, 64, 64, BF16, list(range(0, 120, 3))), (2, 16, 2, 150, 333, 128, 128, BF16, [333, 200]),
    (70, 1, 1, 130, 129, 128, 128, BF16, [(37 * i) % 140 - 5 for i in range(70)]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_parity(la, case):
    *shape, dtype, lengths = case
    q, k, v, do = R.make(*shape, dtype, seed=sum(shape), lengths=lengths, behind=float("nan") if lengths else None)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    x, g, nd = dev(q, k, v), do.to(DEV), None if n is None else n.to(DEV)
    got = la.cross_fwd(*x, lengths=nd, return_state=True)
    assert torch.equal(la.cross_fwd(*x, lengths=nd), got[0])  # the state does not change the output
    clean = R.make(*shape, dtype, seed=sum(shape), lengths=lengths, behind=0.0 if lengths else None)[:3]
    check_fwd(got, *clean, lengths)
    grads = la.cross_bwd(*x, g, lengths=nd)
    check_bwd(grads, *clean, do, lengths)
    if lengths:
        for b, m in enumerate(lengths):
            m = min(max(m, 0), shape[4])
            assert not grads[1][b, :, m:].any() and not grads[2][b, :, m:].any()
    check_bwd(la.cross_bwd(*x, g, lengths=nd, S=got[1], z=got[2]), *clean, do, lengths)
    check_apply(la, x[0], got[1], got[2], clean, got[0])


def check_apply(la, q, S, z, clean, o):
    """The state's answers: all queries, and single tokens, against the same state in fp64."""
    p, Sd, zd = R.phi(to_np(q)), to_np(S), to_np(z)
    G = q.shape[1] // S.shape[1]
    Sd, zd = (np.repeat(t, G, 1) for t in (Sd, zd))
    den = (p * zd[:, :, None]).sum(-1, keepdims=True)
    inv = np.divide(1.0, den, out=np.zeros_like(den), where=den != 0)
    ref, mag = (p @ Sd) * inv, (p @ np.abs(Sd)) * inv
    bf = q.dtype == BF16
    part = (2 * q.shape[3] + 64) * U + (3 * BU if bf else 0)
    within("apply", la.cross_apply(q, S, z), ref, mag, part, BU if bf else U)
    one = q[:, :, 0].contiguous()
    within("token", la.cross_apply(one, S, z), ref[:, :, 0], mag[:, :, 0], part, BU if bf else U)
    few = q[:, :, :5].contiguous()
    within("few", la.cross_apply(few, S, z), ref[:, :, :5], mag[:, :, :5], part, BU if bf else U)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_empty(la, dtype):
    """No key, no query, all lengths 0: outputs, states and gradients are 0, and nothing else is touched."""
    z4 = lambda *s: torch.zeros(s, dtype=dtype, device=DEV)
    q, do = torch.randn(2, 4, 9, 64, device=DEV).to(dtype), torch.randn(2, 4, 9, 32, device=DEV).to(dtype)
    o, S, z = la.cross_fwd(q, z4(2, 2, 0, 64), z4(2, 2, 0, 32), return_state=True)
    assert not o.any() and not S.any() and not z.any() and o.shape == (2, 4, 9, 32)
    dq, dk, dv = la.cross_bwd(q, z4(2, 2, 0, 64), z4(2, 2, 0, 32), do)
    assert not dq.any() and dk.shape == (2, 2, 0, 64) and dv.shape == (2, 2, 0, 32)
    k, v = torch.randn(2, 2, 70, 64, device=DEV).to(dtype), torch.full((2, 2, 70, 32), float("inf"), device=DEV).to(dtype)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    o, S, z = la.cross_fwd(q, k, v, lengths=none, return_state=True)
    assert not o.any() and not S.any() and not z.any()
    assert not la.cross_apply(q, S, z).any() and not la.cross_apply(q[:, :, 0].contiguous(), S, z).any()
    for g in la.cross_bwd(q, k, v, do, lengths=none) + la.cross_bwd(q, k, v, do, lengths=none, S=S, z=z):
        assert not g.any()
    e = q[:, :, :0].contiguous()
    k, v = torch.randn(2, 2, 70, 64, device=DEV).to(dtype), torch.randn(2, 2, 70, 32, device=DEV).to(dtype)
    o, S, z = la.cross_fwd(e, k, v, return_state=True)
    check = la.cross_fwd(q, k, v, return_state=True)
    assert o.shape == (2, 4, 0, 32) and torch.equal(S, check[1]) and torch.equal(z, check[2])
    assert la.cross_apply(e, S, z).shape == (2, 4, 0, 32)
    dq, dk, dv = la.cross_bwd(e, k, v, do[:, :, :0].contiguous())
    assert dq.numel() == 0 and not dk.any() and not dv.any()


def test_refusals(la):
    r = lambda *s: torch.randn(*s, device=DEV)
    q, k, v = r(2, 4, 8, 16), r(2, 2, 9, 16), r(2, 2, 9, 32)
    S, z = r(2, 2, 16, 32), r(2, 2, 16)
    n = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    for bad in (dict(lengths=n.long()), dict(lengths=n[:1]), dict(out=r(2, 4, 8, 16)), dict(lengths=n.cpu())):
        with pytest.raises((ValueError, TypeError)):
            la.cross_fwd(q, k, v, **bad)
    with pytest.raises(ValueError):
        la.cross_fwd(q, k, v[:, :, :8].contiguous())
    with pytest.raises(ValueError):
        la.cross_fwd(q.transpose(1, 2), k, v)
    with pytest.raises(TypeError):
        la.cross_fwd(q, k.bfloat16(), v)
    with pytest.raises(la.LaError) as e:
        la.cross_fwd(r(2, 3, 8, 16), k, v)  # 2 heads of keys do not divide 3
    assert e.value.status == 1
    do = r(2, 4, 8, 32)
    for bad in (dict(S=S), dict(z=z), dict(S=S.bfloat16(), z=z), dict(S=S, z=z[:1].contiguous()), dict(dk=q)):
        with pytest.raises((ValueError, TypeError)):
            la.cross_bwd(q, k, v, do, **bad)
    with pytest.raises(ValueError):
        la.cross_bwd(q, k, v, q)
    with pytest.raises(ValueError):
        la.cross_apply(q, S, z[:, :, :8].contiguous())
    with pytest.raises(ValueError):
        la.cross_apply(r(2, 4, 8, 32), S, z)
    short = torch.empty(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(la.LaError) as e:
        la.cross_fwd(q, r(2, 2, 70, 16), r(2, 2, 70, 32), workspace=short)
    assert e.value.status == 3
    assert la.last_error() == 0


@pytest.mark.parametrize("dtype,D", [(F32, 32), (BF16, 128)])
def test_captured_and_on_another_stream(la, dtype, D):
    """A captured training call replayed on new inputs, and calls on a side stream, give the eager bits."""
    def inputs(seed):
        q, k, v, do = R.make(2, 4, 2, 150, 260, D, D, dtype, seed=seed)
        return dev(q, k, v, do)
    def step(q, k, v, do, n):
        o, S, z = la.cross_fwd(q, k, v, lengths=n, return_state=True)
        return (o, S, z, *la.cross_bwd(q, k, v, do, lengths=n, S=S, z=z), *la.cross_bwd(q, k, v, do, lengths=n),
                la.cross_apply(q, S, z), la.cross_apply(q[:, :, 0].contiguous(), S, z))
    slots, n = inputs(0), torch.tensor([200, 260], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*slots, n)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step(*slots, n)
    for seed, lens in ((1, [0, 260]), (2, [131, 77])):
        fresh = inputs(seed)
        for s, f in zip(slots, fresh):
            s.copy_(f)
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        eager = step(*fresh, n)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            other = la.cross_bwd(*fresh, lengths=n)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, eager[6:9]))


def test_masked_places_and_nonfinite_heads(la):
    """Infinities behind the lengths change nothing; those in one head stay in it."""
    for dtype, D in ((F32, 64), (BF16, 128)):
        n = [100, 30]
        nd = torch.tensor(n, dtype=torch.int32, device=DEV)
        q, k, v, do = dev(*R.make(2, 2, 2, 140, 133, D, D, dtype, seed=3))
        want = la.cross_fwd(q, k, v, lengths=nd, return_state=True) + la.cross_bwd(q, k, v, do, lengths=nd)
        for fill in (float("nan"), float("inf"), torch.finfo(dtype).min):
            kf, vf = k.clone(), v.clone()
            for b in range(2):
                kf[b, :, n[b]:], vf[b, :, n[b]:] = fill, fill
            got = la.cross_fwd(q, kf, vf, lengths=nd, return_state=True) + la.cross_bwd(q, kf, vf, do, lengths=nd)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        vf = v.clone()
        vf[1, 0, 3, 5] = float("inf")
        got = la.cross_fwd(q, k, vf, lengths=nd, return_state=True) + la.cross_bwd(q, k, vf, do, lengths=nd)
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1, 1], b[1, 1])


def test_underflowing_normaliser(la):
    """Queries and keys so negative that phi is 0: no key answers."""
    q, k = torch.full((1, 1, 3, 16), -300.0, device=DEV), torch.zeros(1, 1, 4, 16, device=DEV)
    v = torch.ones(1, 1, 4, 16, device=DEV)
    assert not la.cross_fwd(q, k, v).any()
    for g in la.cross_bwd(q, k, v, torch.ones(1, 1, 3, 16, device=DEV)):
        assert not g.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[0, 0, 900, 0], [1, 0, 0, 64], [900, 1, 1, 1], [0, 65, 0, 0]])
def test_few_live_chunks(la, dtype, lengths):
    """Lengths that leave fewer chunks than a padded batch has blocks, in workspaces full of NaN: every sum read was written."""
    q, k, v, do = R.make(4, 2, 2, 37, 900, 64, 64, dtype, seed=len(lengths), lengths=lengths, behind=0.0)
    x, g, n = dev(q, k, v), do.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    nan = lambda op: torch.full((la.cross_workspace_bytes(op, 4, 2, 2, 37, 900, 64, 64, dtype) // 4,), float("nan"), device=DEV)
    got = la.cross_fwd(*x, lengths=n, return_state=True, workspace=nan(la.OP_CROSS_FWD))
    check_fwd(got, q, k, v, lengths)
    check_bwd(la.cross_bwd(*x, g, lengths=n, workspace=nan(la.OP_CROSS_BWD)), q, k, v, do, lengths)
    check_bwd(la.cross_bwd(*x, g, lengths=n, S=got[1], z=got[2], workspace=nan(la.OP_CROSS_BWD)), q, k, v, do, lengths)


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_heads_of_one_and_two_chunks(la, Dk, Dv):
    """More heads than blocks, of one, two and three chunks: every chunk meets its own head's state, call after call."""
    for N, M in ((100, 120), (130, 260), (300, 100)):
        B, H = 40, 16
        q, k, v, do = R.make(B, H, H, N, M, Dk, Dv, BF16, seed=N)
        x, g = dev(q, k, v), do.to(DEV)
        first = la.cross_fwd(*x, return_state=True) + la.cross_bwd(*x, g)
        for _ in range(6):
            again = la.cross_fwd(*x, return_state=True) + la.cross_bwd(*x, g)
            assert all(torch.equal(a, b) for a, b in zip(again, first))
        for b in (0, 17, B - 1):
            one = [t[b:b + 1] for t in (q, k, v)]
            check_fwd([t[b:b + 1] for t in first[:3]], *one, None)
            check_bwd([t[b:b + 1] for t in first[3:]], *one, do[b:b + 1], None)

"""Cross attention and the gated norm with as many heads as a call may have (B H = 65,535) and with thousands of heads, against fp64 on
the device.

Bounds, relative to each output's terms by their absolute values, as in the parity tests: u = 2^-24, sums of M + G N + 4 D + 64
roundings; bf16 4 * 2^-8 and its result's 2^-8.
"""
import pytest
import torch

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


def within(what, got, ref, mag, part, rounding):
    over = (got.double() - ref).abs() / (part * mag + rounding * ref.abs() + 1e-37)
    assert float(over.max()) <= 1, "%s: %.2f of its bound" % (what, float(over.max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,N,M,D", [(65535, 1, 1, 1, 3, 16), (65535, 1, 1, 5, 70, 16), (1, 65535, 5, 1, 9, 16), (13107, 5, 5, 20, 2, 32), (700, 8, 4, 40, 130, 64)])
def test_cross(la, dtype, B, H, Hk, N, M, D):
    gen = torch.Generator(device=DEV).manual_seed(B + H)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dtype)
    q, k, v, do = r(B, H, N, D), r(B, Hk, M, D), r(B, Hk, M, D), r(B, H, N, D)
    n = torch.randint(-1, M + 2, (B,), generator=gen, device=DEV, dtype=torch.int32)
    G = H // Hk
    live = (torch.arange(M, device=DEV) < n[:, None])[:, None, :, None]
    phi = lambda x: torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))
    group = lambda x: x.double().reshape(B, Hk, G * N, D)
    pk, vv, pq, d = phi(k.double()) * live, v.double() * live, phi(group(q)), group(do)
    S, z, aS = pk.mT @ vv, pk.sum(2), pk.mT @ vv.abs()
    den = (pq * z[:, :, None]).sum(-1, keepdim=True)
    inv = torch.where(den == 0, 0.0, 1 / den)
    x = pq * inv
    base, bf = (M + G * N + 4 * D + 64) * U, dtype == BF16
    own = BU if bf else U
    back = lambda t: t.reshape(B, H, N, D)
    o, gS, gz = la.cross_fwd(q, k, v, lengths=n, return_state=True)
    within("o", o, back(x @ S), back(x @ aS), base + (4 * BU if bf else 0), own)
    within("S", gS, S, aS, base + (BU * BU if bf else 0), U)
    within("z", gz, z, z, base + (BU * BU if bf else 0), U)
    within("apply", la.cross_apply(q, gS, gz), back(x @ S), back(x @ aS), base + (4 * BU if bf else 0), own)
    Y, aY = (d @ S.mT) * inv, (d.abs() @ aS.mT) * inv
    t, at = (pq * Y).sum(-1, keepdim=True), (pq * aY).sum(-1, keepdim=True)
    R, aR = x.mT @ d, x.mT @ d.abs()
    rr, ar = (x * t).sum(2)[:, :, None], (x * at).sum(2)[:, :, None]
    for S_, z_ in ((None, None), (gS, gz)):
        dq, dk, dv = la.cross_bwd(q, k, v, do, lengths=n, S=S_, z=z_)
        slope = pq.clamp(max=1)
        within("dq", dq, back((Y - t * inv * z[:, :, None]) * slope), back((aY + at * inv * z[:, :, None]) * slope), base + (4 * BU * BU if bf else 0), own)
        slope = pk.clamp(max=1)
        within("dk", dk, (vv @ R.mT - rr) * slope * live, (vv.abs() @ aR.mT + ar) * slope, base + (BU + 4 * BU * BU if bf else 0), own)
        within("dv", dv, pk @ R, pk @ aR, base + (2 * BU + 4 * BU * BU if bf else 0), own)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,N,D", [(1, 65535, 1, 16), (3, 2000, 7, 32), (65535, 1, 1, 128), (2, 1025, 3, 64), (1, 32767, 2, 16)])
def test_gated_norm(la, dtype, B, H, N, D):
    """Against the definition and its gradient by autograd in fp64: sums of D or of all rows, 2 B H N D elements in dweight."""
    gen = torch.Generator(device=DEV).manual_seed(H)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dtype)
    o, gate, w, dy = r(B, H, N, D), r(B, N, H * D), r(D), r(B, N, H * D)
    xs = [t.double().requires_grad_(True) for t in (o, gate, w)]
    y = (torch.nn.functional.layer_norm(xs[0], (D,)) * xs[2]).transpose(1, 2).reshape(B, N, H * D) * torch.nn.functional.silu(xs[1])
    y.backward(dy.double())
    own = BU if dtype == BF16 else U
    off = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert off(la.gated_norm_fwd(o, gate, w), y.detach()) <= (2 * D + 64) * U + own
    for what, g, x in zip(("dx", "dgate", "dweight"), la.gated_norm_bwd(o, gate, w, dy), xs):
        assert off(g, x.grad) <= (4 * D + 256) * U + own, what

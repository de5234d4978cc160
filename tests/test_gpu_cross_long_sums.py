"""Cross attention's sums over many queries against fp64, where an accumulator that cuts off would show.

The reference forms R, r and the state in fp64 on the device, a slice of rows at a time.  What is compared is how much of the
reference a gradient holds, <g, ref> / <ref, ref> - 1: a bias of the sums shows there as it is, while roundings of the results and of
the operands (2^-8 at most each, independent, three of them) average out over the n elements, to 6 * 3 * 2^-8 / sqrt(n) with room.
A part that is lost, counted twice or put elsewhere shows as its share.  u = 2^-24.  Accumulators in tensor memory may cut
off 2 u of what they hold at each of the 8 products of a chunk of 128 rows; they hold at most 64 chunks and grow from 0 about evenly,
so half of 512 * 2 u.  Additions of such periods in fp32, and of the blocks' records: at most (periods + 152) u, random; the
formulas' own: 64 u.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U, BU = 2.0 ** -24, 2.0 ** -8
SLICE = 1 << 17


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


def phi(x):
    x = x.double()
    return torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))


def state(k, v):
    """S and z of one head [M, D] in fp64."""
    S, z = k.new_zeros(k.shape[1], v.shape[1], dtype=F64), k.new_zeros(k.shape[1], dtype=F64)
    for a in range(0, k.shape[0], SLICE):
        p = phi(k[a:a + SLICE])
        S += p.T @ v[a:a + SLICE].double()
        z += p.sum(0)
    return S, z


def key_gradients(q, k, v, do):
    """dk and dv of one head of keys [M, D] in fp64; q, do: [rows, D]."""
    S, z = state(k, v)
    R, r = torch.zeros_like(S), torch.zeros_like(z)
    for a in range(0, q.shape[0], SLICE):
        p, d = phi(q[a:a + SLICE]), do[a:a + SLICE].double()
        X = p / (p @ z)[:, None]
        R += X.T @ d
        r -= X.T @ (X * (d @ S.T)).sum(1)
    pk = phi(k)
    return (v.double() @ R.T + r) * pk.clamp(max=1.0), pk @ R


def held(got, ref):
    got, ref = got.double().flatten(), ref.flatten()
    return abs(float(got @ ref / (ref @ ref)) - 1), float((got - ref).norm() / ref.norm())


# B, H, Hk, N, M, D: a block to a head of 131,072 queries; two blocks' shares of every head; one head over all blocks
@pytest.mark.parametrize("B,H,Hk,N,M,D", [(152, 1, 1, 131072, 4096, 64), (38, 8, 2, 32768, 4096, 128), (1, 1, 1, (1 << 23) + 77, 4096, 128)])
def test_sums_over_queries(la, B, H, Hk, N, M, D):
    gen = torch.Generator(device=DEV).manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF16)
    q, k, v, do = r(B, H, N, D), r(B, Hk, M, D), r(B, Hk, M, D), r(B, H, N, D).mul_(0.5).add_(1.0)
    _, dk, dv = la.cross_bwd(q, k, v, do)
    G = H // Hk
    for b, j in {(0, 0), (B // 2, Hk - 1), (B - 1, 0)}:
        rows = slice(G * j, G * j + G)
        want = key_gradients(q[b, rows].flatten(0, 1), k[b, j], v[b, j], do[b, rows].flatten(0, 1))
        periods = G * N / (128 * 64) + 1
        for what, g, w in zip(("dk", "dv"), (dk, dv), want):
            bias, off = held(g[b, j], w)
            assert bias <= (512 + periods + 152 + 64) * U + 18 * BU / w.numel() ** 0.5, "%s of (%d, %d): %.2e lost" % (what, b, j, bias)
            assert off <= 3 * BU, "%s of (%d, %d): %.2e off" % (what, b, j, off)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_repeated_periods(la, Dk, Dv):
    """Heads whose sums are read out several times by either compute group: the same bits, call after call."""
    N = 66 * 152 * 128 + 300  # about 132 chunks to a block, in heads that end inside blocks
    r = lambda *s: torch.empty(s, dtype=BF16, device=DEV).normal_()
    q, k, v, do = r(1, 2, N, Dk), r(1, 2, 333, Dk), r(1, 2, 333, Dv), r(1, 2, N, Dv)
    first, differ = la.cross_bwd(q, k, v, do), torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(30):
        for a, b in zip(la.cross_bwd(q, k, v, do), first):
            differ += (a.view(torch.int16) != b.view(torch.int16)).sum()
    assert int(differ) == 0 and la.last_error() == 0

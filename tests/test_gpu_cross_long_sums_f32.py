"""Cross attention's fp32 sums over many keys and many queries against fp64, in 2-norms, with heads that fill the blocks.

u = 2^-24.  A running sum of n terms of one sign takes n roundings of at most u of what it holds; independent and evenly spread they
leave sqrt(n / 3) u / sqrt(3): 8 u for the 512 rows that one thread adds up, 6 u for the 256 periods that its record takes of
131,072, 9 u for the keys' phi (ex2.approx, 2 ulp, and its argument's rounding) at most.  40 u is twice their sum; a single sum of all
rows has 120 u.  The gradients are linear in such sums; their own products of the head's size D and divisions add
2 D + 64 u, and both count by the terms before the differences (dq: Y / den and t / den z; dk: R v and r).
"""
import pytest
import torch

from test_gpu_cross_long_sums import F64, SLICE, la, phi, state  # noqa: F401  (la: the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32
U = 2.0 ** -24


def off(got, ref, size=None):
    size = ref if size is None else size
    return float((got.double() - ref).norm() / size.norm())


@pytest.mark.parametrize("B,N,M,D", [(304, 200, 131072, 32), (304, 131072, 200, 32), (76, 300, 131072, 64)])
def test_fp32_sums(la, B, N, M, D):  # noqa: F811
    gen = torch.Generator(device=DEV).manual_seed(N + D)
    r = lambda n: torch.randn(B, 1, n, D, generator=gen, device=DEV)
    q, k, v, do = r(N), r(M), r(M).mul_(0.5).add_(1.0), r(N).mul_(0.5).add_(1.0)
    o, S, z = la.cross_fwd(q, k, v, return_state=True)
    dq, dk, dv = la.cross_bwd(q, k, v, do, S=S, z=z)
    for b in (0, B // 2, B - 1):
        wS, wz = state(k[b, 0], v[b, 0])
        assert off(S[b, 0], wS) <= 40 * U, "S %.1f u" % (off(S[b, 0], wS) / U)
        assert off(z[b, 0], wz) <= 40 * U, "z %.1f u" % (off(z[b, 0], wz) / U)
        R, wq, terms = torch.zeros_like(wS), [], []
        wr = torch.zeros_like(wz)
        for a in range(0, N, SLICE):
            p, d = phi(q[b, 0, a:a + SLICE]), do[b, 0, a:a + SLICE].double()
            inv = 1 / (p @ wz)[:, None]
            Y = (d @ wS.T) * inv
            t = (p * Y).sum(1, keepdim=True)
            wq.append((Y - t * inv * wz) * p.clamp(max=1.0))
            terms.append((Y.abs() + t.abs() * inv * wz) * p.clamp(max=1.0))
            R += (p * inv).T @ d
            wr -= (p * inv * t).sum(0)
        part = (40 + 40 + 2 * D + 64) * U
        e = off(dq[b, 0], torch.cat(wq), torch.cat(terms))
        assert e <= part, "dq %.1f u of its terms" % (e / U)
        pk, vv = phi(k[b, 0]), v[b, 0].double()
        slope = pk.clamp(max=1.0)
        e = off(dk[b, 0], (vv @ R.T + wr) * slope, (vv.abs() @ R.abs().T + wr.abs()) * slope)
        assert e <= part, "dk %.1f u of its terms" % (e / U)
        e = off(dv[b, 0], pk @ R, pk @ R.abs())
        assert e <= part, "dv %.1f u" % (e / U)

"""Calls of cross attention and of the norms around a block with stream=, as in test_streams.py, and from two host threads."""
import threading

import pytest
import torch

import test_gpu_threads as H
import test_streams as T

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def operands(device):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen)
    bf = lambda *s: r(*s).to(BF16)
    t = dict(q=bf(2, 4, 700, 128), k=bf(2, 2, 900, 128), v=bf(2, 2, 900, 64), do=bf(2, 4, 700, 64), n=torch.tensor([900, 333], dtype=torch.int32),
             S=r(2, 2, 128, 64), z=r(2, 2, 128).abs() + 1, o=bf(2, 4, 700, 64), gate=bf(2, 700, 256), w=bf(64), dy=bf(2, 700, 256),
             x=r(3000, 128), a=r(3000, 128), sc=r(128), nw=r(128), nb=r(128), mean=r(3000) / 16, rstd=1 + r(3000).abs(), dh=r(3000, 128))
    return {n: x.to(device) for n, x in t.items()}


# name -> (call, whether it has a workspace)
CALLS = {
    "cross_fwd": (lambda la, t, s: la.cross_fwd(t["q"], t["k"], t["v"], lengths=t["n"], stream=s, return_state=True), True),
    "cross_bwd": (lambda la, t, s: la.cross_bwd(t["q"], t["k"], t["v"], t["do"], lengths=t["n"], stream=s), True),
    "cross_apply": (lambda la, t, s: la.cross_apply(t["q"], t["S"], t["z"], stream=s), True),
    "gated_norm_fwd": (lambda la, t, s: la.gated_norm_fwd(t["o"], t["gate"], t["w"], stream=s), False),
    "gated_norm_bwd": (lambda la, t, s: la.gated_norm_bwd(t["o"], t["gate"], t["w"], t["dy"], stream=s), True),
    "residual_norm_fwd": (lambda la, t, s: la.residual_norm_fwd(t["x"], t["a"], t["sc"], t["nw"], t["nb"], stream=s, return_stats=True), False),
    "residual_norm_bwd": (lambda la, t, s: la.residual_norm_bwd(t["x"], t["a"], t["sc"], t["nw"], t["mean"], t["rstd"], t["dh"], t["dh"],
                                                                stream=s), True),
}


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


def patched(monkeypatch, name):
    monkeypatch.setitem(T.CALLS, name, CALLS[name])
    monkeypatch.setattr(T, "operands", operands)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_are_made_on_the_given_stream(name, monkeypatch):
    patched(monkeypatch, name)
    T.test_allocations_are_made_on_the_given_stream(name, monkeypatch)


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_the_current_stream_stays_its_own(la, name, monkeypatch):
    patched(monkeypatch, name)
    T.test_memory_of_the_current_stream_stays_its_own(la, name)


def cross_calls(la, n):
    D, dt = n
    r = lambda *s: torch.randn(*s, device=DEV).to(dt)
    q, k, v, do = r(1, 2, 150, D), r(1, 2, 200, D), r(1, 2, 200, D), r(1, 2, 150, D)
    S, z = torch.randn(1, 2, D, D, device=DEV), torch.rand(1, 2, D, device=DEV) + 1
    code = la.LA_BF16 if dt == BF16 else la.LA_F32
    s = la.CrossShape(1, 2, 2, 150, 200, D, D, code)
    ws = lambda op: [H.empty(la.cross_workspace_bytes(op, 1, 2, 2, 150, 200, D, D, dt)), la.cross_workspace_bytes(op, 1, 2, 2, 150, 200, D, D, dt)]
    outs = [torch.empty_like(t) for t in (q, q, k, v, q)]
    return [H.Call("la_cross_fwd", [q, k, v, None, outs[0], None, None], s, ws(la.OP_CROSS_FWD), [outs[0]]),
            H.Call("la_cross_bwd", [q, k, v, None, None, None, do, *outs[1:4]], s, ws(la.OP_CROSS_BWD), outs[1:4]),
            H.Call("la_cross_apply", [q, S, z, outs[4]], s, ws(la.OP_CROSS_APPLY), [outs[4]])]


def norm_calls(la, C):
    r = lambda *s: torch.randn(*s, device=DEV)
    x, a, dy, w, stat = r(700, C), r(700, C), r(700, C), r(C), r(700).abs() + 1
    s, nb = la.NormShape(700, C, la.LA_F32), la.residual_norm_workspace_bytes(700, C, F32)
    h, y, dx, da, ds, dw, db = (torch.empty_like(t) for t in (x, x, x, x, w, w, w))
    return [H.Call("la_residual_norm_fwd", [x, a, w, w, w, h, y, None, None], s, [0, 1e-5], [h, y]),
            H.Call("la_residual_norm_bwd", [x, a, w, w, stat, stat, dy, dy, dx, da, ds, dw, db], s, [0, H.empty(nb), nb], [dx, da, ds, dw, db])]


PAIRS = [(cross_calls, (128, dt), (16, dt), i) for dt in (F32, BF16) for i in range(3)] + \
    [(norm_calls, *c, i) for c in ((2048, 260), (2047, 259)) for i in (0, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("make,large,small,which", PAIRS)
def test_threads_do_not_disturb_each_other(la, make, large, small, which, monkeypatch):
    monkeypatch.setattr(H, "TIMES", 1000)
    H.test_threads_do_not_disturb_each_other(la, make, large, small, which)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["la_cross_fwd", "la_cross_bwd", "la_cross_apply", "la_causal_fwd", "la_noncausal_fwd"])
def test_first_call_of_a_thread(la, name):
    """A C caller's thread that has used nothing of CUDA before: the call itself gives the thread its context."""
    if name.startswith("la_cross"):
        c = next(c for c in cross_calls(la, (128, BF16)) if c.name == name)
    else:
        B, heads, N, D = 1, 2, 300, 128
        q, k, v = (torch.randn(B, heads, N, D, device=DEV).to(BF16) for _ in range(3))
        nb = la.workspace_bytes(la.OP_CAUSAL_FWD if "noncausal" not in name else la.OP_NONCAUSAL_FWD, B, heads, N, D, D, BF16)
        c = H.Call(name, [q, k, v, torch.empty_like(v)], la.Shape(B, heads, N, D, D, la.LA_BF16), [H.empty(nb), nb], [])
    torch.cuda.synchronize()
    call, got = c.bound(la, torch.cuda.Stream()), []
    th = threading.Thread(target=lambda: got.append((call(), la.library().la_error_detail())))
    th.start()
    th.join()
    torch.cuda.synchronize()
    assert got[0][0] == 0, got

"""Calls with stream=: what a call allocates belongs to the stream that it runs on.

On the CPU the binding runs over host tensors against a library that does nothing, and the allocations are watched; on
the GPU the stream that is given is held back, and the memory that the current stream gets meanwhile has to stay its own.
"""
import contextlib

import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16
CYCLES = 200_000_000  # about 0.1 s


def operands(device):
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen)
    B, H, N, D = 1, 2, 1000, 128
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    return {n: t.to(device) for n, t in dict(
        q=unit(r(B, H, N, D)).to(BF16), k=unit(r(B, H, N, D)).to(BF16), v=r(B, H, N, D).to(BF16), do=r(B, H, N, D).to(BF16),
        g=(-r(B, H, N).abs() / 8).to(BF16), beta=torch.sigmoid(r(B, H, N)).to(BF16), q1=unit(r(B, H, D)).to(BF16),
        v1=r(B, H, D).to(BF16), g1=(-r(B, H).abs()).to(BF16), S=r(B, H, D, D), z=r(B, H, D).abs() + 1,
        gamma=torch.tensor([0.9, 0.99]), x=r(3000, 128), dy=r(3000, 128), w=r(128), b=r(128),
        mean=r(3000) / 16, rstd=1 + r(3000).abs()).items()}


# name -> (call, whether it has a workspace)
CALLS = {
    "noncausal_fwd": (lambda la, t, s: la.noncausal_fwd(t["q"], t["k"], t["v"], stream=s), True),
    "noncausal_bwd": (lambda la, t, s: la.noncausal_bwd(t["q"], t["k"], t["v"], t["do"], stream=s), True),
    "causal_fwd": (lambda la, t, s: la.causal_fwd(t["q"], t["k"], t["v"], stream=s, return_state=True), True),
    "causal_fwd_one_launch": (lambda la, t, s: la.causal_fwd(t["q"], t["k"], t["v"], stream=s, one_launch=True), True),
    "causal_bwd": (lambda la, t, s: la.causal_bwd(t["q"], t["k"], t["v"], t["do"], stream=s), True),
    "recurrent_step": (lambda la, t, s: la.recurrent_step(t["q1"], t["q1"], t["v1"], t["S"], t["z"], stream=s), False),
    "retention_fwd": (lambda la, t, s: la.retention_fwd(t["q"], t["k"], t["v"], t["gamma"], stream=s, return_state=True),
                      True),
    "retention_step": (lambda la, t, s: la.retention_step(t["q1"], t["q1"], t["v1"], t["gamma"], t["S"], stream=s),
                       False),
    "gated_delta_fwd": (lambda la, t, s: la.gated_delta_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], stream=s,
                                                            return_state=True), True),
    "gated_delta_bwd": (lambda la, t, s: la.gated_delta_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["do"], stream=s,
                                                            return_dS0=True), True),
    "gated_delta_step": (lambda la, t, s: la.gated_delta_step(t["q1"], t["q1"], t["v1"], t["g1"], t["g1"], t["S"],
                                                              stream=s), False),
    "layer_norm_fwd": (lambda la, t, s: la.layer_norm_fwd(t["x"], t["w"], t["b"], stream=s, return_stats=True), False),
    "layer_norm_bwd": (lambda la, t, s: la.layer_norm_bwd(t["x"], t["w"], t["mean"], t["rstd"], t["dy"], stream=s), True),
}


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


class Nothing:
    """A library whose calls succeed without doing anything."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_bytes") else 0


class Side:
    cuda_stream = 7


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_are_made_on_the_given_stream(name, monkeypatch):
    import causal_linear_attention_phi_gb300 as la
    side, at, made, kept = Side(), [0], [], []

    @contextlib.contextmanager
    def on(s):
        before, at[0] = at[0], s.cuda_stream
        yield
        at[0] = before

    def watched(f):
        def g(*a, **kw):
            t = f(*a, **kw)
            made.append((t, at[0]))
            return t
        return g

    monkeypatch.setattr(la, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(la, "library", lambda: Nothing())
    monkeypatch.setattr(la, "_stream_ptr", lambda s=None: at[0] if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "Stream", Side)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: at[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t, s)))
    ins = operands("cpu")
    call, workspace = CALLS[name]
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", watched(torch.empty))
        m.setattr(torch, "empty_like", watched(torch.empty_like))
        out = tensors(call(la, ins, side))
    assert at[0] == 0 and {s for _, s in made} == {side.cuda_stream}
    # what the caller gets also waits for the current stream, the workspace (seen by the call alone) need not
    assert {id(t) for t, _ in kept} == {id(t) for t in out} and {s for _, s in kept} == {0}
    assert len(made) == len(out) + workspace


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


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_memory_of_the_current_stream_stays_its_own(la, name):
    call, _ = CALLS[name]
    ins, again, third = (operands("cuda:0") for _ in range(3))  # a step changes its state
    ref = tensors(call(la, ins, None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    out = tensors(call(la, again, side))  # its kernels are yet to start; its workspace is let go
    mine = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda:0") for n in
            [1 << i for i in range(9, 25)] for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert all(bool((t == 0x5A).all()) for t in mine)
    del out, mine

    # the other way round: memory let go by the current stream, whose work on it is still to run
    sizes = [t.numel() * t.element_size() for t in ref]
    old = [torch.full((n,), 0x33, dtype=torch.uint8, device="cuda:0") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    copies = [t.clone() for t in old]
    del old
    side.synchronize()
    out = tensors(call(la, third, side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    torch.cuda.synchronize()
    assert all(bool((t == 0x33).all()) for t in copies)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.gpu
def test_a_stream_known_by_its_handle(la):
    """A stream object of another library, of which only the handle is known."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    ins = operands("cuda:0")
    ref = la.gated_delta_bwd(*(ins[n] for n in ("q", "k", "v", "g", "beta", "do")))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (Handle(side), Handle(torch.cuda.current_stream())):
        out = la.gated_delta_bwd(*(ins[n] for n in ("q", "k", "v", "g", "beta", "do")), stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))

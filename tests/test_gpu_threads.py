"""Two host threads that call the same kernels with different sizes, each on its own stream.

The calls go to the C entry points with arguments made beforehand, so that the threads are in the library nearly all the
time; the sizes of a pair need different amounts of shared memory of one kernel.
"""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32
TIMES = 3000


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


class Call:
    """One C call: its name, its tensors (None: a null pointer) in order, its shape and what follows it."""

    def __init__(self, name, tensors, shape, tail, outs):
        self.name, self.tensors, self.shape, self.tail, self.outs = name, tensors, shape, tail, outs

    def bound(self, la, stream):
        fn = getattr(la.library(), self.name)
        args = [None if t is None else t.data_ptr() for t in self.tensors] + [self.shape]
        args += [x.data_ptr() if isinstance(x, torch.Tensor) else x for x in self.tail] + [stream.cuda_stream]
        return lambda: fn(*args)


def empty(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)


def head_calls(la, D):
    r = lambda *s: torch.randn(*s, device=DEV)
    B, H, N = 1, 2, 80
    q, k, v, do = (r(B, H, N, D) / D ** 0.5 for _ in range(4))
    g, beta, gamma = -r(B, H, N).abs(), r(B, H, N).sigmoid(), torch.tensor([0.9, 0.8], device=DEV)
    like = lambda *ts: [torch.empty_like(t) for t in ts]
    s = la.Shape(B, H, N, D, D, la.LA_F32)

    def call(name, op, ins, outs):
        nb = la.workspace_bytes(op, B, H, N, D, D, F32)
        return Call(name, [*ins, *outs], s, [empty(nb), nb], [o for o in outs if o is not None])

    return [call("la_gated_delta_fwd", la.OP_GATED_DELTA_FWD, (q, k, v, g, beta, None), [torch.empty_like(v), None]),
            call("la_gated_delta_bwd", la.OP_GATED_DELTA_BWD, (q, k, v, g, beta, do), like(q, k, v, g, beta)),
            call("la_causal_fwd", la.OP_CAUSAL_FWD, (q, k, v), like(v)),
            call("la_causal_bwd", la.OP_CAUSAL_BWD, (q, k, v, do), like(q, k, v)),
            call("la_noncausal_fwd", la.OP_NONCAUSAL_FWD, (q, k, v), like(v)),
            call("la_noncausal_bwd", la.OP_NONCAUSAL_BWD, (q, k, v, do), like(q, k, v)),
            call("la_retention_fwd", la.OP_RETENTION_FWD, (q, k, v, gamma), [torch.empty_like(v), None])]


def norm_calls(la, C):
    rows = 700
    x, dy, w, b = (torch.randn(*s, device=DEV) for s in ((rows, C), (rows, C), (C,), (C,)))
    y, dx, dw, db, mean, rstd = (torch.empty_like(t) for t in (x, x, w, w, x[:, 0], x[:, 0]))
    s, nb = la.NormShape(rows, C, la.LA_F32), la.layer_norm_workspace_bytes(rows, C, F32)
    stats = [torch.zeros_like(mean), torch.ones_like(rstd)]
    return [Call("la_layer_norm_fwd", [x, w, b, y, mean, rstd], s, [1e-5], [y, mean, rstd]),
            Call("la_layer_norm_bwd", [x, w, *stats, dy, dx, dw, db], s, [empty(nb), nb], [dx, dw, db])]


# the two threads' sizes: one kernel, much and little of the shared memory that it takes
PAIRS = [(head_calls, 128, 16, i) for i in range(7)] + [(norm_calls, *c, i) for c in ((512, 260), (511, 259)) for i in (0, 1)]


@pytest.mark.parametrize("make,large,small,which", PAIRS)
def test_threads_do_not_disturb_each_other(la, make, large, small, which):
    calls = [make(la, n)[which] for n in (large, small)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    bound = [c.bound(la, s) for c, s in zip(calls, streams)]
    assert [b() for b in bound] == [0, 0]
    torch.cuda.synchronize()
    refs = [[o.clone() for o in c.outs] for c in calls]
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def work(b):
        start.wait()
        for _ in range(TIMES):
            if b() != 0:
                failed.append(la.library().la_error_detail())
                return

    threads = [threading.Thread(target=work, args=(b,)) for b in bound]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(torch.equal(a, b) for c, r in zip(calls, refs) for a, b in zip(c.outs, r))

"""Gated delta and layer norm where element offsets pass 2^31, at the most heads, and under the debug build.

The large inputs repeat a few heads (or rows): the first group is checked against fp64 with the bounds of the small
cases (tests/test_gpu_gated_delta.py, tests/test_gpu_layer_norm.py), and every other group has to have its bits.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import delta_ref as R
from test_gpu_gated_delta import TOL_BF16, TOL_F32, TOL_STATE, close, make
from test_gpu_layer_norm import STEP, make as make_norm, row_err
from util import to_np

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
HEADS, TIMES = 5, 13107  # 65535 heads


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 200 << 30:
        pytest.skip("needs 200 GB")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    la.library()
    la.clear_error()
    yield la
    assert la.last_error() == 0
    torch.cuda.empty_cache()


def repeated(t):
    return t.to(DEV).repeat(1, TIMES, *([1] * (t.dim() - 2)))


def same_groups(t):
    g = t.view(TIMES, HEADS, -1)
    return all(torch.equal(g[i], g[0]) for i in (1, TIMES // 2, TIMES - 1)) and bool((g == g[:1]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_delta(la, dtype):
    """65535 heads of 257 positions of 128 x 128: 2.16e9 elements in q, and four whole chunks and a tail of one position."""
    q, k, v, g, beta, do = make(11, 1, HEADS, 257, 128, 128, dtype, "packed")
    assert TIMES * q.numel() > 2 ** 31
    big = [repeated(t) for t in (q, k, v, g, beta)]
    o, S = la.gated_delta_fwd(*big, return_state=True)
    ro, rS = R.delta_fwd(q, k, v, g, beta)
    close("o", o[:, :HEADS], ro, TOL_BF16 if dtype == BF16 else TOL_F32)
    close("S", S[:, :HEADS], rS, TOL_STATE[dtype])
    assert same_groups(o) and same_groups(S)
    del o, S
    grads = la.gated_delta_bwd(*big, repeated(do))
    for n, x, r in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, R.delta_bwd(q, k, v, g, beta, do)):
        close(n, x[:, :HEADS], r, (16 if n == "dg" else 4) * TOL_F32 if dtype == F32 else 5 * 2.0 ** -8)
        assert same_groups(x), n


def test_gated_delta_step(la):
    """States of 65535 heads: 1.07e9 fp32 elements, 4.3 GB."""
    q, k, v, g, beta, _ = make(12, 1, HEADS, 1, 128, 128, BF16)
    gen = torch.Generator().manual_seed(2)
    S0 = torch.randn(1, HEADS, 128, 128, generator=gen)
    ro, rS = R.delta_fwd(q, k, v, g, beta, S0)
    S = repeated(S0)
    out = la.gated_delta_step(*(repeated(t)[:, :, 0].contiguous() for t in (q, k, v, g, beta)), S)
    close("out", out[:, :HEADS, None], ro, 2.0 ** -8 + TOL_F32)
    close("S", S[:, :HEADS], rS, TOL_F32)
    assert same_groups(out) and same_groups(S)


def test_layer_norm(la):
    """1025 rows of 2048, 1024 times over: 2.15e9 elements."""
    x, w, b, dy = make_norm((1025, 2048), BF16, 13)
    times = 1024
    big = lambda t: t.to(DEV).repeat(times, 1)
    xb, wd = big(x), w.to(DEV)
    assert xb.numel() > 2 ** 31
    y, mean, rstd = la.layer_norm_fwd(xb, wd, b.to(DEV), return_stats=True)
    assert row_err(y[:1025], R.norm_fwd(x, w, b)[0]) <= STEP[BF16]
    assert bool((y.view(times, 1025, 2048) == y[:1025]).all())
    del y
    dyb = big(dy)
    dx, dw, db = la.layer_norm_bwd(xb, wd, mean, rstd, dyb)
    rx, rw, rb = R.norm_bwd(x, w, dy)
    assert row_err(dx[:1025], rx) <= 4 * STEP[F32] * 8 + STEP[BF16]
    assert bool((dx.view(times, 1025, 2048) == dx[:1025]).all())
    h = R.norm_fwd(x)[0]
    # sums of 1.05e6 rows: at most 4096 + 64 additions along any path, each off by half a step of the magnitudes' sum
    for got, ref, mag in ((dw, rw, np.abs(to_np(dy) * h).sum(0)), (db, rb, np.abs(to_np(dy)).sum(0))):
        assert (np.abs(to_np(got) - times * ref) <= times * (2.0 ** -8 * np.abs(ref) + 2.0 ** -24 * 4160 * mag)).all()


def run_debug_cases():
    """Runs in the child: sequences, gradients and steps of both paths, norms of every row form, then the error word."""
    import causal_linear_attention_phi_gb300 as la
    assert la.version().endswith("-debug"), la.version()
    la.clear_error()
    d = lambda *ts: [t.to(DEV) for t in ts]
    for B, H, N, Dk, Dv, dtype in [(1, 2, 65, 16, 128, F32), (2, 2, 200, 128, 64, F32), (1, 3, 129, 32, 64, BF16),
                                   (2, 1, 100, 128, 16, BF16), (1, 2, 1100, 128, 128, BF16), (1, 3, 500, 64, 64, BF16)]:
        q, k, v, g, beta, do = make(N, B, H, N, Dk, Dv, dtype, "packed")
        o, S = la.gated_delta_fwd(*d(q, k, v, g, beta), return_state=True)
        ro, rS = R.delta_fwd(q, k, v, g, beta)
        close("o", o, ro, TOL_BF16 if dtype == BF16 else TOL_F32)
        close("S", S, rS, TOL_STATE[dtype])
        for n, x, r in zip(("dq", "dk", "dv", "dg", "dbeta"), la.gated_delta_bwd(*d(q, k, v, g, beta, do)),
                           R.delta_bwd(q, k, v, g, beta, do)):
            close(n, x, r, (16 if n == "dg" else 4) * TOL_F32 if dtype == F32 else 5 * 2.0 ** -8)
        la.gated_delta_step(*(t[:, :, 0].contiguous() for t in d(q, k, v, g, beta)), S)
    for shape, dtype in [((5, 7), BF16), ((33, 128), F32), ((65, 512), BF16), ((9, 8192), BF16), ((3, 2047), F32)]:
        x, w, b, dy = make_norm(shape, dtype, 3)
        y, mean, rstd = la.layer_norm_fwd(*d(x, w, b), return_stats=True)
        assert row_err(y, R.norm_fwd(x, w, b)[0]) <= 4 * STEP[dtype]
        dx, _, _ = la.layer_norm_bwd(*d(x, w), mean, rstd, *d(dy))
        assert row_err(dx, R.norm_bwd(x, w, dy)[0]) <= 32 * STEP[F32] + STEP[dtype]
    st = la.last_error()
    assert st == 0, "sticky status %d: %s" % (st, la.library().la_error_detail())
    print("debug build cases ok")


def test_under_the_debug_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_linear_attention_phi_gb300 import build
    build.build_library(debug=True)
    env = dict(os.environ, LA_DEBUG="1")
    code = "import sys; sys.path[:0] = [%r, %r]; import test_gpu_gated_delta_large as t; t.run_debug_cases()" % (HERE, ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=900)
    assert r.returncode == 0 and "debug build cases ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]

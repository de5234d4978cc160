"""The parity tests of the gated delta rule (segments among them) and of layer norm's row forms once more under the debug
build: every index check of their kernels holds, so the error word stays clear."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FILES = ["test_gpu_gated_delta.py", "test_gated_delta_pieces.py", "test_gpu_layer_norm.py", "test_gpu_layer_norm_rows.py",
         "test_gpu_layer_norm_params.py", "test_gpu_gated_delta_segments.py"]


def run():
    """In the child: the files' GPU tests (of the segments, one of each padded size and of padded heads)."""
    import causal_linear_attention_phi_gb300 as la
    assert la.version().endswith("-debug"), la.version()
    la.clear_error()
    keep = "not test_segments or 2-1300-64 or 3-1100-16 or 12-1500-128 or 2-1500-32"
    status = pytest.main(["-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", keep] + [os.path.join(HERE, f) for f in FILES])
    word = la.last_error()
    assert status == 0 and word == 0, "status %s, error word %d: %s" % (status, word, la.library().la_error_detail())
    print("debug build tests ok")


def test_parity_tests_under_the_debug_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_linear_attention_phi_gb300 import build
    build.build_library(debug=True)
    env = dict(os.environ, LA_DEBUG="1")
    code = "import sys; sys.path[:0] = [%r, %r]; import test_gpu_debug_build_more as t; t.run()" % (HERE, ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=900, cwd=ROOT)
    assert r.returncode == 0 and "debug build tests ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]

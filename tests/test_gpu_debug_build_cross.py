"""The parity tests of cross attention and of the norms around a block once more under the debug build: every index check of their
kernels holds, so the error word stays clear."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FILES = ["test_gpu_cross.py", "test_gpu_block_norm.py"]


def run():
    """In the child: the files' GPU tests."""
    import causal_linear_attention_phi_gb300 as la
    assert la.version().endswith("-debug"), la.version()
    la.clear_error()
    status = pytest.main(["-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"] + [os.path.join(HERE, f) for f in FILES])
    word = la.last_error()
    assert status == 0 and word == 0, "status %s, error word %d: %s" % (status, word, la.library().la_error_detail())
    print("debug build tests ok")


def test_parity_tests_under_the_debug_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from causal_linear_attention_phi_gb300 import build
    build.build_library(debug=True)
    env = dict(os.environ, LA_DEBUG="1")
    code = "import sys; sys.path[:0] = [%r, %r]; import test_gpu_debug_build_cross as t; t.run()" % (HERE, ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=900, cwd=ROOT)
    assert r.returncode == 0 and "debug build tests ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]

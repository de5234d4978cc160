"""The example layer: it learns to recall, and decoding token by token gives what the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "gated_delta_layer.py")


@pytest.mark.parametrize("graph", [False, True])
def test_example(graph):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    spec = importlib.util.spec_from_file_location("gated_delta_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(steps=200, graph=graph)
    # 48 values to choose from: a loss of ln 48 = 3.9 without recall
    assert r["last_loss"] < 2.0
    # bf16 activations: 16 roundings of half a step along the two layers, at most
    assert r["decode_error"] <= 16 * 2.0 ** -8
    assert la.last_error() == 0

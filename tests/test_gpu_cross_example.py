"""The example decoder: it runs, its gradients are those of the same model in fp64, decoding gives the whole pass's logits.

Bounds.  fp32: the model chains about 20 products and norms of sums of at most 200 terms, 200 * 2^-24 each, relative to each
output's largest: 20 * 200 * 2^-24 = 2.4e-4.  Decoding in bf16 against the whole pass: both round the same values at about 12
places a layer (2^-8 each), in other orders of summation and with S in fp32 instead of bf16: 2 layers * 12 * 2^-8 = 0.1.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import causal_linear_attention_phi_gb300 as la
    la.build.build_library()
    la.clear_error()
    import cross_attention_layer
    yield cross_attention_layer
    assert la.last_error() == 0


def plain(model, params, pairs, lengths, asked):
    """The model's logits from its parameters in elementary operations."""
    p = dict(zip((n for n, _ in model.named_parameters()), params))
    phi = lambda t: torch.nn.functional.elu(t) + 1
    norm = lambda h, w, b: torch.nn.functional.layer_norm(h, h.shape[-1:]) * w + b
    e = p["embed"][pairs]
    m = e[:, :, 0] + e[:, :, 1].roll(e.shape[-1] // 2, -1)
    x = p["embed"][asked]
    a = torch.zeros_like(x)
    live = torch.arange(pairs.shape[1], device=pairs.device) < lengths[:, None]
    for i, layer in enumerate(model.layers):
        g = lambda n: p["layers.%d.%s" % (i, n)]
        H, Hk, D = layer.heads, layer.key_heads, layer.head
        x = x + g("scale") * a
        n = norm(x, g("n_w"), g("n_b"))
        heads = lambda t, c: t.view(*t.shape[:2], c, D).transpose(1, 2)
        kv = m @ g("w_kv")
        k, v = (heads(t, Hk).repeat_interleave(H // Hk, 1) for t in kv.split(Hk * D, -1))
        s = phi(heads(n @ g("w_q"), H)) @ phi(k).transpose(-1, -2) * live[:, None, None]
        o = s / s.sum(-1, keepdim=True) @ v
        o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + 1e-5) * g("h_w")
        a = (o.transpose(1, 2).flatten(2) * torch.nn.functional.silu(n @ g("w_gate"))) @ g("w_out")
    return norm(x + p["f_scale"] * a, p["f_w"], p["f_b"]) @ p["head"]


@pytest.mark.parametrize("heads,key_heads,head", [(4, 2, 32), (2, 1, 128), (3, 3, 16)])
def test_gradients(ex, heads, key_heads, head):
    torch.manual_seed(1)
    gen = torch.Generator().manual_seed(2)
    model = ex.Model(80, width=64, heads=heads, key_heads=key_heads, head=head, dtype=torch.float32).to(DEV)
    pairs, lengths, asked, values = ex.lookup_batch(5, 20, 9, 40, gen, DEV)
    weight = torch.randn(5, 9, 80, device=DEV)
    out = model(pairs, lengths, asked)
    grads = torch.autograd.grad((out * weight).sum(), list(model.parameters()))
    wide = [p.detach().double().requires_grad_() for p in model.parameters()]
    ref = plain(model, wide, pairs, lengths, asked)
    want = torch.autograd.grad((ref * weight.double()).sum(), wide)
    # (the first layer's scale multiplies a of 0: its gradient is 0 on both sides)
    off = lambda a, b: float((a.detach().double() - b.detach()).abs().max() / b.detach().abs().max().clamp(min=1e-30))
    assert off(out, ref) <= 2.4e-4
    for (name, _), a, b in zip(model.named_parameters(), grads, want):
        assert off(a, b) <= 2.4e-4, (name, off(a, b))


def test_example_runs_and_decodes(ex):
    r = ex.main(steps=5)
    assert len(r["losses"]) == 5 and all(x == x and x < 1e3 for x in r["losses"])
    assert r["decode_error"] <= 0.1


def test_training_step_in_bf16(ex):
    """Gradients of a bf16 model are finite, of their parameters' shapes, and the same every time."""
    torch.manual_seed(3)
    gen = torch.Generator().manual_seed(4)
    model = ex.Model(80, head=128).to(DEV)
    pairs, lengths, asked, values = ex.lookup_batch(8, 20, 30, 40, gen, DEV)
    runs = []
    for _ in range(2):
        loss = torch.nn.functional.cross_entropy(model(pairs, lengths, asked).flatten(0, 1), values.flatten())
        named = [(n, p) for n, p in model.named_parameters() if n != "embed"]  # torch's gather sums in no fixed order
        runs.append(torch.autograd.grad(loss, [p for _, p in named]))
    for a, b, (n, p) in zip(*runs, named):
        assert a.shape == p.shape and bool(torch.isfinite(a).all()) and torch.equal(a, b), n

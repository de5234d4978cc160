"""A gated delta layer trained on an associative recall task, then decoded token by token.

    python examples/gated_delta_layer.py [--steps 150] [--graph]

Each sequence lists key-value pairs and then asks for the values of some of the keys; the layer has to write the pairs
into its state and read them back.  Training runs layer_norm_fwd, gated_delta_fwd and their gradients inside autograd
functions; decoding runs one gated_delta_fwd over the prompt, which hands on its state, and then one gated_delta_step and
the norms for each token, optionally replayed from a CUDA graph.  The projections are plain matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import causal_linear_attention_phi_gb300 as la


class Norm(torch.autograd.Function):
    """Layer norm over the last dimension."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = la.layer_norm_fwd(x, weight, bias, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        return la.layer_norm_bwd(x, weight, mean, rstd, dy.contiguous())


class Delta(torch.autograd.Function):
    """The gated delta rule from the zero state."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return la.gated_delta_fwd(q, k, v, g, beta)

    @staticmethod
    def backward(ctx, do):
        return la.gated_delta_bwd(*ctx.saved_tensors, do.contiguous())


class Layer(torch.nn.Module):
    """x + W_o norm(delta(W_q n, W_k n, W_v n, gates(n))) with n = norm(x); q and k of unit length."""

    def __init__(self, width, heads, head, dtype=torch.bfloat16):
        super().__init__()
        self.heads, self.head = heads, head
        lin = lambda i, o, s=1.0: torch.nn.Parameter((s * i ** -0.5 * torch.randn(i, o)).to(dtype))
        one = lambda n, x: torch.nn.Parameter(torch.full((n,), x, dtype=dtype))
        inner = heads * head
        self.w_in = lin(width, 3 * inner)
        self.w_gate = lin(width, 2 * heads, 0.1)
        self.w_out = lin(inner, width)
        self.n_w, self.n_b = one(width, 1.0), one(width, 0.0)
        self.h_w, self.h_b = one(head, 1.0), one(head, 0.0)

    def inputs(self, x):
        """q, k, v [B,H,N,D] and g, beta [B,H,N] of the normed x [B,N,width]."""
        n = Norm.apply(x, self.n_w, self.n_b)
        B, N, _ = x.shape
        q, k, v = (n @ self.w_in).view(B, N, 3, self.heads, self.head).permute(2, 0, 3, 1, 4)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype).contiguous()
        gates = (n @ self.w_gate).view(B, N, 2, self.heads).permute(2, 0, 3, 1).float()
        g = -torch.nn.functional.softplus(gates[0] - 4)
        return unit(q), unit(k), v.contiguous(), g.to(x.dtype).contiguous(), torch.sigmoid(gates[1] + 1).to(
            x.dtype).contiguous()

    def output(self, x, o):
        o = Norm.apply(o, self.h_w, self.h_b)
        return x + o.transpose(1, 2).reshape(*x.shape[:2], -1) @ self.w_out

    def forward(self, x):
        return self.output(x, Delta.apply(*self.inputs(x)))

    def prefill(self, x):
        """The output over a prompt and the state to decode on from."""
        o, S = la.gated_delta_fwd(*self.inputs(x), return_state=True)
        return self.output(x, o), S

    def step(self, x, S):
        """One token x [B,1,width]; S is updated in place."""
        o = la.gated_delta_step(*(t[:, :, 0].contiguous() for t in self.inputs(x)), S)
        return self.output(x, o[:, :, None].contiguous())


class Model(torch.nn.Module):
    def __init__(self, tokens, width=128, heads=2, head=64, layers=2, dtype=torch.bfloat16):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(tokens, width).to(dtype))
        self.layers = torch.nn.ModuleList(Layer(width, heads, head, dtype) for _ in range(layers))
        self.f_w = torch.nn.Parameter(torch.ones(width, dtype=dtype))
        self.f_b = torch.nn.Parameter(torch.zeros(width, dtype=dtype))
        self.head = torch.nn.Parameter((width ** -0.5 * torch.randn(width, tokens)).to(dtype))

    def logits(self, x):
        return (Norm.apply(x, self.f_w, self.f_b) @ self.head).float()

    def embedded(self, tokens):
        """Each token's vector with the one before it, half a width on: the pairs' keys are then beside their values."""
        e = self.embed[tokens]
        before = torch.cat((torch.zeros_like(e[:, :1]), e[:, :-1]), 1)
        return (e + before.roll(e.shape[-1] // 2, -1)).contiguous()

    def forward(self, tokens):
        x = self.embedded(tokens)
        for layer in self.layers:
            x = layer(x)
        return self.logits(x)


def recall_batch(B, pairs, keys, asks, gen, device):
    """Tokens [B, 2 pairs + 2 asks]: k v k v ... then key, value of `asks` of them again; the values are the targets."""
    k = torch.stack([torch.randperm(keys, generator=gen)[:pairs] for _ in range(B)])
    v = keys + torch.randint(keys, (B, pairs), generator=gen)
    pick = torch.stack([torch.randperm(pairs, generator=gen)[:asks] for _ in range(B)])
    ask = torch.stack((k.gather(1, pick), v.gather(1, pick)), -1).flatten(1)
    return torch.cat((torch.stack((k, v), -1).flatten(1), ask), 1).to(device)


def train(model, steps, gen, device, pairs=24, keys=48, asks=8, B=64, lr=3e-3):
    """The losses of the steps: cross entropy of the asked values (fp32 master weights under bf16 parameters)."""
    params = list(model.parameters())
    master = [p.detach().float().requires_grad_(True) for p in params]
    opt = torch.optim.Adam(master, lr=lr, betas=(0.9, 0.98))
    losses = []
    for _ in range(steps):
        tokens = recall_batch(B, pairs, keys, asks, gen, device)
        out = model(tokens[:, :-1].contiguous())
        at = torch.arange(2 * pairs, tokens.shape[1] - 1, 2, device=device)  # the asked keys
        loss = torch.nn.functional.cross_entropy(out[:, at].flatten(0, 1), tokens[:, at + 1].flatten())
        loss.backward()
        for m, p in zip(master, params):
            m.grad, p.grad = p.grad.float(), None
        opt.step()
        with torch.no_grad():
            for m, p in zip(master, params):
                p.copy_(m)
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def decode(model, tokens, prompt, graph=False):
    """Logits at every position from `prompt` on, one token at a time after one pass over the prompt."""
    e = model.embedded(tokens)
    x, states = e[:, :prompt].contiguous(), []
    for layer in model.layers:
        x, S = layer.prefill(x)
        states.append(S)
    outs = [model.logits(x[:, -1:].contiguous())]
    slot = e[:, prompt:prompt + 1].clone() if prompt < e.shape[1] else None

    def one():
        x = slot
        for layer, S in zip(model.layers, states):
            x = layer.step(x, S)
        return model.logits(x)

    replay = None
    if graph and slot is not None:
        kept = [S.clone() for S in states]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            one()  # warm-up: libraries initialise before the capture
        torch.cuda.current_stream().wait_stream(side)
        for S, was in zip(states, kept):
            S.copy_(was)
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            captured = one()
    for t in range(prompt, e.shape[1]):
        slot.copy_(e[:, t:t + 1])
        if replay:
            replay.replay()
            outs.append(captured.clone())
        else:
            outs.append(one())
    return torch.cat(outs, 1)


def main(steps=150, graph=False, device="cuda:0", seed=0):
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = Model(96).to(device)
    losses = train(model, steps, gen, device)
    tokens = recall_batch(16, 24, 48, 8, gen, device)[:, :-1].contiguous()
    with torch.no_grad():
        full = model(tokens)
    stepped = decode(model, tokens, 48, graph)
    tail = full[:, 47:]
    return dict(first_loss=losses[0], last_loss=sum(losses[-10:]) / len(losses[-10:]),
                decode_error=float((stepped - tail).abs().max() / tail.abs().max()),
                losses=losses)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--graph", action="store_true")
    a = ap.parse_args()
    r = main(a.steps, a.graph)
    print("loss %.3f -> %.3f over %d steps; decoding against the whole sequence: max relative difference %.2e"
          % (r["first_loss"], r["last_loss"], a.steps, r["decode_error"]))

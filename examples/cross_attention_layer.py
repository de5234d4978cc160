"""A decoder that looks up values in a padded memory through cross attention, trained, then run token by token.

    python examples/cross_attention_layer.py [--steps 100]

The memory of each batch entry lists a number of key-value pairs of its own; the queries are keys of those pairs in another order
and of another number, and the targets their values.  A layer is

    x, n = residual_norm(x, a, scale)        the sum with the layer before's output, and the norm of it
    o    = cross(W_q n, W_k m, W_v m)        queries' heads share heads of keys; lengths cut the padding off
    a    = W_o gated_norm(o, W_g n)          the heads' norm with its gate, heads merged

and every part runs through this library forward and backward.  Decoding keeps each layer's state (S, z) of the memory and calls
cross_apply for one token at a time.  The projections are plain matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import causal_linear_attention_phi_gb300 as la


class Cross(torch.autograd.Function):
    """Cross attention; the forward's state is kept for the gradient."""

    @staticmethod
    def forward(ctx, q, k, v, lengths):
        o, S, z = la.cross_fwd(q, k, v, lengths=lengths, return_state=True)
        ctx.save_for_backward(q, k, v, lengths, S, z)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, lengths, S, z = ctx.saved_tensors
        return (*la.cross_bwd(q, k, v, do.contiguous(), lengths=lengths, S=S, z=z), None)


class GatedNorm(torch.autograd.Function):
    """The norm of each head with its gate, heads merged."""

    @staticmethod
    def forward(ctx, o, gate, weight):
        ctx.save_for_backward(o, gate, weight)
        return la.gated_norm_fwd(o, gate, weight, rms=True)

    @staticmethod
    def backward(ctx, dy):
        return la.gated_norm_bwd(*ctx.saved_tensors, dy.contiguous(), rms=True)


class ResidualNorm(torch.autograd.Function):
    """h = x + scale a and the layer norm of h."""

    @staticmethod
    def forward(ctx, x, a, scale, weight, bias):
        h, y, mean, rstd = la.residual_norm_fwd(x, a, scale, weight, bias, return_stats=True)
        ctx.save_for_backward(h, a, scale, weight, mean, rstd)
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        h, a, scale, weight, mean, rstd = ctx.saved_tensors
        return la.residual_norm_bwd(h, a, scale, weight, mean, rstd, dy.contiguous(), dh.contiguous())


class Layer(torch.nn.Module):
    def __init__(self, width, heads, key_heads, head, dtype):
        super().__init__()
        self.heads, self.key_heads, self.head = heads, key_heads, head
        lin = lambda i, o: torch.nn.Parameter((i ** -0.5 * torch.randn(i, o)).to(dtype))
        full = lambda n, x: torch.nn.Parameter(torch.full((n,), x, dtype=dtype))
        self.w_q, self.w_kv = lin(width, heads * head), lin(width, 2 * key_heads * head)
        self.w_gate, self.w_out = lin(width, heads * head), lin(heads * head, width)
        self.scale, self.n_w, self.n_b = full(width, 0.5), full(width, 1.0), full(width, 0.0)
        self.h_w = full(head, 1.0)

    def keys(self, memory):
        """k, v [B,Hk,M,D] of the memory [B,M,width]."""
        B, M, _ = memory.shape
        kv = (memory @ self.w_kv).view(B, M, 2, self.key_heads, self.head).permute(2, 0, 3, 1, 4).contiguous()
        return kv[0], kv[1]

    def queries(self, n):
        return (n @ self.w_q).view(*n.shape[:2], self.heads, self.head).transpose(1, 2).contiguous()

    def output(self, o, n):
        return GatedNorm.apply(o, n @ self.w_gate, self.h_w) @ self.w_out

    def forward(self, x, a, memory, lengths):
        x, n = ResidualNorm.apply(x, a, self.scale, self.n_w, self.n_b)
        return x, self.output(Cross.apply(self.queries(n), *self.keys(memory), lengths), n)

    def state(self, memory, lengths):
        """The state of a memory, from which `step` answers."""
        k, v = self.keys(memory)
        none = k.new_empty(k.shape[0], self.heads, 0, self.head)
        return la.cross_fwd(none, k, v, lengths=lengths, return_state=True)[1:]

    def step(self, x, a, state):
        """One token, x and a [B,1,width]."""
        x, n = ResidualNorm.apply(x, a, self.scale, self.n_w, self.n_b)
        o = la.cross_apply(self.queries(n)[:, :, 0].contiguous(), *state)
        return x, self.output(o[:, :, None].contiguous(), n)


class Model(torch.nn.Module):
    def __init__(self, tokens, width=128, heads=4, key_heads=2, head=64, layers=2, dtype=torch.bfloat16):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(tokens, width).to(dtype))
        self.layers = torch.nn.ModuleList(Layer(width, heads, key_heads, head, dtype) for _ in range(layers))
        self.f_scale, self.f_w = (torch.nn.Parameter(torch.ones(width, dtype=dtype)) for _ in range(2))
        self.f_b = torch.nn.Parameter(torch.zeros(width, dtype=dtype))
        self.head = torch.nn.Parameter((width ** -0.5 * torch.randn(width, tokens)).to(dtype))

    def memory(self, pairs):
        """[B,M,2] tokens: a key's vector beside its value's, half a width on."""
        e = self.embed[pairs]
        return (e[:, :, 0] + e[:, :, 1].roll(e.shape[-1] // 2, -1)).contiguous()

    def logits(self, x, a):
        return (ResidualNorm.apply(x, a, self.f_scale, self.f_w, self.f_b)[1] @ self.head).float()

    def forward(self, pairs, lengths, asked):
        m, x = self.memory(pairs), self.embed[asked]
        a = torch.zeros_like(x)
        for layer in self.layers:
            x, a = layer(x, a, m, lengths)
        return self.logits(x, a)

    @torch.no_grad()
    def decode(self, pairs, lengths, asked):
        """The same logits, one asked token at a time from the layers' kept states."""
        m = self.memory(pairs)
        states, outs = [layer.state(m, lengths) for layer in self.layers], []
        for t in range(asked.shape[1]):
            x = self.embed[asked[:, t:t + 1]].contiguous()
            a = torch.zeros_like(x)
            for layer, state in zip(self.layers, states):
                x, a = layer.step(x, a, state)
            outs.append(self.logits(x, a))
        return torch.cat(outs, 1)


def lookup_batch(B, most, asks, keys, gen, device):
    """Pairs [B,most,2], lengths [B] (the first is `most`), asked keys [B,asks] of the pairs that count, their values."""
    k = torch.stack([torch.randperm(keys, generator=gen)[:most] for _ in range(B)])
    v = keys + torch.randint(keys, (B, most), generator=gen)
    n = torch.randint(1, most + 1, (B,), generator=gen)
    n[0] = most
    pick = (torch.rand(B, asks, generator=gen) * n[:, None]).long()
    out = torch.stack((k, v), -1), n.to(torch.int32), k.gather(1, pick), v.gather(1, pick)
    return tuple(t.to(device) for t in out)


def train(model, steps, gen, device, B=64, most=20, asks=24, keys=40, lr=3e-3):
    """The losses of the steps (fp32 master weights under the parameters)."""
    params = list(model.parameters())
    master = [p.detach().float().requires_grad_(True) for p in params]
    opt = torch.optim.Adam(master, lr=lr, betas=(0.9, 0.98))
    losses = []
    for _ in range(steps):
        pairs, lengths, asked, values = lookup_batch(B, most, asks, keys, gen, device)
        loss = torch.nn.functional.cross_entropy(model(pairs, lengths, asked).flatten(0, 1), values.flatten())
        loss.backward()
        for m, p in zip(master, params):
            m.grad, p.grad = p.grad.float(), None
        opt.step()
        with torch.no_grad():
            for m, p in zip(master, params):
                p.copy_(m)
        losses.append(float(loss.detach()))
    return losses


def main(steps=100, device="cuda:0", seed=0):
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = Model(80).to(device)
    losses = train(model, steps, gen, device)
    pairs, lengths, asked, _ = lookup_batch(16, 20, 24, 40, gen, device)
    with torch.no_grad():
        full = model(pairs, lengths, asked)
    stepped = model.decode(pairs, lengths, asked)
    return dict(losses=losses, decode_error=float((stepped - full).abs().max() / full.abs().max()))


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    r = main(ap.parse_args().steps)
    print("loss %.3f -> %.3f over %d steps; decoding against the whole pass: max relative difference %.2e" %
          (r["losses"][0], r["losses"][-1], len(r["losses"]), r["decode_error"]))

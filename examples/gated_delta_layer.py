"""Layers of the gated delta rule, trained and then decoded from.

Each layer is the entry norm (residual addition and root-mean-square norm), plain
projections to q, k, v and the two gates, the gated delta rule and an output
projection:

    y, stream = add_rms_norm(out of the layer before, residual=stream)
    o = delta rule(unit(silu(y Wq)), unit(silu(y Wk)), y Wv; g, beta)
    out = o Wo

A token enters as the sum of its own embedding and one of the token before it, so that a
layer can write "after a comes b" and read it back when a returns.

``train`` takes optimizer steps through delta_backward and add_rms_norm_backward;
``prefill`` runs prompts of different lengths and keeps each layer's final states;
``decode`` takes one token per request with delta_step, which updates the states in
their slots.  Run as ``python examples/gated_delta_layer.py`` on a GB300: it trains on
sequences whose second half repeats the first (guessing costs ln 64 = 4.16), then checks
that decoding token by token gives what the whole sequence gives.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_mamba_gb300 import delta, norm  # noqa: E402

EPS = 1e-5


class AddRmsNorm(torch.autograd.Function):
    """(x, residual, weight) -> (y, stream); one gradient serves x and the residual."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, stream = norm.add_rms_norm(x, weight, EPS, residual=residual)
        ctx.save_for_backward(stream, weight)
        return y, stream

    @staticmethod
    def backward(ctx, dy, d_stream):
        stream, weight = ctx.saved_tensors
        dx, dw = norm.add_rms_norm_backward(dy.contiguous(), stream, weight, EPS,
                                            d_stream=None if d_stream is None else d_stream.contiguous())
        return dx, dx, dw


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return delta.delta_forward(q, k, v, g, beta, return_final_state=False)[0]

    @staticmethod
    def backward(ctx, do):
        d = delta.delta_backward(*ctx.saved_tensors, do.contiguous(), want_d_init=False)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"]


class Layer(torch.nn.Module):
    def __init__(self, width, heads, groups, headdim, dstate):
        super().__init__()
        self.heads, self.groups, self.headdim, self.dstate = heads, groups, headdim, dstate
        self.sizes = [groups * dstate, groups * dstate, heads * headdim, heads, heads]
        self.weight = torch.nn.Parameter(torch.ones(width))
        self.inward = torch.nn.Parameter(torch.randn(sum(self.sizes), width) * width ** -0.5)
        self.outward = torch.nn.Parameter(torch.randn(width, heads * headdim) * (heads * headdim) ** -0.5)

    def project(self, y):
        """q, k [.., G, N], v [.., H, P] in bf16 and the gates [.., H] in fp32 of the normed rows y [.., width]."""
        q, k, v, a, b = (y @ self.inward.to(y.dtype).T).split(self.sizes, -1)
        lead = y.shape[:-1]

        def unit(x):
            return F.normalize(F.silu(x.float()).reshape(*lead, self.groups, self.dstate), dim=-1).bfloat16()

        return (unit(q), unit(k), v.reshape(*lead, self.heads, self.headdim).contiguous(),
                -F.softplus(a.float() - 4.0), torch.sigmoid(b.float()))

    def out(self, o):
        return o.flatten(-2) @ self.outward.to(o.dtype).T


def shifted(tokens):  # the token before each (of the first, itself)
    return torch.cat([tokens[:, :1], tokens[:, :-1]], 1)


def per_head(x):  # gates [b, L, H] as the kernels take them
    return x.transpose(1, 2).contiguous()


class Model(torch.nn.Module):
    def __init__(self, vocab=64, width=256, layers=2, heads=4, groups=2, headdim=64, dstate=64):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(2, vocab, width))
        self.layers = torch.nn.ModuleList(Layer(width, heads, groups, headdim, dstate) for _ in range(layers))
        self.weight = torch.nn.Parameter(torch.ones(width))
        self.head = torch.nn.Parameter(torch.randn(vocab, width) * width ** -0.5)

    def enter(self, tokens, before):
        return (F.embedding(tokens, self.embed[0]) + F.embedding(before, self.embed[1])).bfloat16()

    def forward(self, tokens):
        """Logits [b, L, vocab], differentiable."""
        x = self.enter(tokens, shifted(tokens))
        stream = torch.zeros_like(x)
        for layer in self.layers:
            y, stream = AddRmsNorm.apply(x, stream, layer.weight)
            q, k, v, g, beta = layer.project(y)
            x = layer.out(DeltaRule.apply(q, k, v, per_head(g), per_head(beta)))
        y, _ = AddRmsNorm.apply(x, stream, self.weight)
        return (y @ self.head.to(y.dtype).T).float()

    @torch.no_grad()
    def prefill(self, tokens, lengths):
        """Logits of the prompts tokens [b, L], of which lengths int32 [b] count, and every layer's states [b, H, P, N]."""
        x, stream, states = self.enter(tokens, shifted(tokens)), None, []
        for layer in self.layers:
            y, stream = norm.add_rms_norm(x, layer.weight, EPS, residual=stream)
            q, k, v, g, beta = layer.project(y)
            o, state = delta.delta_forward(q, k, v, per_head(g), per_head(beta), valid_len=lengths)
            states.append(state)
            x = layer.out(o)
        y, _ = norm.add_rms_norm(x, self.weight, EPS, residual=stream)
        return (y @ self.head.to(y.dtype).T).float(), states

    @torch.no_grad()
    def decode(self, tokens, before, states, slots=None, e4m3=False):
        """Logits [b, vocab] of one more token per request, `before` being those they follow; states are
        updated in their slots.  ``e4m3`` takes every layer's projections from the norm's 8-bit output and its scales."""
        x, stream = self.enter(tokens, before), None
        for layer, state in zip(self.layers, states):
            if e4m3:
                y8, scale, stream = norm.add_rms_norm_fp8(x, layer.weight, EPS, residual=stream)
                y = (y8.float() * scale).bfloat16()
            else:
                y, stream = norm.add_rms_norm(x, layer.weight, EPS, residual=stream)
            x = layer.out(delta.delta_step(*layer.project(y), state, state_index=slots))
        y, _ = norm.add_rms_norm(x, self.weight, EPS, residual=stream)
        return (y @ self.head.to(y.dtype).T).float()


def train(model, steps, batch=16, length=128, seed=0):
    """Cross entropy of the second half of sequences that repeat their first half; returns each step's loss."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        half = torch.randint(model.embed.shape[1], (batch, length // 2), generator=gen, device="cuda")
        tokens = torch.cat([half, half], 1)
        logits = model(tokens)[:, length // 2 - 1:-1]
        loss = F.cross_entropy(logits.flatten(0, 1), half.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(x) for x in losses]


def decode_error(model, lengths=(70, 1, 129), more=9, seed=1, e4m3=False):
    """Prefill, then `more` decoded tokens in a larger pool of slots, against the whole sequences:
    the norm of the logits' difference over that of the logits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, longest = len(lengths), max(lengths)
    tokens = torch.randint(model.embed.shape[1], (b, longest + more), generator=gen, device="cuda")
    with torch.no_grad():
        whole = model(tokens)
    _, states = model.prefill(tokens[:, :longest].contiguous(), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    slots = torch.arange(b, dtype=torch.int32, device="cuda").flip(0) * 2  # requests keep their slots in any order
    pools = []
    for state in states:
        pool = torch.zeros(2 * b, *state.shape[1:], device="cuda")
        pool[slots.long()] = state
        pools.append(pool)
    rows, wrong, size = torch.arange(b, device="cuda"), 0.0, 0.0
    for t in range(more):
        at = torch.tensor(lengths, device="cuda") + t
        got, ref = model.decode(tokens[rows, at], tokens[rows, at - 1], pools, slots, e4m3), whole[rows, at]
        wrong += float((got - ref).square().sum())
        size += float(ref.square().sum())
    return (wrong / size) ** 0.5


def main(steps=200):
    torch.manual_seed(0)
    model = Model().cuda()
    losses = train(model, steps)
    for i in range(0, steps, max(1, steps // 8)):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    print(f"step {steps - 1:4d}  loss {losses[-1]:.3f}")
    print(f"decoding against whole sequences: relative difference {decode_error(model):.1e}, "
          f"with 8-bit rows {decode_error(model, e4m3=True):.1e}")


if __name__ == "__main__":
    main()

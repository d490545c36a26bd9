"""Trains a small language model whose activations wait for the backward pass in
8 bits, with every gradient made by libmuon's training operators and every
parameter updated by its Muon and AdamW steps.

    python examples/train_act8.py --steps 60

The model reads one token and predicts the next: embedding, residual blocks of
RMS norm and gated unit, a final norm and an output head.  The data is a fixed
random walk over the vocabulary (each word has a few successors).  Per block the
forward pass keeps n8 and rstd of the norm and the 8-bit gate and up: one byte a
value where bfloat16 takes two.  Matrices of the blocks go to muon_step; embedding,
head and gains to adamw_step.

The first step's gradients are compared with those of the same model in torch
autograd, in float32 from the same weights: they differ by the roundings of
bfloat16 and of the 8-bit activations.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_aware_optimizer_libmuon_amd as muon  # noqa: E402

DEV = "cuda"


class Model:
    """Float32 parameters and the bfloat16 copies that the products take."""

    def __init__(self, vocab, dim, inner, blocks, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.embed_scale = dim ** 0.5
        self.table = rand(vocab, dim) / self.embed_scale
        self.head = rand(vocab, dim) / self.embed_scale
        self.gate_up = [rand(2 * inner, dim) / dim ** 0.5 for _ in range(blocks)]     # gate's rows, then up's
        self.down = [rand(dim, inner) / (blocks * inner) ** 0.5 for _ in range(blocks)]
        self.gains = [torch.ones(dim, device=DEV) for _ in range(blocks + 1)]
        self.inner = inner

    def matrices(self):
        return [w for pair in zip(self.gate_up, self.down) for w in pair]

    def others(self):
        return [self.table, self.head, *self.gains]


def loss_and_grad(logits, targets):
    """Mean cross-entropy and its gradient."""
    logits = logits.float()
    logits = logits - logits.amax(1, keepdim=True)
    p = torch.exp(logits)
    p = p / p.sum(1, keepdim=True)
    rows = torch.arange(len(targets), device=DEV)
    loss = -torch.log(p[rows, targets]).mean()
    p[rows, targets] -= 1.0
    return loss, (p / len(targets)).bfloat16()


def step_gradients(m, tokens, targets):
    """Loss and the gradients of m.matrices() and m.others()."""
    bf = torch.bfloat16
    x = muon.embed(m.table, tokens, scale=m.embed_scale)
    delta, saved = None, []
    for gu_w, down_w, gain in zip(m.gate_up, m.down, m.gains):
        x, y, n8, rstd = muon.rmsnorm_act8(x, gain, residual=delta)
        gu = y @ gu_w.to(bf).t()
        a, gate8, up8 = muon.swiglu_act8(gu[:, :m.inner], gu[:, m.inner:])
        delta = a @ down_w.to(bf).t()
        saved.append((n8, rstd, gate8, up8))
    _, y, n8, rstd = muon.rmsnorm_act8(x, m.gains[-1], residual=delta)
    loss, dlogits = loss_and_grad(y @ m.head.to(bf).t(), targets)

    # backward: n8 with the gain folded in is the input of the layer behind a norm
    d_head = muon.act8_wgrad(dlogits, n8, col_gain=m.gains[-1])
    dx, dgain = muon.rmsnorm_act8_grad(dlogits @ m.head.to(bf), n8, rstd, m.gains[-1])
    d_mats, d_gains = [], [dgain]
    for gu_w, down_w, gain, (n8, rstd, gate8, up8) in reversed(list(zip(m.gate_up, m.down, m.gains, saved))):
        dgu = torch.empty(len(tokens), 2 * m.inner, device=DEV, dtype=bf)
        _, _, a8 = muon.swiglu_act8_grad(dx @ down_w.to(bf), gate8, up8, dgate=dgu[:, :m.inner], dup=dgu[:, m.inner:])
        d_down = muon.act8_wgrad(dx, a8)
        d_gu = muon.act8_wgrad(dgu, n8, col_gain=gain)
        dx, dgain = muon.rmsnorm_act8_grad(dgu @ gu_w.to(bf), n8, rstd, gain, dres=dx)
        d_mats[:0] = [d_gu, d_down]
        d_gains.insert(0, dgain)
    d_table = muon.embed_grad(dx, tokens, m.table.shape[0], scale=m.embed_scale)
    return loss, d_mats, [d_table, d_head, *d_gains]


def autograd_gradients(m, tokens, targets):
    """The same in float32 by torch autograd."""
    params = [p.clone().requires_grad_() for p in m.matrices() + m.others()]
    mats, (table, head, *gains) = params[:len(m.matrices())], params[len(m.matrices()):]
    norm = lambda h, g: h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * g  # noqa: E731
    x = table[tokens] * m.embed_scale
    for gu_w, down_w, gain in zip(mats[::2], mats[1::2], gains):
        gate, up = (norm(x, gain) @ gu_w.t()).chunk(2, dim=1)
        x = x + gate * torch.sigmoid(gate) * up @ down_w.t()
    loss = torch.nn.functional.cross_entropy(norm(x, gains[-1]) @ head.t(), targets)
    loss.backward()
    return loss.detach(), [p.grad for p in params]


def walk(vocab, tokens, seed):
    """(tokens, next tokens): each word is followed by one of two others."""
    g = torch.Generator(device=DEV).manual_seed(1)
    after = torch.randint(0, vocab, (vocab, 2), generator=g, device=DEV)
    g.manual_seed(1000 + seed)
    t = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    return t, after[t, torch.randint(0, 2, (tokens,), generator=g, device=DEV)]


def train(steps=60, vocab=1000, dim=256, inner=768, blocks=2, tokens=4096, lr=0.02, say=print):
    m = Model(vocab, dim, inner, blocks)
    mats, others = m.matrices(), m.others()
    moms = [torch.zeros_like(w) for w in mats]
    first = [torch.zeros_like(p) for p in others]
    second = [torch.zeros_like(p) for p in others]
    ws, aws = muon.alloc_workspace([w.shape for w in mats], DEV), muon.alloc_adamw_workspace(len(others), DEV)
    losses, worst = [], 0.0
    for s in range(steps):
        t, nxt = walk(vocab, tokens, s)
        loss, d_mats, d_others = step_gradients(m, t, nxt)
        if s == 0:
            _, ref = autograd_gradients(m, t, nxt)
            off = [float((a - b).norm() / b.norm()) for a, b in zip(d_mats + d_others, ref)]
            worst = max(off)
            say(f"gradients against float32 autograd, relative: {min(off):.4f} to {worst:.4f}")
        muon.muon_step(mats, d_mats, moms, lr=lr, mu=0.95, wd=0.01, rms_scale="sqrt_max1", workspace=ws)
        muon.adamw_step(others, d_others, first, second, [s + 1] * len(others), lr=3e-3, wd=0.0, workspace=aws)
        losses.append(loss)
        if s % 10 == 0 or s == steps - 1:
            say(f"step {s:4d}  loss {float(loss):.4f}")
    return [float(v) for v in losses], worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=4096)
    a = ap.parse_args()
    train(steps=a.steps, tokens=a.tokens, say=lambda *x: print(*x, flush=True))

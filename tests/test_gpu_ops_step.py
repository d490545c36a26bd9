"""Attention and the losses used as a training step uses them: together with the
library's other operators and steps, captured, on another stream, in debug mode."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from tests.gpu_helpers import DEV
from tests.test_gpu_ops import gen, randn

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# ------------------------------------------------- a block with attention ----
def model(seed, vocab=500, dim=256, heads=4, kv=2):
    d = dim // heads
    w = {"table": randn(seed, vocab, dim), "gain": 1 + 0.1 * randn(seed + 1, dim), "qkv": randn(seed + 2, (heads + 2 * kv) * d, dim) / 16,
         "out": randn(seed + 3, dim, dim) / 16, "head": randn(seed + 4, vocab, dim) / 16}
    return {k: v.to(DEV) for k, v in w.items()}, dict(heads=heads, kv=kv, d=d)


def step_gradients(w, sizes, tokens, starts, loss_of):
    """Forward and backward pass through the library's operators; loss_of(logits) gives (loss, dlogits)."""
    h, kv, d = sizes["heads"], sizes["kv"], sizes["d"]
    x = muon.embed(w["table"], tokens)
    _, y, n8, rstd = muon.rmsnorm_act8(x, w["gain"])
    qkv = (y @ w["qkv"].to(BF).t()).view(len(tokens), h + 2 * kv, d)
    q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    o, lse = muon.attention(q, k, v, starts=starts)
    flat = o.view(len(tokens), h * d)
    x2 = x + flat @ w["out"].to(BF).t()
    logits = x2 @ w["head"].to(BF).t()
    loss, dlogits = loss_of(logits)
    grads = {"head": muon.act8_wgrad(dlogits, muon.act8_pack(x2))}
    dx2 = dlogits @ w["head"].to(BF)
    grads["out"] = muon.act8_wgrad(dx2, muon.act8_pack(flat))
    do = (dx2 @ w["out"].to(BF)).view(len(tokens), h, d)
    dqkv = torch.empty_like(qkv)
    muon.attention_grad(do, q, k, v, o, lse, starts=starts, dq=dqkv[:, :h], dk=dqkv[:, h:h + kv], dv=dqkv[:, h + kv:])
    dqkv = dqkv.view(len(tokens), -1)
    grads["qkv"] = muon.act8_wgrad(dqkv, n8, col_gain=w["gain"])
    dx, grads["gain"] = muon.rmsnorm_act8_grad(dqkv @ w["qkv"].to(BF), n8, rstd, w["gain"], dres=dx2)
    grads["table"] = muon.embed_grad(dx, tokens, len(w["table"]))
    return loss, grads


def autograd(w, sizes, tokens, lengths, loss_of):
    """The same in float32 by torch autograd."""
    h, kv, d = sizes["heads"], sizes["kv"], sizes["d"]
    p = {k: v.clone().requires_grad_() for k, v in w.items()}
    x = p["table"][tokens]
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * p["gain"]
    qkv = (y @ p["qkv"].t()).view(len(tokens), h + 2 * kv, d)
    rows, at = [], 0
    for n in lengths:
        part = qkv[at:at + n].transpose(0, 1)
        q, k, v = part[:h], part[h:h + kv].repeat_interleave(h // kv, 0), part[h + kv:].repeat_interleave(h // kv, 0)
        s = torch.stack([a @ b.t() for a, b in zip(q, k)]) * d ** -0.5
        s = s.masked_fill(torch.ones(n, n, device=DEV).triu(1).bool(), -float("inf"))
        pr = torch.softmax(s, -1)
        rows.append(torch.stack([a @ b for a, b in zip(pr, v)], 1))
        at += n
    flat = torch.cat(rows).reshape(len(tokens), h * d)
    logits = (x + flat @ p["out"].t()) @ p["head"].t()
    loss = loss_of(logits)
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("kind", ["distill", "policy"])
def test_gradients_of_a_block_and_its_loss(kind):
    """Against float32 autograd, relative to each gradient's norm.  Independent roundings on the way: bf16 (2^-8 at
    most, a third of it root mean square) of some ten tensors, and the 8-bit form's 2.7 % of the activations, once in
    each weight gradient and in the norm's: below 6 %."""
    w, sizes = model(3)
    lengths = [100, 1, 210, 64]
    n = sum(lengths)
    tokens = torch.randint(0, 500, (n,), generator=gen(1)).to(DEV)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32), device=DEV)
    weights = ((torch.rand(n, generator=gen(2)) < 0.8).float() / n).to(DEV)
    if kind == "distill":
        teacher, ids = torch.topk(3 * randn(5, n, 500), 16, dim=1)
        teacher, ids = teacher.to(DEV), ids.to(DEV)

        def own(z):
            loss, dz = muon.distill_loss(z, ids, teacher, temperature=2.0, weights=weights)
            return loss.sum(), dz

        def plain(z):
            p, logq = torch.softmax(teacher / 2, 1), torch.log_softmax(z / 2, 1).gather(1, ids)
            return (weights * 4 * (p * (torch.log(p) - logq)).sum(1)).sum()
    else:
        actions = torch.randint(0, 500, (n,), generator=gen(7)).to(DEV)
        adv, ref = randn(8, n).to(DEV), (-6.0 + 0.3 * randn(9, n)).to(DEV)
        old = torch.full((n,), -6.5, device=DEV)

        # a clip that holds nothing: a ratio near its border would decide otherwise in bf16
        def own(z):
            loss, _, dz = muon.policy_loss(z, actions, old, adv, ref_logp=ref, clip=1.0, clip_high=1e4, kl_coef=0.1, weights=weights)
            return loss.sum(), dz

        def plain(z):
            logp = torch.log_softmax(z, 1).gather(1, actions[:, None])[:, 0]
            r, d = torch.exp(logp - old), ref - logp
            return (weights * (-r * adv + 0.1 * (torch.exp(d) - d - 1))).sum()
    loss, grads = step_gradients(w, sizes, tokens, starts, own)
    ref_loss, ref_grads = autograd(w, sizes, tokens, lengths, plain)
    assert abs(float(loss) - float(ref_loss)) <= 0.02 * abs(float(ref_loss)) + 1e-3
    for name, g in grads.items():
        assert float((g - ref_grads[name]).norm()) <= 0.06 * float(ref_grads[name].norm()), name
    # and the steps take them
    mats = ["qkv", "out"]
    before = [w[m].clone() for m in mats]
    muon.muon_step([w[m] for m in mats], [grads[m] for m in mats], [torch.zeros_like(w[m]) for m in mats], lr=0.02)
    others = ["table", "head", "gain"]
    muon.adamw_step([w[m] for m in others], [grads[m] for m in others], [torch.zeros_like(w[m]) for m in others],
                    [torch.zeros_like(w[m]) for m in others], [1] * 3)
    assert all(torch.isfinite(v).all() for v in w.values()) and not any(torch.equal(a, w[m]) for a, m in zip(before, mats))


# ------------------------------------------- streams, graphs, debug mode ----
def inputs(seed, small):
    """Sizes that take one launch, or several with parts and joins."""
    n, nk, h, kv, d, vocab = (90, 90, 4, 2, 64, 900) if small else (2400, 2400, 4, 1, 128, 40000)
    t = dict(q=randn(seed, n, h, d, dtype=BF), k=randn(seed + 1, nk, kv, d, dtype=BF), v=randn(seed + 2, nk, kv, d, dtype=BF),
             do=randn(seed + 3, n, h, d, dtype=BF), starts=torch.tensor([0, n // 3, n], dtype=torch.int32), logits=randn(seed + 4, 60, vocab, dtype=BF),
             ids=torch.randint(-1, vocab, (60, 9), generator=gen(seed)), teacher=randn(seed + 5, 60, 9), act=torch.randint(0, vocab, (60,), generator=gen(seed + 6)),
             old=-8 + randn(seed + 7, 60), adv=randn(seed + 8, 60), ref=-8 + randn(seed + 9, 60), weights=torch.rand(60, generator=gen(seed + 10)))
    return {k: v.to(DEV) for k, v in t.items()}


def everything(t, **kw):
    o, lse = muon.attention(t["q"], t["k"], t["v"], starts=t["starts"], **kw)
    grads = muon.attention_grad(t["do"], t["q"], t["k"], t["v"], o, lse, starts=t["starts"], **kw)
    one, lse1 = muon.attention(t["q"][:20], t["k"], t["v"], causal=False, **kw)
    dis = muon.distill_loss(t["logits"], t["ids"], t["teacher"], temperature=1.5, weights=t["weights"], **kw)
    pol = muon.policy_loss(t["logits"], t["act"], t["old"], t["adv"], ref_logp=t["ref"], kl_coef=0.1, weights=t["weights"], **kw)
    return [o, lse, *grads, one, lse1, *dis, *pol]


@pytest.mark.parametrize("small", [True, False])
def test_graph_replays_match_eager_calls(small):
    sets = [inputs(s, small) for s in (10, 40, 70)]
    want = [[o.clone() for o in everything(t)] for t in sets]
    static = {k: v.clone() for k, v in sets[0].items()}
    everything(static)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                          # two graphs, with workspaces of their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = everything(static)
        graphs.append((g, outs))
    for t, w in list(zip(sets, want)) * 2:
        for k in static:
            static[k].copy_(t[k])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, w))
        eager = everything(t)                                   # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, w))


@pytest.mark.parametrize("small", [True, False])
def test_other_streams(small):
    t = inputs(20, small)
    want = everything(t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:                                           # both at once
        s.wait_stream(torch.cuda.current_stream())
        got.append(everything(t, stream=s))
    for s, g in zip(streams, got):
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    with torch.cuda.stream(streams[0]):
        inside = everything(t)
    streams[0].synchronize()
    assert all(torch.equal(a, b) for a, b in zip(inside, want))


def test_inputs_freed_after_a_call_on_another_stream():
    """A tensor dropped right after a call on another stream is not reused before that stream has read it."""
    s = torch.cuda.Stream()
    t = inputs(30, False)
    want = everything(t)
    torch.cuda.synchronize()
    for _ in range(3):
        u = {k: v.clone() for k, v in t.items()}
        s.wait_stream(torch.cuda.current_stream())
        got = everything(u, stream=s)
        shapes = [(v.shape, v.dtype) for v in u.values()]
        del u
        for shape, dtype in shapes:
            torch.ones(shape, device=DEV).to(dtype)             # would take the freed blocks
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("small", [True, False])
def test_debug_mode_gives_the_same(small, monkeypatch):
    """Under MUON_DEBUG the workspaces start as NaN: nothing is read that no kernel wrote."""
    t = inputs(50, small)
    want = everything(t)
    monkeypatch.setenv("MUON_DEBUG", "1")
    assert all(torch.equal(a, b) for a, b in zip(everything(t), want))


def test_no_autograd_history():
    t = inputs(60, True)
    for k in ("q", "k", "v", "logits"):
        t[k].requires_grad_()
    assert not any(o.requires_grad for o in everything(t) if o is not None)

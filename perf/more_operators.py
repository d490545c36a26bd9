"""The training operators between the projections and the loss, as cases to time and compare.

Attention over sequences of any lengths, with query heads that share key and
value heads, and its backward pass, which recomputes the probabilities from each
row's log-sum-exp; the distillation loss of a teacher's top logits and the
clipped policy loss with a KL term, each with the gradient of the logits.

Each case is a dict: "op" names the operator and its direction, the other
entries its sizes, types and options.  `own` selects the library's kernels;
otherwise `run` computes the same in elementary torch operations.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.25, 0.04


def listed():
    return [
        # two short sequences through a narrow block: only the calls' latency counts
        dict(name="attn_fwd_2x37_4h64", op="attn_fwd", seqs=2, tokens=74, ktokens=0, heads=4, kv=4, dim=64, causal=True),
        # an encoder's ragged batch: every token sees its whole sequence, heads of 80 columns
        dict(name="attn_fwd_10010_16h80", op="attn_fwd", seqs=23, tokens=10010, ktokens=0, heads=16, kv=16, dim=80, causal=False),
        # a training batch of 16 K tokens at width 4096, four query heads to a key and value head
        dict(name="attn_fwd_4x4096_32h128", op="attn_fwd", seqs=4, tokens=16384, ktokens=0, heads=32, kv=8, dim=128, causal=True),
        # backward: the short sequences,
        dict(name="attn_bwd_2x37_4h64", op="attn_bwd", seqs=2, tokens=74, ktokens=0, heads=4, kv=4, dim=64, causal=True),
        # a packed batch of ragged documents at width 768,
        dict(name="attn_bwd_12001_12h64", op="attn_bwd", seqs=9, tokens=12001, ktokens=0, heads=12, kv=12, dim=64, causal=True),
        # and the wide block's batch
        dict(name="attn_bwd_4x4096_32h128", op="attn_bwd", seqs=4, tokens=16384, ktokens=0, heads=32, kv=8, dim=128, causal=True),
        # evaluation of a few tokens' distillation: the loss alone
        dict(name="distill_fwd_37x1000", op="distill", tokens=37, vocab=1000, top=8, dtype="f32", ids="i64", masked=0.0, grad=False),
        # a ragged batch in 32 bits over a vocabulary that no vector load is aligned to, a third of it prompt tokens
        dict(name="distill_2049x50001_f32", op="distill", tokens=2049, vocab=50001, top=100, dtype="f32", ids="i32", masked=0.33,
             grad=True),
        # a training batch over the vocabulary of the library's embedding
        dict(name="distill_16384x32000", op="distill", tokens=16384, vocab=32000, top=64, dtype="bf16", ids="i64", masked=0.1,
             grad=True),
        # one token's policy gradient: latency
        dict(name="policy_1x32000", op="policy", tokens=1, vocab=32000, dtype="bf16", ids="i64", masked=0.0, ref=True, grad=True),
        # answers of a few rollouts over a large vocabulary
        dict(name="policy_1500x131072", op="policy", tokens=1500, vocab=131072, dtype="bf16", ids="i64", masked=0.2, ref=True,
             grad=True),
        # a batch of rollouts, the prompts masked
        dict(name="policy_16384x32000", op="policy", tokens=16384, vocab=32000, dtype="bf16", ids="i32", masked=0.3, ref=True,
             grad=True),
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; every other one a multiple of 32 where that fits."""
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    if rng.random() < 0.5 and -(-n // 32) * 32 <= hi:
        n = -(-n // 32) * 32
    return n


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "attn_bwd", "distill", "policy"])
    pick = lambda *v: rng.choice(v)  # noqa: E731
    while True:
        if op.startswith("attn"):
            kv = pick(1, 2, 4, 8, 12)
            tokens = _size(rng, 1, 16384)
            c = dict(op=op, seqs=min(tokens, _size(rng, 1, 32)), tokens=tokens, ktokens=0, heads=kv * pick(1, 1, 2, 4), kv=kv,
                     dim=pick(64, 128, 8 * rng.randint(2, 16)), causal=rng.random() < 0.6)
            if not c["causal"] and rng.random() < 0.4:       # queries over another sequence's keys
                c["ktokens"] = max(c["seqs"], _size(rng, 1, 8192))
            ok = c["heads"] <= 32 and c["heads"] * c["dim"] * _pairs(c) <= 32 * 128 * 4 * 4096 * 4097 // 2
        else:
            c = dict(op=op, tokens=_size(rng, 1, 16384), vocab=_size(rng, 200, 200000), dtype=pick("bf16", "bf16", "f32"),
                     ids=pick("i32", "i64"), masked=pick(0.0, 0.1, 0.5), grad=rng.random() < 0.75)
            if op == "distill":
                c["top"] = min(c["vocab"], _size(rng, 1, 256))
            else:
                c["ref"] = rng.random() < 0.7
            ok = c["tokens"] * c["vocab"] <= 16384 * 32000 * (2 if c["dtype"] == "bf16" else 1) // 2
        if ok:
            return c


def _lengths(tokens, seqs):
    """`tokens` cut into `seqs` lengths: equal where that comes out even, else uneven, the same for the same two numbers."""
    if tokens % seqs == 0:
        return [tokens // seqs] * seqs
    rng = random.Random(tokens * 1000003 + seqs)
    cuts = sorted(rng.sample(range(1, tokens), seqs - 1))
    return [b - a for a, b in zip([0, *cuts], [*cuts, tokens])]


def _spans(case):
    """(first query, queries, first key, keys) of each sequence."""
    nq = _lengths(case["tokens"], case["seqs"])
    nk = _lengths(case["ktokens"], case["seqs"]) if case["ktokens"] else nq
    out, q, k = [], 0, 0
    for a, b in zip(nq, nk):
        out.append((q, a, k, b))
        q, k = q + a, k + b
    return out


def _pairs(case):
    """Pairs of a query and a key that it sees, over the sequences."""
    return sum(a * (a + 1) // 2 if case["causal"] else a * b for _, a, _, b in _spans(case))


# ---------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _weights(g, case):
    """1 / (tokens that count), 0 for the others."""
    live = torch.rand(case["tokens"], generator=g, device=DEV) >= case["masked"]
    return live.float() / live.sum().clamp(min=1)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"].startswith("attn"):
        t, h, kv, d = case["tokens"], case["heads"], case["kv"], case["dim"]
        # queries and keys as a projection gives them: heads of different sharpness
        sharp = 2.0 ** torch.randint(-1, 2, (h, 1), generator=g, device=DEV)
        if case["ktokens"]:
            s["q"] = (_randn(g, t, h, d) * sharp).bfloat16()
            kvs = _randn(g, case["ktokens"], 2 * kv, d).bfloat16()
            s["k"], s["v"] = kvs[:, :kv], kvs[:, kv:]
        else:
            # slices of one projection's output
            qkv = _randn(g, t, h + 2 * kv, d)
            qkv[:, :h] *= sharp
            qkv = qkv.bfloat16()
            s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        spans = _spans(case)
        s["starts"] = _starts([n for _, n, _, _ in spans]) if case["seqs"] > 1 else None
        s["k_starts"] = _starts([n for _, _, _, n in spans]) if case["ktokens"] and case["seqs"] > 1 else None
        if case["op"] == "attn_bwd":
            out = _attend(s)
            s["o"], s["lse"] = out["o"], out["lse"]
            s["do"] = _randn(g, t, h, d).bfloat16()
        return s
    t, v = case["tokens"], case["vocab"]
    z = 2.5 * _randn(g, t, v)
    s["weights"] = _weights(g, case)
    if case["op"] == "distill":
        s["teacher"], ids = torch.topk(0.8 * z + _randn(g, t, v), case["top"], dim=1)
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        s["logits"] = z.to(TYPES[case["dtype"]])
        s["tau"] = 2.0
        return s
    s["logits"] = z.to(TYPES[case["dtype"]])
    z = s["logits"].float()
    # actions drawn from the policy
    ids = torch.argmax(z - torch.log(-torch.log(torch.rand(t, v, generator=g, device=DEV).clamp(1e-30, 1 - 1e-7))), dim=1)
    logp = z[torch.arange(t, device=DEV), ids] - torch.logsumexp(z, 1)
    s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
    # log ratios on a grid that avoids the clip's borders, where a rounding would decide between a gradient and none
    s["old"] = logp - torch.round(0.15 * 64 * _randn(g, t)) / 64
    s["adv"] = _randn(g, t)
    s["ref"] = logp + 0.3 * _randn(g, t) if case["ref"] else None
    return s


# ------------------------------------------------------------ plain form ----
def _visible(case, nq, nk):
    if not case["causal"]:
        return None
    i = torch.arange(nq, device=DEV)[:, None] + (nk - nq)
    return torch.arange(nk, device=DEV)[None, :] <= i


def _pieces(case):
    """Sequences, and groups of heads that are small enough to be worked on at once."""
    share = case["heads"] // case["kv"]
    for q0, nq, k0, nk in _spans(case):
        step = max(1, min(case["kv"], (1 << 30) // (nq * nk * share)))
        for j in range(0, case["kv"], step):
            m = min(step, case["kv"] - j)
            yield slice(q0, q0 + nq), slice(k0, k0 + nk), slice(j * share, (j + m) * share), slice(j, j + m)


def _by_head(x, share=1):
    """heads x tokens x columns, in 32 bits, each head `share` times."""
    return x.transpose(0, 1).float().repeat_interleave(share, dim=0).contiguous()


def _attend(s):
    c = s["case"]
    t, h, d = s["q"].shape
    share, scale = h // c["kv"], d ** -0.5
    o = torch.empty(t, h, d, device=DEV, dtype=torch.bfloat16)
    lse = torch.empty(h, t, device=DEV)
    for tq, tk, hq, hk in _pieces(c):
        q, k, v = _by_head(s["q"][tq, hq]), _by_head(s["k"][tk, hk], share), _by_head(s["v"][tk, hk], share)
        p = torch.matmul(q, k.transpose(1, 2).contiguous()) * scale
        seen = _visible(c, p.shape[1], p.shape[2])
        if seen is not None:
            p.masked_fill_(~seen, -math.inf)
        top = p.amax(-1, keepdim=True)
        p = torch.exp(p - top)
        total = p.sum(-1, keepdim=True)
        o[tq, hq] = (torch.matmul(p, v) / total).transpose(0, 1).bfloat16()
        lse[hq, tq] = (top + torch.log(total)).squeeze(-1)
    return dict(o=o, lse=lse)


def _attend_grad(s):
    c = s["case"]
    h, d = s["q"].shape[1:]
    share, scale = h // c["kv"], d ** -0.5
    dq, dk, dv = (torch.empty(x.shape, device=DEV, dtype=torch.bfloat16) for x in (s["q"], s["k"], s["v"]))
    for tq, tk, hq, hk in _pieces(c):
        q, k, v = _by_head(s["q"][tq, hq]), _by_head(s["k"][tk, hk], share), _by_head(s["v"][tk, hk], share)
        do, o = _by_head(s["do"][tq, hq]), _by_head(s["o"][tq, hq])
        p = torch.exp(torch.matmul(q, k.transpose(1, 2).contiguous()) * scale - s["lse"][hq, tq].unsqueeze(-1))
        seen = _visible(c, p.shape[1], p.shape[2])
        if seen is not None:
            p.masked_fill_(~seen, 0.0)
        ds = p * (torch.matmul(do, v.transpose(1, 2).contiguous()) - (do * o).sum(-1, keepdim=True)) * scale
        dq[tq, hq] = torch.matmul(ds, k).transpose(0, 1).bfloat16()
        # the heads that share a key and value head are summed
        for out, a, b in ((dk, ds, q), (dv, p, do)):
            g = torch.matmul(a.transpose(1, 2).contiguous(), b).view(-1, share, k.shape[1], d).sum(1)
            out[tk, hk] = g.transpose(0, 1).bfloat16()
    return dict(dq=dq, dk=dk, dv=dv)


def _softmax_parts(x):
    """exp(x - max) and the log of its sum, the sum in 64 bits."""
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    return e, total, top.double() + torch.log(total)


def _plain_distill(s):
    c, tau = s["case"], s["tau"]
    x = s["logits"].float() / tau
    ids, w = s["ids"].long(), s["weights"][:, None]
    t = s["teacher"].float() / tau
    t = t - t.amax(1, keepdim=True)
    logp = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    p = torch.exp(logp)
    e, total, lse = _softmax_parts(x)
    logq = x.gather(1, ids).double() - lse
    loss = w.double() * tau * tau * (p * (logp - logq)).sum(1, keepdim=True)
    out = dict(loss=loss.squeeze(1).float())
    if c["grad"]:
        g = e.div_(total.float()).scatter_add_(1, ids, -p)
        out["dlogits"] = g.mul_(w * tau).to(s["logits"].dtype)
    return out


def _plain_policy(s):
    c = s["case"]
    x = s["logits"].float()
    ids, w = s["ids"].long()[:, None], s["weights"].double()
    e, total, lse = _softmax_parts(x)
    logp = (x.gather(1, ids).double() - lse).squeeze(1)
    r, adv = torch.exp(logp - s["old"].double()), s["adv"].double()
    free, held = r * adv, r.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv
    loss = -torch.minimum(free, held)
    g = torch.where(free <= held, -free, torch.zeros_like(free))
    if s["ref"] is not None:
        d = s["ref"].double() - logp
        loss = loss + KL_COEF * (torch.expm1(d) - d)
        g = g - KL_COEF * torch.expm1(d)
    # tokens of weight 0 take no part: their log-probabilities are 0 like their losses
    out = dict(loss=(w * loss).float(), logp=torch.where(w != 0, logp, torch.zeros_like(logp)).float())
    if c["grad"]:
        g = (w * g)[:, None].float()
        p = e.div_(total.float()).mul_(-g)
        out["dlogits"] = p.scatter_add_(1, ids, g).to(s["logits"].dtype)
    return out


def _plain(s):
    return {"attn_fwd": _attend, "attn_bwd": _attend_grad, "distill": _plain_distill, "policy": _plain_policy}[s["case"]["op"]](s)


# ------------------------------------------------------- the library's own ----
def _library(s):
    import matrix_aware_optimizer_libmuon_amd as muon
    c = s["case"]
    op = c["op"]
    if op == "attn_fwd":
        o, lse = muon.attention(s["q"], s["k"], s["v"], starts=s["starts"], k_starts=s["k_starts"], causal=c["causal"])
        return dict(o=o, lse=lse)
    if op == "attn_bwd":
        views = {}
        if not c["ktokens"]:
            # the gradients side by side, as the projection's weight gradient takes them
            h, kv = c["heads"], c["kv"]
            dqkv = torch.empty(c["tokens"], h + 2 * kv, c["dim"], device=DEV, dtype=torch.bfloat16)
            views = dict(dq=dqkv[:, :h], dk=dqkv[:, h:h + kv], dv=dqkv[:, h + kv:])
        dq, dk, dv = muon.attention_grad(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], starts=s["starts"],
                                         k_starts=s["k_starts"], causal=c["causal"], **views)
        return dict(dq=dq, dk=dk, dv=dv)
    if op == "distill":
        loss, dlogits = muon.distill_loss(s["logits"], s["ids"], s["teacher"], temperature=s["tau"], weights=s["weights"],
                                          want_grad=c["grad"])
        return dict(loss=loss, dlogits=dlogits) if c["grad"] else dict(loss=loss)
    loss, logp, dlogits = muon.policy_loss(s["logits"], s["ids"], s["old"], s["adv"], ref_logp=s["ref"], clip=CLIP_LOW,
                                           clip_high=CLIP_HIGH, kl_coef=KL_COEF, weights=s["weights"], want_grad=c["grad"])
    out = dict(loss=loss, logp=logp)
    return dict(out, dlogits=dlogits) if c["grad"] else out


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ work ----
def work(case):
    if case["op"].startswith("attn"):
        d, pairs = case["dim"], _pairs(case)
        q, k = case["tokens"] * case["heads"], (case["ktokens"] or case["tokens"]) * case["kv"]
        if case["op"] == "attn_fwd":   # q, k, v -> o, lse: two products
            return dict(bytes=4 * d * q + 4 * d * k + 4 * q, flops=4 * pairs * case["heads"] * d)
        # do, q, o, k, v, lse -> dq, dk, dv: five products
        return dict(bytes=8 * d * q + 8 * d * k + 4 * q, flops=10 * pairs * case["heads"] * d)
    n, v = case["tokens"], case["vocab"]
    b = {"f32": 4, "bf16": 2}[case["dtype"]]
    i = {"i32": 4, "i64": 8}[case["ids"]]
    live = max(1, round(n * (1.0 - case["masked"])))   # the others' logits need not be read
    moved = live * v * b + (n * v * b if case["grad"] else 0) + 8 * n
    if case["op"] == "distill":
        return dict(bytes=moved + live * case["top"] * (4 + i), flops=6 * live * v)
    return dict(bytes=moved + live * (i + 8 + (4 if case["ref"] else 0)) + 4 * n, flops=6 * live * v)


# ------------------------------------------------------- in 64 bits, apart ----
def exact(case, seed):
    """The outputs of `run` in 64 bits: attention head by head, its gradients those of the exact probabilities; the
    losses row block by row block, with log_softmax."""
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attention(case, s)
    n, v = case["tokens"], case["vocab"]
    out = {"loss": torch.empty(n, dtype=torch.float64, device=DEV)}
    if case["op"] == "policy":
        out["logp"] = torch.empty_like(out["loss"])
    if case["grad"]:
        out["dlogits"] = torch.empty(n, v, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 28) // v)
    for at in range(0, n, step):
        rows = slice(at, min(n, at + step))
        tau = s.get("tau", 1.0)
        logq = torch.log_softmax(s["logits"][rows].double() / tau, dim=1)
        here = torch.arange(logq.shape[0], device=DEV)
        w, ids = s["weights"][rows].double(), s["ids"][rows].long()
        if case["op"] == "distill":
            target = torch.zeros_like(logq)
            logp = torch.log_softmax(s["teacher"][rows].double() / tau, dim=1)
            target[here[:, None], ids] = torch.exp(logp)
            kl = torch.linalg.vecdot(torch.exp(logp), logp - logq[here[:, None], ids])
            out["loss"][rows] = w * tau ** 2 * kl
            if case["grad"]:
                out["dlogits"][rows] = (torch.exp(logq) - target) * (w * tau)[:, None]
            continue
        logp = logq[here, ids]
        adv, up = s["adv"][rows].double(), logp - s["old"][rows].double()
        ratio = torch.exp(up)
        # the clip holds a ratio above the range where the advantage is positive, below it where it is negative
        held = ((adv > 0) & (ratio > 1 + CLIP_HIGH)) | ((adv < 0) & (ratio < 1 - CLIP_LOW))
        limit = torch.where(adv > 0, torch.full_like(adv, 1 + CLIP_HIGH), torch.full_like(adv, 1 - CLIP_LOW))
        loss = -adv * torch.where(held, limit, ratio)
        slope = torch.where(held, torch.zeros_like(adv), -adv * ratio)
        if s["ref"] is not None:
            gap = s["ref"][rows].double() - logp
            loss = loss + KL_COEF * (torch.exp(gap) - gap - 1)
            slope = slope + KL_COEF * (1 - torch.exp(gap))
        out["loss"][rows], out["logp"][rows] = w * loss, logp * (w != 0)
        if case["grad"]:
            grad = torch.exp(logq) * -(w * slope)[:, None]
            grad[here, ids] += w * slope
            out["dlogits"][rows] = grad
    return out


def _exact_attention(case, s):
    h, kv, d = case["heads"], case["kv"], case["dim"]
    back = case["op"] == "attn_bwd"
    names = {"dq": "q", "dk": "k", "dv": "v"} if back else {"o": "q"}
    out = {n: torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for n, x in names.items()}
    if not back:
        out["lse"] = torch.empty(h, case["tokens"], dtype=torch.float64, device=DEV)
    for q0, nq, k0, nk in _spans(case):
        a, b = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for head in range(h):
            shared = head // (h // kv)
            q, k, v = s["q"][a, head].double(), s["k"][b, shared].double(), s["v"][b, shared].double()
            x = q @ k.t() / math.sqrt(d)
            if case["causal"]:
                x = x + torch.full_like(x, -math.inf).triu(nk - nq + 1)
            p = torch.softmax(x, dim=1)
            if not back:
                out["o"][a, head] = p @ v
                out["lse"][head, a] = torch.logsumexp(x, dim=1)
                continue
            do = s["do"][a, head].double()
            dp = do @ v.t()
            dx = p * (dp - torch.linalg.vecdot(p, dp).unsqueeze(1)) / math.sqrt(d)
            out["dq"][a, head] = dx @ k
            out["dk"][b, shared] += dx.t() @ q
            out["dv"][b, shared] += p.t() @ do
    return out

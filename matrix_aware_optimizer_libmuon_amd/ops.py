"""Training operators beside the optimizer step: what makes the gradients that
``muon_step`` and ``adamw_step`` take, from activations kept in 8 bits
(include/muon.h, "Training operators").  Marshalling only: every computation
runs in libmuon.so, on the current stream of the tensors' device, or on
``stream``, to which the memory of the outputs then belongs.

    x8 = muon.act8_pack(x)                                # 8-bit copy for the backward pass
    h, y, n8, rstd = muon.rmsnorm_act8(x, gain, residual=r)
    a, gate8, up8 = muon.swiglu_act8(gate, up)
    dw = muon.act8_wgrad(dy, n8, col_gain=gain)           # the gradient of y W^T's W
    dx, dgain = muon.rmsnorm_act8_grad(dy, n8, rstd, gain, dres=dh)
    table_grad = muon.embed_grad(dx, ids, vocab)

Beside them attention with its backward pass and two losses that return the
gradient of the logits:

    o, lse = muon.attention(q, k, v, starts=starts)
    dq, dk, dv = muon.attention_grad(do, q, k, v, o, lse, starts=starts)
    loss, dlogits = muon.distill_loss(logits, ids, teacher, temperature=2.0)
    loss, logp, dlogits = muon.policy_loss(logits, actions, old_logp, advantages)

Matrices are 2-D with unit column stride, float32 or bfloat16; rows may be
strided (a column slice of a wider buffer is one).  The operators take no part in
autograd: what they return has no history, whether or not an argument requires a
gradient; the backward pass is called, as examples/train_act8.py does.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib, _marshaller


class Act8(NamedTuple):
    """A matrix in 8 bits: ``codes`` (float8_e4m3fn, rows x cols) and one
    ``scales`` byte (uint8, e + 127 for a scale of 2^e) per row and group of 32
    columns.  A value is its code times its group's scale."""
    codes: torch.Tensor
    scales: torch.Tensor


_bound = None


def _calls():
    """The marshalling module, bound to the library's entries."""
    global _bound
    if _bound is None:
        m, lib = _marshaller(), _lib.load()
        m.bind_ops({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                    for n in _lib.EXPORTED if n.startswith(("muon_act8", "muon_rmsnorm", "muon_swiglu", "muon_embed", "muon_attention",
                                      "muon_distill", "muon_policy"))})
        _bound = m
    return _bound


def _run(entry, first, stream, *args):
    """One call of the marshalling module; its outputs without the status."""
    call = getattr(_calls(), entry)
    if stream is None:
        status, *outs = call(*args)
    else:
        if stream.device != first.device:
            raise ValueError("stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            status, *outs = call(*args)
        # memory of other streams stays until this one has read it
        for t in args:
            for u in t if isinstance(t, tuple) else (t,):
                if isinstance(u, torch.Tensor):
                    u.record_stream(stream)
    if status:
        _lib.check(status, "muon_" + entry)
    return outs


def act8_pack(x, *, stream=None) -> Act8:
    """The 8-bit form of a matrix.  Each group of 32 columns takes the smallest
    power of two 2^e with max |v| <= 448 * 2^e (-117 <= e <= 119) as its scale;
    values round to nearest.  Infinities and NaN become NaN."""
    return Act8(*_run("act8_pack", x, stream, x))


def act8_unpack(x8: Act8, dtype=torch.bfloat16, *, stream=None):
    """The values an 8-bit matrix stands for (bfloat16 holds them exactly)."""
    return _run("act8_unpack", x8[0], stream, x8, dtype)[0]


def rmsnorm_act8(x, gain=None, residual=None, *, eps: float = 1e-6, save: bool = True, stream=None):
    """RMS norm of h = x + residual: n = h / sqrt(mean(h^2) + eps), y = n * gain.

    Returns (h, y, n8, rstd): h is x itself without a residual; n8 (Act8 of n,
    before the gain) and rstd (float32) are what the backward pass needs, and
    n8 with ``col_gain=gain`` what the weight gradients of layers fed by y need.
    ``save=False`` keeps neither and returns (h, y).  At most 16384 columns."""
    outs = _run("rmsnorm_act8", x, stream, x, gain, residual, float(eps), bool(save))
    if not save:
        return outs[0], outs[1]
    h, y, codes, scales, rstd = outs
    return h, y, Act8(codes, scales), rstd


def rmsnorm_act8_grad(dy, n8: Act8, rstd, gain=None, dres=None, *, want_dgain: bool = True, stream=None):
    """(dx, dgain) of rmsnorm_act8 for the gradient dy of y, with ``dres`` (the
    gradient that reaches h past the norm) added to dx; dx is the gradient of x
    and of the residual alike.  dgain is float32, None if not wanted."""
    return tuple(_run("rmsnorm_act8_grad", dy, stream, dy, n8, rstd, gain, dres, bool(want_dgain)))


def swiglu_act8(gate, up, *, save: bool = True, stream=None):
    """a = silu(gate) * up.  Returns (a, gate8, up8), the last two Act8 for the
    backward pass; ``save=False`` keeps neither and returns a."""
    outs = _run("swiglu_act8", gate, stream, gate, up, bool(save))
    if not save:
        return outs[0]
    a, gc, gs, uc, us = outs
    return a, Act8(gc, gs), Act8(uc, us)


def swiglu_act8_grad(da, gate8: Act8, up8: Act8, *, dgate=None, dup=None, want_a8: bool = True, stream=None):
    """(dgate, dup, a8) of swiglu_act8 for the gradient da of a; a8 is a again
    in 8 bits, for the next layer's weight gradient (None if not wanted).
    ``dgate`` and ``dup`` may be given, e.g. as the halves of one buffer."""
    outs = _run("swiglu_act8_grad", da, stream, da, gate8, up8, dgate, dup, bool(want_a8))
    return outs[0], outs[1], Act8(outs[2], outs[3]) if want_a8 else None


def act8_wgrad(dy, x8: Act8, *, col_gain=None, out=None, dtype=torch.float32, accumulate: bool = False, stream=None):
    """dw = dy^T x (n x k) from bfloat16 dy (tokens x n) and an 8-bit x (tokens
    x k), columns times ``col_gain``: the gradient of W in y = x W^T.  Written to
    ``out`` (float32 or bfloat16), or added to it with ``accumulate``; a new
    tensor of ``dtype`` otherwise."""
    return _run("act8_wgrad", dy, stream, dy, x8, col_gain, out, dtype, bool(accumulate))[0]


def embed(table, ids, *, scale: float = 1.0, out=None, dtype=torch.bfloat16, stream=None):
    """out[t] = scale * table[ids[t]].  ids: int32 or int64 vector; one outside
    the table (-1 for padding) gives a row of zeros and no gradient."""
    return _run("embed", table, stream, table, ids, float(scale), out, dtype)[0]


def embed_grad(dy, ids, vocab: int, *, scale: float = 1.0, out=None, dtype=torch.float32, accumulate: bool = False,
               stream=None):
    """The gradient of embed()'s table (vocab x cols): scale * the sum of the
    rows of dy with each id, in an order that depends on the ids alone.  Every
    row of the result is written; with ``accumulate`` the sums are added to
    ``out``, of which only the rows that have tokens are touched."""
    return _run("embed_grad", dy, stream, dy, ids, int(vocab), float(scale), out, dtype, bool(accumulate))[0]


def attention(q, k, v, *, starts=None, k_starts=None, causal: bool = True, scale: float | None = None, out=None, stream=None):
    """Softmax attention: (o, lse) of bfloat16 q (tokens, heads, dim) and k, v
    (k_tokens, kv_heads, dim); query head h reads key and value head
    h // (heads // kv_heads).  dim: a multiple of 8, at most 128.  The last axis has
    unit stride; tokens and heads may be strided (slices of a fused projection).

    ``starts`` (int32, on the GPU, from 0, not decreasing) holds the first token of
    each sequence and the end of the last; None is one sequence.  ``k_starts``: that
    of k and v, where it differs.  ``causal``: query i of nq sees keys j <= i + nk - nq.
    ``scale``: 1 / sqrt(dim) if None.  lse (float32, (heads, tokens)) is each row's log
    of the sum of exponentials, for the backward pass; a query that sees no key gets
    zeros and -infinity.  Tokens behind the last sequence: left as they are in
    ``out``, zeros in a new tensor; their lse is -infinity.  A value that is not finite
    may reach every row of its sequence and head, masked or not, but no other sequence."""
    return tuple(_run("attention", q, stream, q, k, v, starts, k_starts, bool(causal), None if scale is None else float(scale), out))


def attention_grad(do, q, k, v, o, lse, *, starts=None, k_starts=None, causal: bool = True, scale: float | None = None, dq=None,
                   dk=None, dv=None, stream=None):
    """(dq, dk, dv) of attention() for the gradient ``do`` of o, from what it took and
    returned; the probabilities are computed again.  ``dq``, ``dk`` and ``dv`` may be
    given, e.g. as slices of one buffer."""
    return tuple(_run("attention_grad", do, stream, do, q, k, v, o, lse, starts, k_starts, bool(causal),
                      None if scale is None else float(scale), dq, dk, dv))


def distill_loss(logits, ids, teacher, *, temperature: float = 1.0, weights=None, want_grad: bool = True, out=None, stream=None):
    """Distillation from a teacher's top logits: (loss, dlogits).  Row by row, with
    p the softmax of ``teacher`` / temperature (tokens, top) and q that of all
    ``logits`` / temperature (tokens, vocab):

        loss = weight * temperature^2 * sum_k p_k (log p_k - log q[ids_k])

    float32 per token, and ``dlogits`` the gradient of loss.sum(), in the logits'
    type (None if not wanted).  ``ids``: int32 or int64; an entry outside the
    vocabulary (-1) is not there; at most 1024 entries a token.  ``weights``: float32
    per token, e.g. a mask over the number of tokens; at 0 the logits are not read."""
    return tuple(_run("distill_loss", logits, stream, logits, ids, teacher, weights, out, float(temperature), bool(want_grad)))


def policy_loss(logits, actions, old_logp, advantages, *, ref_logp=None, clip: float = 0.2, clip_high: float | None = None,
                kl_coef: float = 0.0, temperature: float = 1.0, weights=None, want_grad: bool = True, out=None, stream=None):
    """Clipped policy loss with a KL term: (loss, logp, dlogits).  Token by token,
    with logp the action's log-probability under softmax(logits / temperature), r =
    exp(logp - old_logp) and d = ref_logp - logp:

        loss = weight * (-min(r A, clamp(r, 1 - clip, 1 + clip_high) A) + kl_coef (exp(d) - d - 1))

    float32 per token, and ``dlogits`` the gradient of loss.sum(), in the logits' type
    (None if not wanted).  No KL term without ``ref_logp`` or at a ``kl_coef`` of 0;
    ``clip``: 0 .. 1; ``clip_high``: clip if None.
    ``weights``: float32 per token; a token of weight 0, or whose action is outside
    the vocabulary, has loss and logp 0, and its logits are not read."""
    return tuple(_run("policy_loss", logits, stream, logits, actions, old_logp, advantages, ref_logp, weights, out, float(clip),
                      float(clip if clip_high is None else clip_high), float(kl_coef), float(temperature), bool(want_grad)))

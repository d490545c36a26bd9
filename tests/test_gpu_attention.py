"""Attention and its backward pass on the GPU against the 64-bit oracle.

Tolerances.  u = 2^-24 is the unit of fp32, b = 2^-8 the rounding to bf16.
A product of bf16 numbers is exact in fp32, so a sum of n of them, in any order, is
off by at most n u times the sum of their magnitudes; N = n + 16 also covers the few
roundings around it.  With A_ij = scale sum |q||k|, a score is off by
N A u, the exponent's argument by 4 u (A + |lse|) more, and the exponential by 2^-22:
  P is off by a factor of at most 1 + e,  e = (N + 4) A u + 4 u |lse| + 2^-21.
o sums P rounded to bf16 times v: |error| <= (b + 2 e + 2 n u) sum P|v| before its own
rounding; lse is off by at most e + n u.
In the backward pass dP - rowsum(do o) is off by D = N u (sum |do||v| + sum |do||o|), so
dS by (e + b)|dS| + P D (1 + b), and the sums over queries or keys as above."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from oracle import ops_oracle as O
from tests.gpu_helpers import DEV, say
from tests.test_gpu_ops import gen, near, np64

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16
LAYOUTS = ["plain", "fused", "heads_first", "interleaved", "odd"]


def tensors(seed, nq, nk, heads, kv, dim, layout="plain", sharp=1.0):
    """q, k, v on the GPU in a memory layout; everything around them is NaN."""
    g = gen(seed)
    q, k, v = (torch.randn(n, h, dim, generator=g) for n, h in ((nq, heads), (nk, kv), (nk, kv)))
    q = (q * sharp).to(BF)
    k, v = k.to(BF), v.to(BF)
    return [placed(t, layout, i) for i, t in enumerate((q, k, v))]


def placed(t, layout, which=0):
    n, h, d = t.shape
    nan = lambda *s: torch.full(s, float("nan"), device=DEV, dtype=BF)  # noqa: E731
    if layout == "plain":
        view = nan(n, h, d)
    elif layout == "fused":                                  # columns of a wider projection
        view = nan(n, h + 3, d)[:, 1:1 + h]
    elif layout == "heads_first":
        view = nan(h, n, d).transpose(0, 1)
    elif layout == "interleaved":                            # q, k, v of a head side by side
        view = nan(n, h, 3, d)[:, :, which]
    else:                                                    # 2-byte alignment, odd strides
        view = nan(n * h * (d + 3) + 1)[1:].view(n, h, d + 3)[:, :, 1:1 + d]
    view.copy_(t.to(DEV))
    return view


def starts_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32), device=DEV)


def pieces(nq_list, nk_list, heads, kv):
    q0 = k0 = 0
    for nq, nk in zip(nq_list, nk_list):
        for h in range(heads):
            yield slice(q0, q0 + nq), slice(k0, k0 + nk), h, h // (heads // kv)
        q0, k0 = q0 + nq, k0 + nk


def exp_error(q, k, lse, scale):
    a = scale * (np.abs(q) @ np.abs(k).T)
    return (q.shape[1] + 20) * U * a + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0))[:, None] + 2.0 ** -21


def check(q, k, v, nq_list, nk_list, causal, scale=None, seed=7, layout="plain", starts=True):
    dim = q.shape[2]
    c = float(np.float32(dim ** -0.5 if scale is None else scale))
    st = dict(starts=starts_of(nq_list) if starts else None,
              k_starts=starts_of(nk_list) if starts and nq_list is not nk_list else None, causal=causal, scale=scale)
    o, lse = muon.attention(q, k, v, **st)
    do = placed(torch.randn(q.shape, generator=gen(seed)).to(BF), layout)
    grads = muon.attention_grad(do, q, k, v, o, lse, **st)
    compare(q, k, v, do, o, lse, grads, nq_list, nk_list, causal, c)
    return (o, lse, *grads)


def compare(q, k, v, do, o, lse, grads, nq_list, nk_list, causal, c):
    """Outputs of both directions against the oracle; c: the scale."""
    heads, kv, dim = q.shape[1], k.shape[1], q.shape[2]
    want = [np.zeros(t.shape) for t in (q, q, k, v)]
    tol = [np.zeros(t.shape) for t in (q, q, k, v)]
    lse_want, lse_tol = np.zeros(lse.shape), np.zeros(lse.shape)
    q_, k_, v_, do_, o_, l_ = (np64(t) for t in (q, k, v, do, o, lse))
    for tq, tk, h, s in pieces(nq_list, nk_list, heads, kv):
        a, b, w, g = q_[tq, h], k_[tk, s], v_[tk, s], do_[tq, h]
        nq, nk = len(a), len(b)
        want[0][tq, h], lse_want[h, tq] = O.attention(a, b, w, c, causal)
        lw = lse_want[h, tq]
        e = exp_error(a, b, lw, c)
        see = O.visible(nq, nk, causal)
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(see, np.exp(c * (a @ b.T) - lw[:, None]), 0.0)
        row = (np.where(see, e, 0.0).max(1, initial=0.0))[:, None]
        tol[0][tq, h] = (B * (1 + B) + 2 * row + 2 * (nk + 16) * U) * (p @ np.abs(w))
        lse_tol[h, tq] = row[:, 0] + (nk + 64) * U
        # the backward pass on the o and lse that it was given
        oo, ll = o_[tq, h], l_[h, tq]
        dq, dk, dv = O.attention_grad(g, a, b, w, oo, ll, c, causal)
        want[1][tq, h] = dq
        want[2][tk, s] += dk
        want[3][tk, s] += dv
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(see, np.exp(c * (a @ b.T) - ll[:, None]), 0.0)
        ds = np.abs(p * (g @ w.T - (g * oo).sum(1, keepdims=True)))
        dd = (dim + 16) * U * (np.abs(g) @ np.abs(w).T + (np.abs(g) * np.abs(oo)).sum(1, keepdims=True))
        err = (B * (1 + B) + 2 * e) * ds + p * dd * (1 + 2 * B)
        n = heads // kv * nq
        tol[1][tq, h] = c * ((err + 2 * (nk + 16) * U * ds) @ np.abs(b))
        tol[2][tk, s] += c * ((err + 2 * (n + 16) * U * ds).T @ np.abs(a))
        tol[3][tk, s] += (((B * (1 + B) + 2 * e) + 2 * (n + 16) * U) * p).T @ np.abs(g)
    for name, got, ref, t in zip(("o", "dq", "dk", "dv"), (o, *grads), want, tol):
        try:
            near(got, ref, BF, 1.0, t)
        except AssertionError as err:
            raise AssertionError(f"{name}: {err}") from None
    same = l_ == lse_want                                    # -infinity among them
    off = np.abs(np.where(same, 0.0, l_) - np.where(same, 0.0, lse_want))
    assert (off <= lse_tol + 4 * U * np.abs(np.where(same, 0.0, lse_want))).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257, 400])
def test_lengths_of_one_sequence(n, causal):
    check(*tensors(n, n, n, 2, 2, 64), [n], [n], causal, starts=False)


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 56, 64, 72, 80, 96, 104, 120, 128])
def test_columns_of_a_head(dim):
    check(*tensors(dim, 150, 150, 2, 1, dim), [150], [150], True, starts=False)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dim", [40, 64, 80, 128])
def test_layouts_with_nothing_of_their_neighbours(layout, dim):
    """NaN lies between and around the rows, and behind the columns."""
    lengths = [70, 1, 0, 130]
    check(*tensors(3, 201, 201, 4, 2, dim, layout), lengths, lengths, True, layout=layout)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (6, 2), (5, 1), (8, 4)])
def test_shared_heads(heads, kv, causal):
    lengths = [100, 33, 129]
    check(*tensors(heads, 262, 262, heads, kv, 64), lengths, lengths, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [([5, 100], [90, 7]), ([1, 1, 1], [300, 1, 64]), ([130, 3], [0, 200]), ([0, 65], [70, 65]),
                                   ([200], [40]), ([40], [333]), ([64, 64], [64, 128])])
def test_queries_over_other_keys(nq, nk, causal):
    """Fewer keys than queries under a causal mask, and no keys at all: rows that see nothing."""
    out = check(*tensors(len(nq), sum(nq), sum(nk), 4, 2, 64), nq, nk, causal)
    q0 = 0
    for a, b in zip(nq, nk):
        blind = a if b == 0 else max(0, a - b) if causal else 0
        rows = slice(q0, q0 + blind)
        assert not out[0][rows].any() and not out[2][rows].any() and (out[1][:, rows] == -float("inf")).all()
        q0 += a


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("count", [62, 63, 64, 65, 127, 128, 700, 4097])
def test_many_sequences(count, causal):
    """Found by their work or by a search of one, two and three rounds; none of them long, a few long, many empty."""
    lengths = torch.randint(0, 9 if count < 1000 else 2, (count,), generator=gen(count)).tolist()
    lengths[count // 3] += 300
    lengths[-1] += 140
    n = sum(lengths)
    check(*tensors(count, n, n, 2, 1, 32), lengths, lengths, causal)
    keys = torch.randint(0, 4, (count,), generator=gen(count + 1)).tolist()
    check(*tensors(count, n, sum(keys), 2, 2, 32), lengths, keys, causal)


@pytest.mark.parametrize("sharp,scale", [(20.0, None), (1.0, 1e-3), (1.0, 3.0), (0.0, None)])
def test_sharp_and_flat_rows(sharp, scale):
    """Maxima that grow from tile to tile, single keys that take all, all keys alike."""
    q, k, v = tensors(5, 300, 300, 2, 2, 64, sharp=sharp)
    k *= torch.linspace(0.1, 2.0, 300, device=DEV)[:, None, None].to(BF)   # later keys larger
    check(q, k, v, [300], [300], False, scale=scale, starts=False)
    check(q, k.flip(0), v, [300], [300], True, scale=scale, starts=False)


def test_single_queries_over_long_keys():
    check(*tensors(8, 3, 3000, 4, 1, 128), [1, 2], [1000, 2000], True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,kv,dim", [(4, 1, 64), (6, 2, 80), (5, 1, 128), (32, 8, 40), (48, 1, 64), (200, 1, 24)])
@pytest.mark.parametrize("nq,nk", [([1], [1]), ([1, 1, 1], [70, 1, 300]), ([3, 0, 2], [64, 9, 700]), ([1, 150, 2, 0, 4], [200, 150, 1, 33, 3]),
                                   ([11], [2000]), ([1] * 70, [3] * 70), ([64], [64]), ([5, 2], [0, 1])])
def test_few_queries_of_heads_that_share_keys(nq, nk, heads, kv, dim, causal):
    """A block takes the queries of all heads of a key head, most of its rows empty."""
    out = check(*tensors(heads, sum(nq), sum(nk), heads, kv, dim), nq, nk, causal)
    q, k, v = tensors(heads, sum(nq) + 3, sum(nk) + 5, heads, kv, dim)
    st = dict(starts=starts_of(nq), k_starts=starts_of(nk), causal=causal)
    kept, (fresh, lse) = torch.full_like(q, 7.0), muon.attention(q, k, v, **st)
    muon.attention(q, k, v, out=kept, **st)
    n = sum(nq)
    assert (kept[n:] == 7).all() and not fresh[n:].any() and torch.equal(kept[:n], fresh[:n]) and (lse[:, n:] == -float("inf")).all()
    assert out[0].shape == (n, heads, dim)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_layouts_of_few_queries(layout, causal):
    check(*tensors(3, 12, 312, 4, 2, 72, layout), [7, 1, 0, 4], [7, 200, 5, 100], causal, layout=layout)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,heads,kv,dim", [([40], [4096], 4, 2, 64), ([1], [5000], 2, 1, 128), ([3, 0, 70], [3000, 9, 2500], 2, 2, 80),
                                                ([2500], [2500], 1, 1, 64), ([2100, 30], [2100, 30], 4, 1, 128), ([3000], [50], 2, 1, 40),
                                                ([1500], [1400], 3, 3, 96)])
def test_steps_cut_into_parts(nq, nk, heads, kv, dim, causal):
    """Few blocks of many steps (tests/test_ops_launches.py has the launches that these sizes make)."""
    check(*tensors(heads, sum(nq), sum(nk), heads, kv, dim), nq, nk, causal)
    kept = torch.full((sum(nq) + 9, heads, dim), 7.0, dtype=BF, device=DEV)
    q, k, v = tensors(heads, sum(nq) + 9, sum(nk) + 5, heads, kv, dim)
    st = dict(starts=starts_of(nq), k_starts=starts_of(nk), causal=causal)
    o, lse = muon.attention(q, k, v, out=kept, **st)
    fresh, _ = muon.attention(q, k, v, **st)
    assert (o[-9:] == 7).all() and not fresh[-9:].any() and torch.equal(o[:-9], fresh[:-9]) and (lse[:, -9:] == -float("inf")).all()
    mine = [torch.full_like(t, 7.0) for t in (q, k, v)]
    grads = muon.attention_grad(o, q, k, v, o, lse, dq=mine[0], dk=mine[1], dv=mine[2], **st)
    news = muon.attention_grad(o, q, k, v, o, lse, **st)
    for a, b, n in zip(grads, news, (9, 5, 5)):
        assert (a[-n:] == 7).all() and not b[-n:].any() and torch.equal(a[:-n], b[:-n])


def test_gradients_by_differences():
    """The inner product of do with the change of o (in 64 bits) along random directions."""
    q, k, v = tensors(9, 60, 60, 2, 1, 64)
    o, lse = muon.attention(q, k, v)
    do = torch.randn(q.shape, generator=gen(1)).to(BF).to(DEV)
    grads = muon.attention_grad(do, q, k, v, o, lse)

    def value(q_, k_, v_):
        return sum((np64(do)[:, h] * O.attention(q_[:, h], k_[:, 0], v_[:, 0], 0.125, True)[0]).sum() for h in range(2))
    base = [np64(t) for t in (q, k, v)]
    rng = np.random.default_rng(0)
    for i, g in enumerate(grads):
        way = rng.normal(size=base[i].shape)
        moved = [[x + (s * 1e-4 * way if i == j else 0.0) for j, x in enumerate(base)] for s in (1, -1)]
        slope = (value(*moved[0]) - value(*moved[1])) / 2e-4
        # each entry is off by about 3 b of its size (o, P and dS rounded to bf16, itself too), the signs of way apart
        assert abs(slope - (np64(g) * way).sum()) <= 4 * 4 * B * np.linalg.norm(np64(g))


def test_rows_behind_the_last_sequence():
    lengths = [40, 90]
    q, k, v = tensors(11, 150, 150, 2, 1, 64)
    st = starts_of(lengths)
    o, lse = muon.attention(q, k, v, starts=st)
    assert not o[130:].any() and (lse[:, 130:] == -float("inf")).all()
    do = torch.randn(q.shape, generator=gen(1)).to(BF).to(DEV)
    grads = muon.attention_grad(do, q, k, v, o, lse, starts=st)
    assert not any(g[130:].any() for g in grads)
    kept = torch.full_like(q, 7.0)
    o2, lse2 = muon.attention(q, k, v, starts=st, out=kept)
    assert o2 is kept and torch.equal(o2[:130], o[:130]) and (o2[130:] == 7).all() and torch.equal(lse2, lse)
    mine = [torch.full_like(t, 7.0) for t in (q, k, v)]
    for some in ([0, 1, 2], [0], [1], [2]):
        for m in mine:
            m.fill_(7.0)
        out = muon.attention_grad(do, q, k, v, o, lse, starts=st, **{("dq", "dk", "dv")[i]: mine[i] for i in some})
        for i in range(3):
            assert torch.equal(out[i][:130], grads[i][:130])
            assert (out[i][130:] == 7).all() if i in some else not out[i][130:].any()


def test_no_tokens():
    q, k, v = tensors(1, 0, 0, 2, 1, 64)
    o, lse = muon.attention(q, k, v)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert [tuple(g.shape) for g in muon.attention_grad(q, q, k, v, o, lse)] == [(0, 2, 64), (0, 1, 64), (0, 1, 64)]
    q, k, v = tensors(1, 0, 30, 2, 1, 64)
    o, lse = muon.attention(q, k, v)
    dq, dk, dv = muon.attention_grad(q, q, k, v, o, lse)
    assert not dk.any() and not dv.any()
    q, k, v = tensors(1, 30, 0, 2, 1, 64)
    o, lse = muon.attention(q, k, v, causal=False)
    assert not o.any() and (lse == -float("inf")).all() and not muon.attention_grad(q, q, k, v, o, lse)[0].any()


def test_not_finite_values_stay_in_their_sequence_and_head():
    lengths = [70, 64, 66]
    q, k, v = tensors(12, 200, 200, 4, 2, 64)
    st = starts_of(lengths)
    clean = muon.attention(q, k, v, starts=st)
    do = torch.randn(q.shape, generator=gen(1)).to(BF).to(DEV)
    clean = (*clean, *muon.attention_grad(do, q, k, v, *clean, starts=st))
    for t in (q, k, v):
        t[100, 0, 3] = float("nan")
        t[90, 0, 5] = float("inf")
    dirty = muon.attention(q, k, v, starts=st)
    dirty = (*dirty, *muon.attention_grad(do, q, k, v, *dirty, starts=st))
    for a, b in zip(clean, dirty):
        if a.dim() == 2:
            a, b = a.t().unsqueeze(2), b.t().unsqueeze(2)
        others = torch.ones(a.shape[:2], dtype=torch.bool, device=DEV)
        others[70:134, :2 if a.shape[1] == 4 else 1] = False          # the heads that share key head 0
        assert torch.equal(a[others], b[others]) and not torch.isfinite(b[~others]).all()


def test_starts_out_of_order_or_range_stay_inside():
    """Undefined values, but nothing outside the outputs is written."""
    q, k, v = tensors(13, 100, 100, 2, 1, 64)
    do = torch.randn(q.shape, generator=gen(1)).to(BF).to(DEV)
    noise = torch.randint(-150, 250, (500,), generator=gen(2)).tolist()
    for bad, causal in [(b, c) for c in (True, False) for b in (
            [0, 500, 100], [-9, 60, 40, 100], [90, 10, 1 << 30], [0, -5, -7], [-(1 << 31), (1 << 31) - 1], noise[:30], noise, noise[::-1])]:
        st = torch.tensor(bad, dtype=torch.int32, device=DEV)
        bufs = [torch.full((t.shape[0] + 200, *t.shape[1:]), 3.0, dtype=BF, device=DEV) for t in (q, q, k, v)]
        outs = [b[100:200] for b in bufs]
        _, lse = muon.attention(q, k, v, starts=st, causal=causal, out=outs[0])
        muon.attention_grad(do, q, k, v, outs[0], lse, starts=st, causal=causal, dq=outs[1], dk=outs[2], dv=outs[3])
        torch.cuda.synchronize()
        assert all((b[:100] == 3).all() and (b[200:] == 3).all() for b in bufs)


def test_the_same_bits_every_time():
    q, k, v = tensors(14, 700, 700, 8, 2, 128)
    st = starts_of([300, 400])
    do = torch.randn(q.shape, generator=gen(1)).to(BF).to(DEV)

    def once():
        o, lse = muon.attention(q, k, v, starts=st)
        return (o, lse, *muon.attention_grad(do, q, k, v, o, lse, starts=st))
    first = once()
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_offsets_past_32_bits():
    """q, k, v of more than 2^32 bytes: the first and the last sequence."""
    n, dim, tail = 1 << 20, 128, 300
    big = torch.zeros(n, 18, dim, dtype=BF, device=DEV)
    st = torch.tensor([0, 64, n - tail, n], dtype=torch.int32, device=DEV)
    # the long middle has no keys: two sets of starts
    ks = torch.tensor([0, 64, 64, 64 + tail], dtype=torch.int32, device=DEV)
    ends = torch.cat([torch.arange(64), torch.arange(n - tail, n)]).to(DEV)
    g = gen(2)
    q, k, v = big[:, :16], big[n - 64 - tail:, 16:17], big[n - 64 - tail:, 17:]
    q[ends] = torch.randn(64 + tail, 16, dim, generator=g).to(BF).to(DEV)
    k.copy_(torch.randn(64 + tail, 1, dim, generator=g).to(BF))
    v.copy_(torch.randn(64 + tail, 1, dim, generator=g).to(BF))
    do = torch.zeros(n, 16, dim, dtype=BF, device=DEV)
    do[ends] = torch.randn(64 + tail, 16, dim, generator=g).to(BF).to(DEV)
    o, lse = muon.attention(q, k, v, starts=st, k_starts=ks)
    say("attended")
    dq, dk, dv = muon.attention_grad(do, q, k, v, o, lse, starts=st, k_starts=ks)
    assert not o[64:n - tail].any() and not dq[64:n - tail].any()
    compare(q[ends], k, v, do[ends], o[ends], lse[:, ends], (dq[ends], dk, dv), [64, tail], [64, tail], True,
            float(np.float32(dim ** -0.5)))


def test_refusals_name_the_argument():
    q, k, v = tensors(1, 10, 10, 4, 2, 64)
    o, lse = muon.attention(q, k, v)
    st = starts_of([10])
    att = muon.attention
    grad = lambda **kw: muon.attention_grad(q, q, k, v, o, kw.pop("lse", lse), **kw)  # noqa: E731
    for err, match, call in (
            (TypeError, "q must be bfloat16", lambda: att(q.float(), k, v)),
            (TypeError, "k must be bfloat16", lambda: att(q, k.half(), v)),
            (ValueError, "q must be 3-D", lambda: att(q[0], k, v)),
            (ValueError, "k must have shape", lambda: att(q, k[:, :, :56], v)),
            (ValueError, "v must have shape", lambda: att(q, k, v[:9])),
            (ValueError, "divides", lambda: att(q[:, :3], k, v)),
            (ValueError, "multiple of 8", lambda: att(q[:, :, :60], k[:, :, :60], v[:, :, :60])),
            (ValueError, "unit stride along its last axis", lambda: att(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)),
            (ValueError, "must be a GPU tensor", lambda: att(q, k.cpu(), v)),
            (TypeError, "starts must be int32", lambda: att(q, k, v, starts=st.long())),
            (ValueError, "starts must be a contiguous vector", lambda: att(q, k, v, starts=st[None])),
            (ValueError, "k_starts must come with starts", lambda: att(q, k, v, k_starts=st)),
            (ValueError, "k_starts must be as long", lambda: att(q, k, v, starts=st, k_starts=starts_of([5, 5]))),
            (ValueError, "k_starts must be given", lambda: att(q, k[:9], v[:9], starts=st)),
            (ValueError, "out must have shape", lambda: att(q, k, v, out=q[:9].clone())),
            (TypeError, "lse must be float32", lambda: grad(lse=lse.double())),
            (ValueError, "lse must have shape", lambda: grad(lse=lse[:, :9])),
            (ValueError, "dk must have shape", lambda: grad(dk=torch.empty_like(q)))):
        with pytest.raises(err, match=match):
            call()
    for status, call in ((muon.MUON_EINVAL, lambda: att(q, k, v, scale=-1.0)), (muon.MUON_EINVAL, lambda: att(q, k, v, scale=float("nan"))),
                         (muon.MUON_EINVAL, lambda: att(q, k[:, :1].expand(10, 2, 64), v)),
                         (muon.MUON_EALIAS, lambda: att(q, k, v, out=q)), (muon.MUON_EALIAS, lambda: grad(dk=k)),
                         (muon.MUON_EALIAS, lambda: grad(dk=(s := torch.empty_like(k)), dv=s))):
        with pytest.raises(muon.LibMuonError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("pad", [8, 5])
@pytest.mark.parametrize("form", ["heads of a kind apart", "heads side by side", "padded columns"])
def test_slices_of_a_padded_buffer(form, pad):
    """q, k, v in one buffer, dq, dk, dv in one, q and o in one: the same bits as in tensors of their own."""
    lengths, h, d = [70, 1, 130], 4, 64
    n = sum(lengths)

    def three():
        if form == "padded columns":
            x = torch.full((n, 3 * h, d + pad), 7.0, device=DEV, dtype=BF)
            return x, [x[:, i * h:(i + 1) * h, :d] for i in range(3)]
        x = torch.full((n, 3 * h * d + pad), 7.0, device=DEV, dtype=BF)
        parts = x[:, :3 * h * d].unflatten(1, (3, h, d) if form == "heads of a kind apart" else (h, 3, d))
        return x, [parts[:, i] if form == "heads of a kind apart" else parts[:, :, i] for i in range(3)]
    plain = tensors(21, n, n, h, h, d)
    _, qkv = three()
    for a, b in zip(qkv, plain):
        a.copy_(b)
    st = dict(starts=starts_of(lengths))
    o, lse = muon.attention(*plain, **st)
    do = torch.randn(o.shape, generator=gen(1)).to(BF).to(DEV)
    want = muon.attention_grad(do, *plain, o, lse, **st)
    whole, grads = three()
    muon.attention_grad(do, *qkv, o, lse, dq=grads[0], dk=grads[1], dv=grads[2], **st)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert int((whole == 7).sum()) == whole.numel() - sum(int((g != 7).sum()) for g in grads)
    _, (q, out, _) = three()
    q.copy_(plain[0])
    assert torch.equal(muon.attention(q, plain[1], plain[2], out=out, **st)[0], o)

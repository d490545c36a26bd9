"""Distillation and policy losses on the GPU against the 64-bit oracle.

Tolerances.  u = 2^-24.  With k = log2(e) / temperature and X the largest |x - max| of
a row, in units of the temperature: an exponential's argument is off by at most 4 u X
log2(e) (the difference, k, the product), its value by e = 6 u X + 2^-22 relative; a sum
of positive terms goes through at most 130 in a thread, 6 steps in a wave and 17 over the
waves and passes: S = 160 u + e relative.  A log-probability (x - max) k - log2(sum) is off by
L = S + 4 u (X + log of the sum), absolutely.
Distillation: p is off by e' + S' relative in the same way (X' over the teacher's entries), a
term p (log p - log q) by p (L + L') + |term| (e' + S'), sums of them by top u more.  The
gradient softmax - sum of p is off by softmax (e + S) + p (e' + S' + top u) before its rounding.
Policy: the ratio is off by R = L + 4 u |log ratio| + 2^-21 relative, exp(d) - 1 - d by
(L + 2 u |ref|) |exp(d) - 1| + 2^-20 of itself + the square of L."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from oracle import ops_oracle as O
from tests.gpu_helpers import DEV, say
from tests.test_gpu_ops import TYPES, U, gen, ids_of, near, np64, on_gpu

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
# a width of every layout: one wave, 256, 512 and 1024 threads with 1 to 16 vectors each, rows read twice
COLS = [1, 7, 8, 9, 100, 511, 512, 513, 1000, 2048, 2049, 5000, 8193, 16384, 16385, 32000, 32768, 32769, 50001, 65537, 70001, 131072,
        131073, 200003]


def spread(x):
    """(X, log of the sum) of rows already divided by the temperature."""
    top = x.max(1, keepdims=True)
    gap = np.where(np.isfinite(x), top - x, 0.0)
    return np.minimum(gap, 200.0).max(1), np.log(np.exp(np.maximum(x - top, -700)).sum(1))


def soft_errors(x):
    """e, S, L of the rows."""
    wide, total = spread(x)
    e = 6 * U * wide + 2.0 ** -22
    s = 160 * U + e
    return e, s, s + 4 * U * (wide + total)


def entries(seed, rows, vocab, top, id_type):
    g = gen(seed)
    ids = torch.randint(0, vocab, (rows, top), generator=g)
    ids[torch.rand(rows, top, generator=g) < 0.1] = -1
    ids[torch.rand(rows, top, generator=g) < 0.05] = vocab           # just outside
    if rows > 1:
        ids[1] = ids[1, 0]                                           # one id, over and over
    ids[0, 0] = vocab - 1
    return ids.to(id_type)


def check_distill(logits, ids, teacher, temperature=1.0, weights=None, layout="plain"):
    rows, vocab = logits.shape
    w = np.ones(rows) if weights is None else np64(weights)
    tau = float(np.float32(temperature))
    put = lambda t: on_gpu(t, layout)  # noqa: E731
    wg = None if weights is None else weights.to(DEV)
    got = muon.distill_loss(put(logits), put(ids), put(teacher), temperature=temperature, weights=wg)
    alone, none = muon.distill_loss(put(logits), put(ids), put(teacher), temperature=temperature, weights=wg, want_grad=False)
    assert none is None and torch.equal(alone, got[0])
    z, t, i = np64(logits), np64(teacher), ids.numpy().astype(np.int64)
    loss, grad = O.distill(z, i, t, tau, w)
    e, s, lim = soft_errors(z / tau)
    near_rows = []
    for r in range(rows):
        live = (i[r] >= 0) & (i[r] < vocab) & (t[r] != -np.inf)
        if w[r] == 0 or not live.any():
            near_rows.append((0.0, np.zeros(vocab)))
            continue
        te, ts, tl = (float(v[0]) for v in soft_errors(t[r:r + 1, live] / tau))
        lp = O.log_softmax(t[r:r + 1, live] / tau)[0]
        lq = O.log_softmax(z[r:r + 1] / tau)[0]
        p = np.exp(lp)
        terms = np.abs(p * (lp - lq[i[r][live]]))
        tol = (p * (lim[r] + tl)).sum() + (te + ts + 2 * (len(p) + 24) * U) * terms.sum()
        at = np.exp(lq) * (e[r] + s[r] + 8 * U)
        np.add.at(at, i[r][live], p * (te + ts + (len(p) + 8) * U))
        near_rows.append((abs(w[r]) * tau ** 2 * tol, abs(w[r]) * tau * at))
    near(got[0], loss, F32, 1.0, np.array([a for a, _ in near_rows]) * (1 + 1e-6) + 8 * U * np.abs(loss))
    near(got[1], grad, logits.dtype, 1.0, np.stack([b for _, b in near_rows]) + 8 * U * np.abs(grad))
    return got


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("cols", COLS)
def test_distillation_of_every_width(cols, dtype):
    logits = (3 * torch.randn(3, cols, generator=gen(cols))).to(dtype)
    ids = entries(cols, 3, cols, 20, torch.int64)
    teacher = 2 * torch.randn(3, 20, generator=gen(cols + 1))
    check_distill(logits, ids, teacher, 1.5)


@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64], ids=ids_of)
@pytest.mark.parametrize("top", [1, 2, 3, 4, 5, 63, 65, 257, 1000, 1024])
def test_entries_of_the_teacher(top, id_type, layout):
    for cols, dtype in ((300, BF), (3001, F32)):
        logits = (2 * torch.randn(5, cols, generator=gen(top))).to(dtype)
        check_distill(logits, entries(top, 5, cols, top, id_type), torch.randn(5, top, generator=gen(3)).to(dtype), 2.0,
                      torch.tensor([1.0, 0.25, 0.0, -2.0, 1e-4]), layout)


def test_distillation_of_rows_without_entries_and_of_weight_zero():
    nan = float("nan")
    logits = torch.full((4, 600), nan)
    logits[3] = torch.randn(600, generator=gen(1))
    ids = torch.full((4, 3), -1)
    ids[0], ids[3] = 5, torch.tensor([1, 2, 1])
    teacher = torch.zeros(4, 3)
    ids[2], teacher[2] = 7, -float("inf")                            # entries that are not there
    for dtype in TYPES:
        loss, grad = check_distill(logits.to(dtype), ids, teacher, 1.0, torch.tensor([0.0, 1.0, 1.0, 1.0]))
        assert not loss[:3].any() and not grad[:3].any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
def test_distillation_over_masked_columns(dtype):
    """-infinity and the type's lowest value among the logits; a whole row of the lowest."""
    low = torch.finfo(dtype).min
    logits = torch.randn(4, 4000, generator=gen(2)).to(dtype)
    logits[0, ::2], logits[1, 1::2], logits[2] = -float("inf"), low, low
    logits[3, 64:] = -float("inf")
    ids = torch.tensor([[1, 3], [0, 2], [0, 3999], [5, 63]])
    check_distill(logits, ids, torch.randn(4, 2, generator=gen(3)), 0.7)
    # a teacher's entry on a column that cannot be: an infinite loss, a finite gradient
    loss, grad = muon.distill_loss(logits.to(DEV), torch.tensor([[0], [1], [1], [100]], device=DEV), torch.zeros(4, 1, device=DEV))
    assert loss[0] == float("inf") and loss[3] == float("inf") and torch.isfinite(grad).all() and grad[3, 100] == -1
    bad = logits.clone()
    bad[0, 1], bad[1, 0] = float("nan"), float("inf")
    loss, grad = muon.distill_loss(bad.to(DEV), ids.to(DEV), torch.zeros(4, 2, device=DEV))
    assert torch.isnan(loss[:2]).all() and torch.isnan(grad[:2]).any(1).all() and torch.isfinite(grad[2:]).all()


def check_policy(logits, actions, old, adv, ref=None, clip=0.2, clip_high=None, kl=0.0, temperature=1.0, weights=None, layout="plain"):
    rows = len(logits)
    w = np.ones(rows) if weights is None else np64(weights)
    high = clip if clip_high is None else clip_high
    f = lambda v: float(np.float32(v))  # noqa: E731
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    args = (on_gpu(logits, layout), dev(actions), dev(old), dev(adv))
    kw = dict(ref_logp=dev(ref), clip=clip, clip_high=clip_high, kl_coef=kl, temperature=temperature, weights=dev(weights))
    got = muon.policy_loss(*args, **kw)
    alone = muon.policy_loss(*args, **kw, want_grad=False)
    assert alone[2] is None and torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])
    tau = f(temperature)
    z, a = np64(logits), actions.numpy().astype(np.int64)
    o, ad, rf = np64(old), np64(adv), None if ref is None else np64(ref)
    loss, logp, grad = O.policy(z, a, o, ad, rf, f(clip), f(high), f(kl), tau, w)
    e, s, lim = soft_errors(z / tau)
    ltol, ptol, gtol = np.zeros(rows), np.zeros(rows), np.zeros(z.shape)
    for r in range(rows):
        if w[r] == 0 or not 0 <= a[r] < z.shape[1]:
            continue
        up = logp[r] - o[r]
        ratio, part = np.exp(up), lim[r] + 4 * U * (abs(up) + abs(o[r]) + abs(logp[r])) + 2.0 ** -21
        hold = np.clip(ratio, 1 - f(clip), 1 + f(high))
        ltol[r] = part * abs(ratio * ad[r]) + 4 * U * abs(hold * ad[r])
        gt = part * abs(ratio * ad[r])
        if rf is not None:
            d = rf[r] - logp[r]
            off = lim[r] + 4 * U * (abs(rf[r]) + abs(logp[r]))
            ltol[r] += abs(f(kl)) * (off * abs(np.expm1(d)) + off ** 2 + 2.0 ** -20 * (np.exp(d) - 1 - d) + 4 * U * (abs(d) > .25) * (1 + abs(d)))
            gt += abs(f(kl)) * (2 * off * np.exp(d) + 8 * U * abs(np.expm1(d)))
        ltol[r] *= abs(w[r])
        ptol[r] = lim[r] + 4 * U * abs(logp[r])
        q = np.exp(O.log_softmax(z[r:r + 1] / tau)[0])
        one = np.zeros(len(q))
        one[a[r]] = 1
        slope = np.abs(grad[r]).max() if len(q) == 1 else None
        g = abs(w[r]) / tau * gt
        size = np.abs(grad[r])
        # g (1 - q): both terms' errors, the difference's own rounding
        full = abs(grad[r, a[r]]) / max(1 - q[a[r]], 1e-300) if slope is None and q[a[r]] < 1 else 0.0
        gtol[r] = g * (q + one) + full * q * (e[r] + s[r] + 8 * U) + 8 * U * (size + full * one)
    near(got[1], logp, F32, 1.0, ptol)
    near(got[0], loss, F32, 1.0, ltol + 8 * U * np.abs(loss))
    near(got[2], grad, logits.dtype, 1.0, gtol)
    return got


def policy_inputs(seed, rows, cols, dtype, id_type=torch.int64):
    """Ratios from half to twice, at a distance from the borders 0.8 and 1.2 of the clip."""
    g = gen(seed)
    logits = (2 * torch.randn(rows, cols, generator=g)).to(dtype)
    actions = torch.randint(0, cols, (rows,), generator=g)
    if rows > 1:
        actions[1] = cols - 1
    logp = torch.from_numpy(O.log_softmax(np64(logits)))[torch.arange(rows), actions]
    old = (logp - torch.round(0.4 * 64 * torch.randn(rows, generator=g)) / 64).float()
    return logits, actions.to(id_type), old, torch.randn(rows, generator=g), (logp + 0.5 * torch.randn(rows, generator=g)).float()


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("cols", COLS)
def test_policy_of_every_width(cols, dtype):
    logits, actions, old, adv, ref = policy_inputs(cols, 4, cols, dtype)
    check_policy(logits, actions, old, adv, ref, kl=0.1)


@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64], ids=ids_of)
def test_policy_options(id_type, layout):
    logits, actions, old, adv, ref = policy_inputs(3, 200, 1003, BF, id_type)
    weights = torch.rand(200, generator=gen(4))
    weights[::7] = 0
    adv[5] = 0
    actions[3], actions[4] = -1, 1003                                # outside: no part
    for kw in (dict(), dict(ref=ref, kl=0.05), dict(ref=ref), dict(weights=weights, clip=0.1, clip_high=0.3), dict(clip=0.0),
               dict(clip=1.0, clip_high=50.0), dict(ref=ref, kl=-0.5, weights=weights), dict(temperature=0.5), dict(temperature=3.0)):
        loss, logp, grad = check_policy(logits, actions, old, adv, layout=layout, **kw)
        assert not loss[3:5].any() and not logp[3:5].any() and not grad[3:5].any()
        if "weights" in kw:
            assert not loss[::7].any() and not grad[::7].any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
def test_policy_over_masked_columns_and_skipped_rows(dtype):
    logits, actions, old, adv, ref = policy_inputs(6, 4, 3000, dtype)
    actions[:] = torch.tensor([1, 2, 2999, 7])
    logits[0, ::2], logits[1, 1::2], logits[2] = -float("inf"), torch.finfo(dtype).min, torch.finfo(dtype).min
    old = torch.from_numpy(O.log_softmax(np64(logits)))[torch.arange(4), actions].float()
    check_policy(logits, actions, old, adv, ref, kl=0.1)
    logits[3] = float("nan")
    weights = torch.tensor([1.0, 1.0, 1.0, 0.0])
    loss, logp, grad = muon.policy_loss(logits.to(DEV), actions.to(DEV), old.to(DEV), adv.to(DEV), weights=weights.to(DEV))
    assert loss[3] == 0 and logp[3] == 0 and not grad[3].any()
    loss, logp, grad = muon.policy_loss(logits.to(DEV), actions.to(DEV), old.to(DEV), adv.to(DEV))
    assert torch.isnan(loss[3]) and torch.isnan(logp[3]) and torch.isnan(grad[3]).all() and torch.isfinite(grad[:3]).all()
    # an action that cannot be, and a ratio past the largest number
    z, one = torch.zeros(3, 64), torch.ones(3)
    z[:, 1] = -float("inf")
    old = torch.tensor([-1.0, -200.0, -200.0])
    loss, logp, grad = muon.policy_loss(z.to(DEV), torch.tensor([1, 0, 0], device=DEV), old.to(DEV), torch.tensor([1.0, 1.0, 0.0]).to(DEV))
    assert logp[0] == -float("inf") and loss.tolist()[0] == 0 and loss[1] == -np.float32(1.2) and loss[2] == 0
    assert not grad[1:].any()


def test_gradients_by_differences():
    """Of the 64-bit losses, at the operators' own gradients."""
    z = torch.randn(3, 40, generator=gen(8))
    ids, teacher = torch.tensor([[1, 5, 5], [0, 39, 2], [7, -1, 8]]), torch.randn(3, 3, generator=gen(9))
    w = torch.tensor([1.0, 0.5, 2.0])
    _, got = muon.distill_loss(z.to(DEV), ids.to(DEV), teacher.to(DEV), temperature=1.7, weights=w.to(DEV))
    args = (torch.tensor([3, 39, 0]), torch.tensor([-3.0, -4.0, -2.5]), torch.tensor([1.0, -0.7, 0.4]))
    ref = torch.tensor([-4.0, -3.0, -3.5])
    _, _, got_p = muon.policy_loss(z.to(DEV), *(a.to(DEV) for a in args), ref_logp=ref.to(DEV), kl_coef=0.3, clip=0.9, clip_high=9.0,
                                   weights=w.to(DEV), temperature=1.7)
    tau = float(np.float32(1.7))
    one = lambda x: O.distill(x, ids.numpy(), np64(teacher), tau, np64(w))[0].sum()  # noqa: E731
    two = lambda x: O.policy(x, args[0].numpy(), np64(args[1]), np64(args[2]), np64(ref), 0.9, 9.0, float(np.float32(0.3)), tau,  # noqa: E731
                             np64(w))[0].sum()
    for f, g in ((one, np64(got)), (two, np64(got_p))):
        for i in range(z.numel()):
            up, down = np64(z), np64(z)
            up.flat[i] += 1e-5
            down.flat[i] -= 1e-5
            # the difference's own error, 1e-10 / 6 of a third derivative, and 64 u of numbers around one
            assert abs((f(up) - f(down)) / 2e-5 - g.flat[i]) < 64 * U


def test_no_rows_and_given_outputs():
    e = torch.empty(0, 50, device=DEV)
    i = torch.empty(0, dtype=torch.int64, device=DEV)
    f = torch.empty(0, device=DEV)
    loss, grad = muon.distill_loss(e, i.view(0, 1), f.view(0, 1))
    assert loss.shape == (0,) and grad.shape == (0, 50)
    assert [tuple(t.shape) for t in muon.policy_loss(e, i, f, f)] == [(0,), (0,), (0, 50)]
    logits, actions, old, adv, ref = (t.to(DEV) for t in policy_inputs(3, 5, 777, BF))
    out = on_gpu(torch.zeros(5, 777).to(BF), "odd")
    around = out.as_strided((5, 782), out.stride(), out.storage_offset() - 1)
    got = muon.policy_loss(logits, actions, old, adv, out=out)
    assert got[2] is out and torch.equal(out, muon.policy_loss(logits, actions, old, adv)[2])
    assert torch.isnan(around[:, 0]).all() and torch.isnan(around[:4, 778:]).all()


def test_more_rows_than_blocks_and_past_32_bits():
    rows = (1 << 21) + 5
    logits = torch.zeros(rows, 16, device=DEV)
    logits[-3:] = torch.randn(3, 16, generator=gen(1)).to(DEV)
    ids = torch.ones(rows, 1, dtype=torch.int32, device=DEV)
    loss, grad = muon.distill_loss(logits, ids, torch.zeros(rows, 1, device=DEV))
    tail = muon.distill_loss(logits[-3:], ids[-3:], torch.zeros(3, 1, device=DEV))
    assert torch.equal(loss[-3:], tail[0]) and torch.equal(grad[-3:], tail[1]) and torch.equal(grad[0], grad[rows - 4])
    say("many rows")
    rows, cols = 34_000, 131_072                                     # 2^32 elements and more
    logits = torch.zeros(rows, cols, dtype=BF, device=DEV)
    logits[-2:] = torch.randn(2, cols, generator=gen(2)).to(BF).to(DEV)
    act = torch.full((rows,), cols - 1, device=DEV)
    zero, weights = torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)
    weights[-2:] = 1
    loss, logp, grad = muon.policy_loss(logits, act, zero - 11.0, zero + 1, weights=weights)
    want = muon.policy_loss(logits[-2:].clone(), act[-2:], zero[-2:] - 11.0, zero[-2:] + 1)
    assert all(torch.equal(a[-2:], b) for a, b in zip((loss, logp, grad), want)) and not grad[:100].any()


def test_refusals_name_the_argument():
    z, i, f = torch.zeros(4, 50, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV)
    ii, t = i[:, None].expand(4, 1).contiguous(), torch.zeros(4, 1, device=DEV)
    dis, pol = muon.distill_loss, muon.policy_loss
    for err, match, call in (
            (TypeError, "logits must be float32 or bfloat16", lambda: dis(z.half(), ii, t)),
            (ValueError, "logits must be 2-D", lambda: dis(z[0], ii, t)),
            (ValueError, "logits must have unit column stride", lambda: dis(z.t(), ii, t)),
            (TypeError, "ids must be int32 or int64", lambda: dis(z, t, t)),
            (ValueError, "ids must have shape", lambda: dis(z, ii[:3], t)),
            (ValueError, "at most 1024", lambda: dis(z, ii.expand(4, 1025).contiguous(), t)),
            (ValueError, "teacher must have shape", lambda: dis(z, ii, z)),
            (TypeError, "teacher must be float32 or bfloat16", lambda: dis(z, ii, t.double())),
            (ValueError, "weights must be a contiguous vector of 4", lambda: dis(z, ii, t, weights=f[:3])),
            (TypeError, "out must have the type of logits", lambda: dis(z, ii, t, out=z.bfloat16())),
            (ValueError, "out must not be given", lambda: dis(z, ii, t, out=z.clone(), want_grad=False)),
            (ValueError, "must be a GPU tensor", lambda: dis(z, ii.cpu(), t)),
            (ValueError, "actions must be a contiguous vector of 4", lambda: pol(z, ii, f, f)),
            (TypeError, "actions must be int32 or int64", lambda: pol(z, f, f, f)),
            (TypeError, "old_logp must be float32", lambda: pol(z, i, f.double(), f)),
            (ValueError, "advantages must be a contiguous vector", lambda: pol(z, i, f, f[:1])),
            (ValueError, "ref_logp must be a contiguous vector", lambda: pol(z, i, f, f, ref_logp=f[:1]))):
        with pytest.raises(err, match=match):
            call()
    for status, call in ((muon.MUON_EINVAL, lambda: dis(z, ii, t, temperature=0.0)), (muon.MUON_EINVAL, lambda: dis(z, ii, t, temperature=-1.0)),
                         (muon.MUON_EINVAL, lambda: pol(z, i, f, f, temperature=float("nan"))),
                         (muon.MUON_EINVAL, lambda: pol(z, i, f, f, clip=1.5)), (muon.MUON_EINVAL, lambda: pol(z, i, f, f, clip_high=-0.1)),
                         (muon.MUON_EINVAL, lambda: pol(z, i, f, f, kl_coef=float("inf"))),
                         (muon.MUON_EALIAS, lambda: dis(z, ii, t, out=z)), (muon.MUON_EALIAS, lambda: pol(z, i, f, f, out=z))):
        with pytest.raises(muon.LibMuonError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
def test_a_kl_coefficient_of_zero_takes_no_part(dtype):
    """Whatever the reference: exp(d) past the largest number, an action that cannot be."""
    z = torch.randn(4, 900, generator=gen(2))
    z[0, 3], z[1, 3] = -float("inf"), -200.0
    actions, adv = torch.full((4,), 3, device=DEV), torch.tensor([1.0, -1.0, 0.5, 0.0]).to(DEV)
    old, ref = torch.full((4,), -7.0, device=DEV), torch.tensor([-1.0, 0.0, -5.0, float("inf")]).to(DEV)
    z = z.to(dtype).to(DEV)
    with_ref = muon.policy_loss(z, actions, old, adv, ref_logp=ref)
    without = muon.policy_loss(z, actions, old, adv)
    for a, b in zip(with_ref, without):
        assert torch.equal(a, b) and not torch.isnan(a).any()


@pytest.mark.parametrize("temperature", [1.0, 1.25, 2.0, 4.0])
@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
def test_entries_on_a_column_of_the_lowest_value(dtype, temperature):
    """A column masked with the type's lowest value has a log-probability of about -3e38 / temperature, not of -infinity.
    Relative to it: the difference, log2(e) / temperature (two roundings), the product with it, the log's subtraction and the
    product with ln 2 (two): 8 u; the log of the sum is 2^-120 of it."""
    low = torch.finfo(dtype).min
    z = torch.randn(2, 700, generator=gen(4)).to(dtype)
    z[:, 5] = low
    want = (O.log_softmax(np64(z) / temperature))[:, 5]
    off = 8 * U * np.abs(want)
    zero = torch.zeros(2, device=DEV)
    loss, logp, grad = muon.policy_loss(z.to(DEV), torch.full((2,), 5, device=DEV), zero - 1, zero + 1, temperature=temperature)
    assert (np.abs(np64(logp) - want) <= off).all() and not loss.any() and not grad.any()
    # a quarter of the teacher's mass on it
    loss, grad = muon.distill_loss(z.to(DEV), torch.tensor([[5, 6, 7, 8]] * 2, device=DEV), torch.zeros(2, 4, device=DEV), temperature=temperature,
                                   weights=zero + 1 / 8)
    want = -want / 4 * temperature ** 2 / 8
    assert (np.abs(np64(loss) - want) <= (8 + 30) * U * want).all() and torch.isfinite(grad).all()

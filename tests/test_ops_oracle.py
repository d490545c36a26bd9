"""The 64-bit oracle of the training operators against closed forms,
differences and torch's own 8-bit conversion (CPU)."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as O


def test_e4m3_table_and_rounding_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    vals = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_decode(codes), vals, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(size=4000), rng.normal(size=4000) * 2.0 ** -8,
                        (O.E4M3[1:] + O.E4M3[:-1]) / 2, O.E4M3, [0.0, -0.0, 2.0 ** -10, 2.0 ** -11]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_encode(x), want)


def test_scale_is_the_smallest_that_holds_the_group():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(40, 70)) * 2.0 ** rng.integers(-130, 125, (40, 1))
    x[3] = 0.0
    e = O.scale_exponents(x)
    assert e.shape == (40, 3) and e.min() >= -117 and e.max() <= 119
    amax = np.abs(O._grouped(x)).max(-1)
    free = (e > -117) & (e < 119)
    assert np.all(amax[free] <= 448 * 2.0 ** e[free].astype(float)) and np.all(amax[free] > 224 * 2.0 ** e[free].astype(float))
    assert np.all(e[3] == -117)
    # exactly 448 * 2^k keeps the exponent k, the next fp32 number above does not
    v = np.zeros((2, 32))
    v[0, 5], v[1, 5] = 448.0 * 8, np.nextafter(np.float32(448.0 * 8), np.float32(np.inf))
    assert O.scale_exponents(v).ravel().tolist() == [3, 4]


def test_pack_error_bound_and_non_finite():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(16, 100)) * 10.0 ** rng.uniform(-6, 6, (16, 100))
    codes, scales = O.act8_pack(x)
    back = O.act8_unpack(codes, scales)
    s = np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)[:, :100]
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))
    y = x.copy()
    y[0, 3], y[1, 40], y[2, 99] = np.nan, np.inf, -np.inf
    c2, s2 = O.act8_pack(y)
    assert np.isnan(O.e4m3_decode(c2))[[0, 1, 2], [3, 40, 99]].all() and np.isnan(O.act8_unpack(c2, s2)).sum() == 3


def _difference(f, x, i, h):
    a, b = x.copy(), x.copy()
    a.flat[i] += h
    b.flat[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("gain", [False, True])
def test_norm_gradient_by_differences(gain):
    rng = np.random.default_rng(3)
    x, dy, dres = rng.normal(size=(3, 3, 11))
    g = rng.normal(size=11) if gain else None
    _, _, n, rstd = O.rmsnorm(x, g, None, 1e-3)
    dx, dgain = O.rmsnorm_grad(dy, n, rstd, g, dres)

    def loss(v):
        h, y, _, _ = O.rmsnorm(v, g, None, 1e-3)
        return (y * dy).sum() + (h * dres).sum()
    for i in range(x.size):
        assert abs(_difference(loss, x, i, 1e-5) - dx.flat[i]) < 1e-8
    if gain:
        for i in range(11):
            assert abs(_difference(lambda v: (O.rmsnorm(x, v, None, 1e-3)[1] * dy).sum(), g, i, 1e-5) - dgain[i]) < 1e-8


def test_gate_wgrad_and_embed_gradients_by_differences():
    rng = np.random.default_rng(4)
    gate, up, da = rng.normal(size=(3, 4, 5)) * 2
    dgate, dup, a = O.swiglu_grad(da, gate, up)
    assert np.allclose(a, O.swiglu(gate, up))
    for i in range(gate.size):
        assert abs(_difference(lambda v: (O.swiglu(v, up) * da).sum(), gate, i, 1e-5) - dgate.flat[i]) < 1e-8
        assert abs(_difference(lambda v: (O.swiglu(gate, v) * da).sum(), up, i, 1e-5) - dup.flat[i]) < 1e-8
    x, w, dy, gain = rng.normal(size=(6, 5)), rng.normal(size=(3, 5)), rng.normal(size=(6, 3)), rng.normal(size=5)
    dw = O.wgrad(dy, x, gain)
    for i in range(w.size):
        assert abs(_difference(lambda v: ((x * gain) @ v.T * dy).sum(), w, i, 1e-4) - dw.flat[i]) < 1e-9
    table, ids = rng.normal(size=(7, 3)), np.array([2, 2, -1, 6, 0, 7, 2])
    de = rng.normal(size=(7, 3))
    grad = O.embed_grad(de, ids, 7, 1.5)
    for i in range(table.size):
        assert abs(_difference(lambda v: (O.embed(v, ids, 1.5) * de).sum(), table, i, 1e-4) - grad.flat[i]) < 1e-9


@pytest.mark.parametrize("nq,nk,causal", [(5, 5, True), (4, 6, True), (6, 4, True), (3, 7, False), (2, 0, False)])
def test_attention_against_loops_and_differences(nq, nk, causal):
    rng = np.random.default_rng(nq * 10 + nk)
    q, k, v, do = (rng.normal(size=(n, 3)) for n in (nq, nk, nk, nq))
    o, lse = O.attention(q, k, v, 0.7, causal)
    for i in range(nq):
        seen = [j for j in range(nk) if not causal or j <= i + nk - nq]
        e = [np.exp(0.7 * float(q[i] @ k[j])) for j in seen]
        if not seen:
            assert not o[i].any() and lse[i] == -np.inf
            continue
        assert abs(lse[i] - np.log(sum(e))) < 1e-12
        assert np.allclose(o[i], sum(w * v[j] for w, j in zip(e, seen)) / sum(e), rtol=1e-12)
    grads = O.attention_grad(do, q, k, v, o, lse, 0.7, causal)
    at = [q, k, v]
    for which, g in enumerate(grads):
        def value(x):
            return (O.attention(*(x if n == which else t for n, t in enumerate(at)), 0.7, causal)[0] * do).sum()
        for i in range(g.size):
            assert abs(_difference(value, at[which], i, 1e-5) - g.flat[i]) < 1e-8


def test_losses_against_torch_and_differences():
    rng = np.random.default_rng(4)
    z, w = rng.normal(size=(4, 9)), np.array([1.0, 0.0, 0.5, -2.0])
    ids, teacher = np.array([[1, 1, 4], [0, 1, 2], [-1, 9, 3], [8, 0, 5]]), rng.normal(size=(4, 3))
    loss, grad = O.distill(z, ids, teacher, 1.5, w)
    for t in range(4):
        live = [(i, x) for i, x in zip(ids[t], teacher[t]) if 0 <= i < 9]
        p = torch.softmax(torch.tensor([x for _, x in live]) / 1.5, 0)
        logq = torch.log_softmax(torch.from_numpy(z[t]) / 1.5, 0)
        want = sum(float(a * (torch.log(a) - logq[i])) for a, (i, _) in zip(p, live)) * 2.25 * w[t]
        assert abs(loss[t] - want) < 1e-12
    actions, old, adv, ref = np.array([3, 1, 8, 9]), np.full(4, -2.2), np.array([1.0, 1.0, -0.5, 1.0]), np.full(4, -2.0)
    args = (actions, old, adv, ref, 0.2, 0.3, 0.1, 1.5, w)
    ploss, logp, pgrad = O.policy(z, *args)
    assert not ploss[[1, 3]].any() and not pgrad[[1, 3]].any()
    for t in (0, 2):
        lp = float(torch.log_softmax(torch.from_numpy(z[t]) / 1.5, 0)[actions[t]])
        r = np.exp(lp - old[t])
        want = -min(r * adv[t], min(max(r, 0.8), 1.3) * adv[t]) + 0.1 * (np.exp(ref[t] - lp) - (ref[t] - lp) - 1)
        assert abs(logp[t] - lp) < 1e-12 and abs(ploss[t] - w[t] * want) < 1e-12
    for i in range(z.size):
        assert abs(_difference(lambda x: O.distill(x, ids, teacher, 1.5, w)[0].sum(), z, i, 1e-5) - grad.flat[i]) < 1e-8
        assert abs(_difference(lambda x: O.policy(x, *args)[0].sum(), z, i, 1e-5) - pgrad.flat[i]) < 1e-8

"""The training operators in 64 bits (numpy), written from their formulas.
Test infrastructure only."""
import numpy as np

GROUP = 32
MIN_E, MAX_E = -117, 119


def _e4m3_values():
    """Values of the codes 0 .. 0x7E (4 exponent bits with bias 7, 3 mantissa bits; 0x7F is NaN)."""
    c = np.arange(0x7F)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = _e4m3_values()


def e4m3_encode(a):
    """Codes of the nearest values of |a| <= 448 (ties to the even code), sign kept; NaN for NaN."""
    a = np.asarray(a, dtype=np.float64)
    mag = np.abs(a)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6)
    e = np.where(mag > 0, e, -6)
    step = 2.0 ** (e - 3)
    q = np.rint(mag / step) * step
    code = np.searchsorted(E4M3, np.where(np.isnan(q), 0.0, q)).astype(np.uint8)
    code = np.where(np.isnan(a), np.uint8(0x7F), code)
    return (code | (np.signbit(a).astype(np.uint8) << 7)).astype(np.uint8)


def e4m3_decode(code):
    code = np.asarray(code, dtype=np.uint8)
    mag = np.append(E4M3, np.nan)[code & 0x7F]
    return np.where(code & 0x80, -mag, mag)


def _grouped(x):
    rows, cols = x.shape
    g = -(-cols // GROUP)
    out = np.zeros((rows, g * GROUP))
    out[:, :cols] = x
    return out.reshape(rows, g, GROUP)


def scale_exponents(x):
    """e of each group: the smallest with max finite |v| <= 448 * 2^e, in [-117, 119]."""
    v = _grouped(np.asarray(x, dtype=np.float64))
    amax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)
    e = np.full(amax.shape, MIN_E)
    for _ in range(MIN_E, MAX_E):
        e = np.where((amax > 448.0 * 2.0 ** e.astype(np.float64)) & (e < MAX_E), e + 1, e)
    return e


def act8_pack(x):
    """(codes, scale bytes) of a matrix."""
    x = np.asarray(x, dtype=np.float64)
    e = scale_exponents(x)
    with np.errstate(invalid="ignore"):
        q = _grouped(np.where(np.isfinite(x), x, np.nan)) / (2.0 ** e.astype(np.float64))[..., None]
        q = np.clip(q, -448.0, 448.0)
    return e4m3_encode(q).reshape(x.shape[0], -1)[:, :x.shape[1]], (e + 127).astype(np.uint8)


def act8_unpack(codes, scales):
    s = np.repeat(2.0 ** (np.asarray(scales, dtype=np.float64) - 127), GROUP, axis=1)[:, :codes.shape[1]]
    return e4m3_decode(codes) * s


def rmsnorm(x, gain, residual, eps):
    """(h, y, n, rstd)."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    n = h * rstd[:, None]
    return h, n if gain is None else n * gain, n, rstd


def rmsnorm_grad(dy, n, rstd, gain, dres):
    """(dx, dgain) from the normalised rows."""
    gd = dy if gain is None else dy * gain
    dx = rstd[:, None] * (gd - n * (gd * n).mean(1, keepdims=True))
    return dx if dres is None else dx + dres, (dy * n).sum(0)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_grad(da, gate, up):
    """(dgate, dup, a)."""
    s = sigmoid(gate)
    return da * up * s * (1.0 + gate * (1.0 - s)), da * gate * s, gate * s * up


def wgrad(dy, x, col_gain=None, base=None):
    dw = dy.T @ x
    if col_gain is not None:
        dw = dw * col_gain
    return dw if base is None else base + dw


def embed(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    live = (ids >= 0) & (ids < len(table))
    out[live] = table[ids[live]] * scale
    return out


def embed_grad(dy, ids, vocab, scale, base=None):
    out = np.zeros((vocab, dy.shape[1])) if base is None else base.copy()
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            out[i] += dy[t] * scale
    return out


def visible(nq, nk, causal):
    """Which keys each query sees (a causal mask is aligned at the end)."""
    if not causal:
        return np.ones((nq, nk), dtype=bool)
    return np.arange(nk)[None, :] <= np.arange(nq)[:, None] + (nk - nq)


def attention(q, k, v, scale, causal):
    """(o, lse) of one sequence and head."""
    s = np.where(visible(len(q), len(k), causal), scale * (q @ k.T), -np.inf)
    top = s.max(1, initial=-np.inf, keepdims=True)
    base = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - base)
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, base + np.log(total), -np.inf)
    return (e / np.where(total > 0, total, 1.0)) @ v, lse[:, 0]


def attention_grad(do, q, k, v, o, lse, scale, causal):
    """(dq, dk, dv) of one sequence and head, from the rows' o and lse."""
    see = visible(len(q), len(k), causal)
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(see, np.exp(scale * (q @ k.T) - lse[:, None]), 0.0)
    ds = p * (do @ v.T - (do * o).sum(1, keepdims=True))
    return scale * (ds @ k), scale * (ds.T @ q), p.T @ do


def log_softmax(x):
    top = x.max(1, keepdims=True)
    return x - top - np.log(np.exp(x - top).sum(1, keepdims=True))


def distill(logits, ids, teacher, temperature, weights):
    """(loss, dlogits), row by row, entry by entry."""
    loss, grad = np.zeros(len(logits)), np.zeros(logits.shape)
    for t, w in enumerate(weights):
        live = (ids[t] >= 0) & (ids[t] < logits.shape[1]) & (teacher[t] != -np.inf)
        if w == 0 or not live.any():
            continue
        logp = log_softmax(teacher[t:t + 1, live] / temperature)[0]
        logq = log_softmax(logits[t:t + 1] / temperature)[0]
        grad[t] = np.exp(logq)
        for i, lp in zip(ids[t][live], logp):
            if np.exp(lp) > 0:
                loss[t] += np.exp(lp) * (lp - logq[i])
            grad[t, i] -= np.exp(lp)
        loss[t] *= w * temperature ** 2
        grad[t] *= w * temperature
    return loss, grad


def policy(logits, actions, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, temperature, weights):
    """(loss, logp, dlogits), row by row."""
    loss, logp, grad = np.zeros(len(logits)), np.zeros(len(logits)), np.zeros(logits.shape)
    for t, (a, w, adv) in enumerate(zip(actions, weights, advantages)):
        if w == 0 or not 0 <= a < logits.shape[1]:
            continue
        logq = log_softmax(logits[t:t + 1] / temperature)[0]
        logp[t] = logq[a]
        r = np.exp(logq[a] - old_logp[t])
        held = np.clip(r, 1 - clip_low, 1 + clip_high)
        loss[t], g = -min(r * adv, held * adv), -adv * r * (r * adv <= held * adv)
        if ref_logp is not None:
            d = ref_logp[t] - logq[a]
            loss[t] += kl_coef * (np.exp(d) - d - 1)
            g += kl_coef * (1 - np.exp(d))
        loss[t] *= w
        grad[t] = -np.exp(logq)
        grad[t, a] += 1
        grad[t] *= w * g / temperature
    return loss, logp, grad

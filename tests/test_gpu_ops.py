"""The training operators on the GPU against the 64-bit oracle.

Tolerances.  u = 2^-24 is the unit of fp32.  A sum of n terms in any order is
off by at most n u times the sum of the terms' magnitudes; sums of integers
below 2^24 are exact, which the integer cases use: there the results have to be
equal.  Row statistics go through at most 16 terms in a lane, 6 steps in a wave,
16 waves and a handful of roundings, below 64 u = 2^-18 relative (the terms of
the mean square are positive).  The fast exponential's argument is off by at
most |g| u, its value by |g| u + 2^-22 relative, for |g| <= 88 below 2^-17; with
the reciprocal and the products 2^-16 covers the gated unit.  A result has to be the rounding to
its type of some value within its bound."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from oracle import ops_oracle as O
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STAT, GATE = 2.0 ** -17, 2.0 ** -16
TYPES = [torch.float32, torch.bfloat16]
ids_of = lambda v: str(v).replace("torch.", "").replace(" ", "")  # noqa: E731


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed)).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def on_gpu(t, layout="plain"):
    """The tensor on the GPU: contiguous, or rows at odd strides and offsets inside a larger buffer."""
    if t is None or layout == "plain" or t.dim() < 2:
        return None if t is None else t.to(DEV)
    rows, cols = t.shape
    buf = torch.full((rows * (cols + 5) + 3,), float("nan"), device=DEV).to(t.dtype)
    view = buf[3:].view(rows, cols + 5)[:, 1:1 + cols] if rows else buf[:0].view(0, cols)
    view.copy_(t.to(DEV))
    return view


def values(x8):
    return O.act8_unpack(x8.codes.view(torch.uint8).cpu().numpy(), x8.scales.cpu().numpy())


def check_pack_equal(x8, x):
    codes, scales = O.act8_pack(np64(x))
    got = x8.codes.view(torch.uint8).cpu().numpy()
    nan = (codes & 0x7F) == 0x7F
    assert np.array_equal(x8.scales.cpu().numpy(), scales)
    assert np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], codes[~nan])


def check_pack_near(x8, ref, rel):
    """8-bit values of a result that is off by at most rel (relative) before its rounding."""
    e = x8.scales.cpu().numpy().astype(np.float64) - 127
    s = 2.0 ** e
    amax = np.abs(O._grouped(ref)).max(-1)
    assert np.all(amax <= 448 * s * (1 + rel))
    assert np.all((amax * (1 + rel) >= 224 * s) | (e == -117))
    s = np.repeat(s, 32, axis=1)[:, :ref.shape[1]]
    err = np.abs(values(x8) - ref)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) * (1 + 2 * rel) + 2 * rel * np.abs(ref))


def rounded(v, dtype):
    """64-bit values rounded once to the type (to nearest even)."""
    bits = 24 if dtype == torch.float32 else 8
    m, e = np.frexp(v)
    low = np.maximum(e, -125)                                   # subnormals keep the spacing 2^(-125 - bits)
    return np.ldexp(np.rint(np.ldexp(m, bits + e - low)), low - bits)


def near(got, ref, dtype, rel, scale=None):
    """The result is the rounding of a value within rel * scale (by default the result's own magnitude) of ref."""
    tol = rel * (np.abs(ref) if scale is None else scale) + 1e-30
    assert got.dtype == dtype and got.shape == ref.shape
    v = np64(got)
    out = (v < rounded(ref - tol, dtype)) | (v > rounded(ref + tol, dtype)) | np.isnan(v)
    assert not out.any(), f"{out.sum()} outside; worst {np.max(np.abs(v - ref)[out] / tol[out])} times the bound"


# ------------------------------------------------------------ pack, unpack ----
@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (5, 33), (7, 100), (64, 256), (33, 1001), (2, 4096)])
@pytest.mark.parametrize("layout", ["plain", "odd"])
def test_pack_and_unpack(dtype, rows, cols, layout):
    x = (randn(rows * cols, rows, cols) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=gen(1)).float())).to(dtype)
    xg = on_gpu(x, layout)
    x8 = muon.act8_pack(xg)
    check_pack_equal(x8, x)
    for out in TYPES:
        back = muon.act8_unpack(x8, out)
        assert back.dtype == out and np.array_equal(np64(back), values(x8))
    if layout == "odd":            # codes and scales at odd places too
        wide = torch.zeros(rows, cols + 3, dtype=torch.uint8, device=DEV)
        wide[:, 1:1 + cols] = x8.codes.view(torch.uint8)
        c8 = muon.Act8(wide.view(torch.float8_e4m3fn)[:, 1:1 + cols], x8.scales)
        assert np.array_equal(np64(muon.act8_unpack(c8)), values(x8))


def test_pack_every_code_tie_and_extreme():
    """All representable values, all halfway points, the ends of the scale's range, infinities, NaN, zeros, subnormals."""
    rows = []
    for e in (-117, -116, -1, 0, 3, 118, 119):
        s = 2.0 ** e
        mid = (O.E4M3[1:] + O.E4M3[:-1]) / 2
        v = np.concatenate([O.E4M3, mid, mid * (1 + 2.0 ** -20), -O.E4M3, -mid])
        v = np.resize(v, (len(v) + 30) // 31 * 31).reshape(-1, 31)
        rows.append(np.concatenate([np.full((len(v), 1), 448.0), v], axis=1) * s)   # 448 holds the scale at e
    big = np.float64(np.finfo(np.float32).max)
    special = np.zeros((8, 32))
    special[1, :4] = [np.inf, 1.0, -np.inf, 300.0]
    special[2, :3] = [np.nan, 2.0 ** -20, -np.nan]
    special[3, :4] = [big, -big, 448 * 2.0 ** 119, 2.0 ** 127]
    special[4, :4] = [2.0 ** -149, -2.0 ** -149, 2.0 ** -126, 2.0 ** -130]
    special[5, :2] = [np.inf, np.nan]
    special[6, :2] = [-0.0, 0.0]
    special[7, :3] = [448.0, np.nextafter(np.float32(448.0), np.float32(500)), 224.0]
    x = torch.from_numpy(np.concatenate(rows + [special]).astype(np.float32))
    x8 = muon.act8_pack(x.to(DEV))
    check_pack_equal(x8, x)
    finite = np.isfinite(np64(x))
    assert np.array_equal(np.isfinite(values(x8)), finite)          # finite values stay finite
    for dt in TYPES:
        assert np.array_equal(np64(muon.act8_unpack(x8, dt)), values(x8), equal_nan=True)
    check_pack_equal(muon.act8_pack(x.bfloat16().to(DEV)), x.bfloat16())


# -------------------------------------------------------------------- norm ----
NORM_SIZES = [(1, 1), (1, 768), (2, 40), (5, 512), (9, 513), (3, 1000), (4, 1025), (6, 2048), (3, 2049), (2, 4100), (3, 8192),
              (2, 8200), (2, 16384), (67, 96)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("form", ["plain", "residual", "odd"])
def test_norm(dtype, rows, cols, form):
    x, r = randn(cols, rows, cols, dtype=dtype), randn(cols + 1, rows, cols, dtype=dtype)
    r = None if form == "plain" else r
    gain = None if form == "plain" and cols % 2 else 1 + 0.3 * randn(7, cols)
    layout = "odd" if form == "odd" else "plain"
    xg = on_gpu(x, layout)
    h, y, n8, rstd = muon.rmsnorm_act8(xg, on_gpu(gain), residual=on_gpu(r, layout), eps=1e-5)
    ho, yo, no, ro = O.rmsnorm(np64(x), None if gain is None else np64(gain), None if r is None else np64(r), np.float64(np.float32(1e-5)))
    if r is None:
        assert h is xg
    else:
        near(h, ho, dtype, U)
    near(y, yo, dtype, STAT)
    near(rstd, ro, torch.float32, STAT)
    check_pack_near(n8, no, STAT)
    h2, y2 = muon.rmsnorm_act8(xg, on_gpu(gain), residual=on_gpu(r, layout), eps=1e-5, save=False)
    assert torch.equal(y2, y) and torch.equal(h2, h)


@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(3000, 64), (2500, 1100), (1300, 4096)])
@pytest.mark.parametrize("form", ["plain", "residual", "odd"])
def test_norm_gradient(dtype, rows, cols, form):
    n8 = muon.act8_pack(randn(cols, rows, cols).to(DEV))
    n, rstd = values(n8), torch.rand(rows, generator=gen(3)) + 0.5
    dy, dres = randn(cols + 2, rows, cols, dtype=dtype), randn(cols + 3, rows, cols, dtype=dtype)
    dres = None if form == "plain" else dres
    gain = None if form == "plain" and cols % 2 else 1 + 0.3 * randn(7, cols)
    layout = "odd" if form == "odd" else "plain"
    args = (on_gpu(dy, layout), n8, rstd.to(DEV), on_gpu(gain))
    dx, dgain = muon.rmsnorm_act8_grad(*args, dres=on_gpu(dres, layout))
    g = 1.0 if gain is None else np64(gain)
    dxo, dgo = O.rmsnorm_grad(np64(dy), n, np64(rstd), None if gain is None else np64(gain), None if dres is None else np64(dres))
    gd = np64(dy) * g
    scale = np64(rstd)[:, None] * (np.abs(gd) + np.abs(n) * np.abs(gd * n).mean(1, keepdims=True))
    near(dx, dxo, dtype, STAT, scale + (0 if dres is None else np.abs(np64(dres))))
    near(dgain, dgo, torch.float32, (rows + 2) * U, np.abs(np64(dy) * n).sum(0))
    again, none = muon.rmsnorm_act8_grad(*args, dres=on_gpu(dres, layout), want_dgain=False)
    assert none is None and torch.equal(again, dx)
    dx2, dgain2 = muon.rmsnorm_act8_grad(*args, dres=on_gpu(dres, layout))
    assert torch.equal(dx2, dx) and torch.equal(dgain2, dgain)


def test_norm_gain_gradient_is_exact_on_integers():
    for rows, cols in ((1, 8), (777, 96), (4099, 1000), (2100, 2304)):
        n = torch.randint(-8, 9, (rows, cols), generator=gen(rows)).float()
        dy = torch.randint(-4, 5, (rows, cols), generator=gen(cols)).bfloat16()
        n8 = muon.act8_pack(n.to(DEV))
        assert np.array_equal(values(n8), np64(n))
        _, dgain = muon.rmsnorm_act8_grad(dy.to(DEV), n8, torch.ones(rows, device=DEV))
        assert np.array_equal(np64(dgain), (np64(dy) * np64(n)).sum(0)), (rows, cols)


def test_norm_gradient_by_differences():
    """Rows whose normalised values 8 bits hold exactly (1 / 2 and 3 / 2 in the ratio 5 : 3 and ones have mean square 1),
    so that the 8-bit backward pass is the true gradient; central differences in 64 bits."""
    g = gen(11)
    base = torch.tensor([0.5] * 5 + [1.5] * 3 + [1.0] * 8).repeat(3)
    h = torch.stack([base[torch.randperm(48, generator=g)] * (1 - 2 * torch.randint(0, 2, (48,), generator=g)) * s for s in (1.0, 4.0)])
    gain, dy, dres = 1 + 0.3 * randn(1, 48), randn(2, 2, 48), randn(3, 2, 48)
    _, _, n8, rstd = muon.rmsnorm_act8(h.to(DEV), gain.to(DEV), eps=0.0)
    assert np.array_equal(values(n8), np64(h) / np.array([[1.0], [4.0]]))
    dx, dgain = muon.rmsnorm_act8_grad(dy.to(DEV), n8, rstd, gain.to(DEV), dres=dres.to(DEV))

    def loss(hv, gv):
        hh, y, _, _ = O.rmsnorm(hv, gv, None, 0.0)
        return (y * np64(dy)).sum() + (hh * np64(dres)).sum()
    hv, gv, step = np64(h), np64(gain), 1e-5
    for i in range(h.numel()):
        a, b = hv.copy(), hv.copy()
        a.flat[i] += step
        b.flat[i] -= step
        # differences: step^2 / 6 times third derivatives below 50, roundings below 1e-9; fp32 results: 2^-17 of values below 8
        assert abs((loss(a, gv) - loss(b, gv)) / (2 * step) - np64(dx).flat[i]) < 1e-4
    for i in range(48):
        a, b = gv.copy(), gv.copy()
        a[i] += step
        b[i] -= step
        assert abs((loss(hv, a) - loss(hv, b)) / (2 * step) - np64(dgain)[i]) < 1e-4


def test_norm_bad_values_stay_in_their_row():
    x = randn(5, 6, 300)
    x[2, 17], x[4, 299] = float("inf"), float("nan")
    _, y, n8, rstd = muon.rmsnorm_act8(x.to(DEV))
    bad = ~np.isfinite(np64(y)).all(1)
    assert bad.tolist() == [False, False, True, False, True, False]
    ok = [0, 1, 3, 5]
    near(y[ok], O.rmsnorm(np64(x)[ok], None, None, 1e-6)[1], torch.float32, STAT)
    zero = torch.zeros(3, 64, device=DEV)
    _, y, n8, rstd = muon.rmsnorm_act8(zero, eps=1e-6)
    assert not y.any() and not values(n8).any() and np.allclose(np64(rstd), 1e3, rtol=STAT)


# -------------------------------------------------------------------- gate ----
@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (3, 40), (7, 33), (17, 1536), (5, 1001), (2, 14336)])
@pytest.mark.parametrize("layout", ["plain", "halves", "odd"])
def test_gate(dtype, rows, cols, layout):
    gu = (4 * randn(cols, rows, 2 * cols)).to(dtype)
    gu[0, 0] = -87.0
    gate, up = gu[:, :cols], gu[:, cols:]
    if layout == "halves":
        buf = gu.to(DEV)
        gg, ug = buf[:, :cols], buf[:, cols:]
    else:
        gg, ug = on_gpu(gate.contiguous(), layout), on_gpu(up.contiguous(), layout)
    a, gate8, up8 = muon.swiglu_act8(gg, ug)
    near(a, O.swiglu(np64(gate), np64(up)), dtype, GATE)
    check_pack_equal(gate8, gate)
    check_pack_equal(up8, up)
    assert torch.equal(muon.swiglu_act8(gg, ug, save=False), a)

    da = randn(cols + 1, rows, cols, dtype=dtype)
    g, u = values(gate8), values(up8)
    outs = {}
    if layout == "halves":
        both = torch.full((rows, 2 * cols), float("nan"), device=DEV, dtype=dtype)
        outs = dict(dgate=both[:, :cols], dup=both[:, cols:])
    dgate, dup, a8 = muon.swiglu_act8_grad(on_gpu(da, layout if layout == "odd" else "plain"), gate8, up8, **outs)
    dgo, duo, ao = O.swiglu_grad(np64(da), g, u)
    s = O.sigmoid(g)
    near(dgate, dgo, dtype, GATE, np.abs(np64(da) * u) * s * (1 + np.abs(g)))
    near(dup, duo, dtype, GATE)
    check_pack_near(a8, ao, GATE)
    dg2, du2, none = muon.swiglu_act8_grad(da.to(DEV), gate8, up8, want_a8=False)
    assert none is None and torch.equal(dg2, dgate) and torch.equal(du2, dup)


def test_gate_gradient_by_differences():
    g8 = torch.tensor([[k * 0.25 for k in range(-16, 16)]])          # values that 8 bits hold exactly
    u8 = torch.tensor([[((k * 7) % 16 - 8) * 0.5 for k in range(32)]])
    da = randn(4, 1, 32)
    _, gate8, up8 = muon.swiglu_act8(g8.to(DEV), u8.to(DEV))
    assert np.array_equal(values(gate8), np64(g8)) and np.array_equal(values(up8), np64(u8))
    dgate, dup, _ = muon.swiglu_act8_grad(da.to(DEV), gate8, up8)
    g, u, d, step = np64(g8), np64(u8), np64(da), 1e-5
    # elementwise: differences are off by step^2 / 6 times third derivatives below 20, the results by 2^-16 of values below 32
    assert np.all(np.abs((O.swiglu(g + step, u) - O.swiglu(g - step, u)) / (2 * step) * d - np64(dgate)) < 5e-4)
    assert np.all(np.abs((O.swiglu(g, u + step) - O.swiglu(g, u - step)) / (2 * step) * d - np64(dup)) < 5e-4)


def test_gate_extremes():
    g = torch.tensor([[-3e38, -200.0, -89.0, -0.0, 0.0, 89.0, 200.0, 1e30]], device=DEV)
    a, _, _ = muon.swiglu_act8(g, torch.ones_like(g))
    want = np64(g) * O.sigmoid(np64(g))
    assert np.allclose(np64(a), want, rtol=GATE, atol=1e-30)


# ------------------------------------------------------------------- wgrad ----
WGRAD_SIZES = [(1, 1, 1), (1, 8, 32), (31, 16, 33), (32, 128, 128), (33, 80, 96), (100, 129, 257), (257, 256, 768), (300, 1, 500),
               (300, 500, 1), (1000, 80, 1536), (513, 300, 1000), (2000, 40, 64), (96, 520, 264), (4097, 24, 40)]


def int_case(tokens, n, k, seed=0):
    """Integers whose sums stay below 2^24, so fp32 sums in any order are exact."""
    lim = 8 if tokens * 64 < 1 << 24 else 2
    dy = torch.randint(-lim, lim + 1, (tokens, n), generator=gen(seed + tokens)).bfloat16()
    x = torch.randint(-8, 9, (tokens, k), generator=gen(seed + n)).float()
    return dy, x


@pytest.mark.parametrize("tokens,n,k", WGRAD_SIZES)
@pytest.mark.parametrize("layout", ["plain", "odd"])
def test_wgrad_is_exact_on_integers(tokens, n, k, layout):
    dy, x = int_case(tokens, n, k)
    want = np64(dy).T @ np64(x)
    x8 = muon.act8_pack(x.to(DEV))
    if layout == "odd":
        wide = torch.zeros(tokens, k + 3, dtype=torch.uint8, device=DEV)
        wide[:, 1:1 + k] = x8.codes.view(torch.uint8)
        x8 = muon.Act8(wide.view(torch.float8_e4m3fn)[:, 1:1 + k], x8.scales)
    dyg = on_gpu(dy, layout)
    dw = muon.act8_wgrad(dyg, x8)
    assert dw.dtype == torch.float32 and np.array_equal(np64(dw), want)
    half = muon.act8_wgrad(dyg, x8, dtype=torch.bfloat16)
    assert torch.equal(half.cpu(), torch.from_numpy(want).float().bfloat16())
    # the gain (powers of two here) and the sum into what is there, in a strided output
    gain = torch.exp2(torch.randint(-1, 2, (k,), generator=gen(5)).float())
    base = torch.randint(-50, 50, (n, k), generator=gen(6)).float()
    out = on_gpu(base, layout)
    got = muon.act8_wgrad(dyg, x8, col_gain=gain.to(DEV), out=out, accumulate=True)
    assert got.data_ptr() == out.data_ptr() and np.array_equal(np64(got), np64(base) + want * np64(gain))


@pytest.mark.parametrize("tokens,n,k", [(260, 4352, 4100), (1000, 4100, 4352), (33, 5000, 4099), (640, 2304, 4608)])
def test_wgrad_of_large_tiles_is_exact_on_integers(tokens, n, k):
    """Sizes that 256 x 256 tiles serve, more of them than the chip holds at once: the last ones in token ranges."""
    dy, x = int_case(tokens, n, k)
    want = (dy.to(DEV).double().t().contiguous() @ x.to(DEV).double())
    x8 = muon.act8_pack(x.to(DEV))
    assert torch.equal(muon.act8_wgrad(dy.to(DEV), x8).double(), want)
    gain = torch.exp2(torch.randint(-1, 2, (k,), generator=gen(5)).float()).to(DEV)
    out = torch.ones(n, k + 3, device=DEV)[:, 1:1 + k]
    muon.act8_wgrad(dy.to(DEV), x8, col_gain=gain, out=out, accumulate=True)
    assert torch.equal(out.double(), 1 + want * gain)
    assert torch.equal(muon.act8_wgrad(dy.to(DEV), x8, dtype=torch.bfloat16), want.float().bfloat16())


@pytest.mark.parametrize("tokens,n,k", [(700, 200, 300), (64, 1024, 96), (3001, 80, 1536)])
def test_wgrad_random(tokens, n, k):
    dy, x8 = randn(1, tokens, n, dtype=torch.bfloat16), muon.act8_pack((randn(2, tokens, k) * torch.exp2(4 * randn(3, tokens, 1))).to(DEV))
    gain = 1 + 0.2 * randn(4, k)
    x = values(x8)
    want, mag = O.wgrad(np64(dy), x, np64(gain)), np.abs(np64(dy)).T @ np.abs(x) * np.abs(np64(gain))
    dw = muon.act8_wgrad(dy.to(DEV), x8, col_gain=gain.to(DEV))
    near(dw, want, torch.float32, (tokens + 4) * U, mag)
    assert torch.equal(dw, muon.act8_wgrad(dy.to(DEV), x8, col_gain=gain.to(DEV)))        # the same bits again
    near(muon.act8_wgrad(dy.to(DEV), x8, col_gain=gain.to(DEV), dtype=torch.bfloat16), want, torch.bfloat16, (tokens + 4) * U, mag)


def test_wgrad_bad_values_stay_in_their_row_and_column():
    dy, x = int_case(100, 150, 170)
    dy[40, 7] = float("nan")
    x[99, 160] = float("inf")
    dw = np64(muon.act8_wgrad(dy.to(DEV), muon.act8_pack(x.to(DEV))))
    bad = np.zeros((150, 170), bool)
    bad[7, :] = bad[:, 160] = True
    assert np.array_equal(~np.isfinite(dw), bad)


def test_wgrad_of_no_tokens():
    x8 = muon.Act8(torch.empty(0, 40, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(0, 2, dtype=torch.uint8, device=DEV))
    dy = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV)
    assert not muon.act8_wgrad(dy, x8).any()
    out = torch.full((24, 40), 3.0, device=DEV)
    assert (muon.act8_wgrad(dy, x8, out=out, accumulate=True) == 3).all()
    assert not muon.act8_wgrad(dy, x8, out=out).any()
    n8 = x8
    dx, dgain = muon.rmsnorm_act8_grad(torch.empty(0, 40, device=DEV), n8, torch.empty(0, device=DEV))
    assert dx.shape == (0, 40) and not dgain.any()
    assert muon.act8_pack(torch.empty(0, 40, device=DEV)).codes.shape == (0, 40)
    assert muon.embed(torch.ones(5, 8, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)).shape == (0, 8)
    assert not muon.embed_grad(torch.empty(0, 8, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), 5).any()


# --------------------------------------------------------------- embedding ----
@pytest.mark.parametrize("table_dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("out_dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (5, 10, 64), (300, 1000, 33), (37, 300, 4096), (1025, 50, 520)])
def test_embed(table_dtype, out_dtype, tokens, vocab, cols):
    table = randn(1, vocab, cols, dtype=table_dtype)
    ids = torch.randint(-2, vocab + 2, (tokens,), generator=gen(2))
    scale = 1.7
    want = torch.zeros(tokens, cols)
    live = (ids >= 0) & (ids < vocab)
    want[live] = table[ids[live]].float() * torch.tensor(scale, dtype=torch.float32)
    for it in (torch.int64, torch.int32):
        for layout in ("plain", "odd"):
            out = muon.embed(on_gpu(table, layout), ids.to(it).to(DEV), scale=scale, dtype=out_dtype)
            assert torch.equal(out.cpu(), want.to(out_dtype))


def embed_ids(kind, tokens, vocab):
    if kind == "uniform":
        return torch.randint(-1, vocab + 1, (tokens,), generator=gen(tokens))
    if kind == "one":                                      # every token the same id
        return torch.full((tokens,), vocab // 2)
    if kind == "none":                                     # nothing but padding
        return torch.full((tokens,), -1)
    if kind == "far":                                      # ids far outside the table, 64 bits wide
        return torch.randint(-1, 2, (tokens,), generator=gen(3)) * (1 << 40) + torch.randint(0, vocab, (tokens,), generator=gen(4))
    ids = torch.randint(0, vocab, (tokens,), generator=gen(5))
    ids[torch.rand(tokens, generator=gen(6)) < 0.6] = 3 % vocab   # one id of most tokens, first and last rows used
    ids[0], ids[-1] = 0, vocab - 1
    return ids


@pytest.mark.parametrize("kind", ["uniform", "one", "none", "far", "skewed"])
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 8), (2, 7, 5), (63, 100, 64), (65, 1, 40), (200, 255, 33), (700, 256, 72),
                                               (1500, 65536, 16), (4097, 300, 520), (9001, 70000, 24), (20000, 1000, 8), (32768, 2000, 8)])
def test_embed_gradient_is_exact_on_integers(kind, tokens, vocab, cols):
    ids = embed_ids(kind, tokens, vocab)
    dy = torch.randint(-8, 9, (tokens, cols), generator=gen(7)).float()
    live = (ids >= 0) & (ids < vocab)
    want = torch.zeros(vocab, cols, dtype=torch.float64).index_add_(0, ids[live], dy[live].double()) * 0.5
    for it in (torch.int64, torch.int32) if kind != "far" else (torch.int64,):
        got = muon.embed_grad(dy.to(DEV), ids.to(it).to(DEV), vocab, scale=0.5)
        assert torch.equal(got.cpu().double(), want)
    got = muon.embed_grad(dy.bfloat16().to(DEV), ids.to(DEV), vocab, scale=0.5, dtype=torch.bfloat16)
    assert torch.equal(got.cpu(), want.float().bfloat16())
    base = torch.randint(-9, 9, (vocab, cols), generator=gen(8)).float()
    out = on_gpu(base, "odd")
    muon.embed_grad(on_gpu(dy, "odd"), ids.to(DEV), vocab, scale=0.5, out=out, accumulate=True)
    assert torch.equal(out.cpu().double(), want + base.double())


@pytest.mark.parametrize("tokens,vocab", [(256, 40), (257, 40), (4096, 600), (4097, 600), (262144, 3000), (262145, 3000), (700001, 300000),
                                          (32768, 255), (32768, 256), (32769, 256), (3000, 130815), (3000, 130816), (3000, 261631),
                                          (3000, 261632), (32767, 261631)])
def test_embed_gradient_at_the_sort_s_limits(tokens, vocab):
    """Unsorted, one launch (with 256 and 512 blocks), one step a block, several steps a block."""
    g = gen(tokens)
    ids = (torch.rand(tokens, generator=g) ** 3 * vocab).long()
    ids[torch.rand(tokens, generator=g) < 0.1] = -7
    dy = torch.randint(-8, 9, (tokens, 3), generator=g).float()
    live = ids >= 0
    want = torch.zeros(vocab, 3, dtype=torch.float64).index_add_(0, ids[live], dy[live].double())
    for it in (torch.int64, torch.int32):
        assert torch.equal(muon.embed_grad(dy.to(DEV), ids.to(it).to(DEV), vocab).cpu().double(), want)


def test_embed_gradient_random_and_repeatable():
    ids, dy = embed_ids("skewed", 5000, 400), randn(9, 5000, 264, dtype=torch.bfloat16)
    want = O.embed_grad(np64(dy), ids.numpy(), 400, 0.7)
    mag = O.embed_grad(np.abs(np64(dy)), ids.numpy(), 400, 0.7)
    got = muon.embed_grad(dy.to(DEV), ids.to(DEV), 400, scale=0.7)
    near(got, want, torch.float32, 5002 * U, mag)
    for _ in range(3):
        assert torch.equal(got, muon.embed_grad(dy.to(DEV), ids.to(DEV), 400, scale=0.7))


def test_embed_gradient_by_differences():
    table, dy = np.zeros((6, 3)), np64(randn(1, 5, 3))
    ids = np.array([4, 0, 4, -1, 5])
    got = np64(muon.embed_grad(torch.from_numpy(dy).float().to(DEV), torch.from_numpy(ids).to(DEV), 6, scale=1.5))
    dy = dy.astype(np.float32).astype(np.float64)
    for i in range(table.size):
        a = table.copy()
        a.flat[i] = 1.0                                    # linear: any step gives the derivative
        assert abs((O.embed(a, ids, 1.5) * dy).sum() - got.flat[i]) <= 8 * U * 16


# ------------------------------------------- streams, graphs, refusals, size ----
def everything(t):
    """One call of each operator on the tensors of `t`; all outputs."""
    h, y, n8, rstd = muon.rmsnorm_act8(t["x"], t["gain"], residual=t["r"])
    a, g8, u8 = muon.swiglu_act8(t["x"], t["r"])
    dg, du, a8 = muon.swiglu_act8_grad(t["dy"], g8, u8)
    dx, dgain = muon.rmsnorm_act8_grad(t["dy"], n8, rstd, t["gain"], dres=t["r"])
    dw = muon.act8_wgrad(t["dy"], a8, col_gain=t["gain"])
    e = muon.embed(t["table"], t["ids"])
    de = muon.embed_grad(dx, t["ids"], t["table"].shape[0])
    x8 = muon.act8_pack(t["x"])
    return [h, y, rstd, a, dg, du, dx, dgain, dw, e, de, muon.act8_unpack(n8), muon.act8_unpack(a8), muon.act8_unpack(x8)]


def inputs(seed, rows=1500, cols=328, vocab=90):
    return dict(x=randn(seed, rows, cols, dtype=torch.bfloat16).to(DEV), r=randn(seed + 1, rows, cols, dtype=torch.bfloat16).to(DEV),
                gain=(1 + 0.1 * randn(seed + 2, cols)).to(DEV), dy=randn(seed + 3, rows, cols, dtype=torch.bfloat16).to(DEV),
                table=randn(seed + 4, vocab, cols).to(DEV), ids=torch.randint(-1, vocab, (rows,), generator=gen(seed)).to(DEV))


def test_graph_replays_match_eager_calls():
    sets = [inputs(s) for s in (10, 20, 30)]
    want = [[o.clone() for o in everything(t)] for t in sets]
    static = {k: v.clone() for k, v in sets[0].items()}
    everything(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything(static)
    for t, w in list(zip(sets, want)) * 2:
        for k in static:
            static[k].copy_(t[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, w):
            assert torch.equal(a, b)
        eager = everything(t)                                # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, w))


def test_other_stream():
    t = inputs(40)
    want = everything(t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, y, n8, rstd = muon.rmsnorm_act8(t["x"], t["gain"], residual=t["r"], stream=s)
    dx, dgain = muon.rmsnorm_act8_grad(t["dy"], n8, rstd, t["gain"], dres=t["r"], stream=s)
    de = muon.embed_grad(dx, t["ids"], t["table"].shape[0], stream=s)
    with torch.cuda.stream(s):
        rest = everything(t)
    s.synchronize()
    for a, b in zip([y, dx, dgain, de], [want[1], want[6], want[7], want[10]]):
        assert torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(rest, want))


def test_inputs_freed_after_a_call_on_another_stream():
    """A tensor dropped right after a call on another stream is not reused before that stream has read it."""
    s = torch.cuda.Stream()
    x = randn(1, 2048, 4096)
    for _ in range(4):
        xg = x.to(DEV)
        s.wait_stream(torch.cuda.current_stream())
        x8 = muon.act8_pack(xg, stream=s)
        del xg
        torch.full((2048, 4096), float("nan"), device=DEV)   # would take the freed block
        s.synchronize()
        assert np.isfinite(values(x8)).all()


def test_debug_mode_gives_the_same(monkeypatch):
    t = inputs(50)
    want = everything(t)
    monkeypatch.setenv("MUON_DEBUG", "1")
    assert all(torch.equal(a, b) for a, b in zip(everything(t), want))


def test_refusals_name_the_argument():
    x, x16 = torch.zeros(4, 64, device=DEV), torch.zeros(4, 64, device=DEV, dtype=torch.bfloat16)
    x8 = muon.act8_pack(x)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    rstd, gain = torch.ones(4, device=DEV), torch.ones(64, device=DEV)
    for err, match, call in (
            (TypeError, "x must be float32 or bfloat16", lambda: muon.act8_pack(x.half())),
            (ValueError, "x must be 2-D", lambda: muon.act8_pack(x[0])),
            (ValueError, "x must have unit column stride", lambda: muon.act8_pack(x.t())),
            (ValueError, "rows that do not overlap", lambda: muon.act8_pack(x[:1].expand(4, 64))),
            (ValueError, "x must have a column", lambda: muon.act8_pack(x[:, :0])),
            (ValueError, "residual must have shape", lambda: muon.rmsnorm_act8(x, residual=x[:2])),
            (TypeError, "residual must have the type of x", lambda: muon.rmsnorm_act8(x, residual=x16)),
            (ValueError, "gain must be a contiguous vector of 64", lambda: muon.rmsnorm_act8(x, gain[:9])),
            (TypeError, "gain must be float32", lambda: muon.rmsnorm_act8(x, gain.double())),
            (ValueError, "residual must be a GPU tensor", lambda: muon.rmsnorm_act8(x, residual=x.cpu())),
            (TypeError, "codes of float8_e4m3fn", lambda: muon.act8_unpack(muon.Act8(x, x8.scales))),
            (TypeError, "scales of uint8", lambda: muon.act8_unpack(muon.Act8(x8.codes, x[:, :2].contiguous()))),
            (ValueError, "scales must have shape", lambda: muon.act8_unpack(muon.Act8(x8.codes, x8.scales[:, :1]))),
            (ValueError, "n8 must have shape", lambda: muon.rmsnorm_act8_grad(x[:3], x8, rstd[:3])),
            (ValueError, "rstd must be a contiguous vector of 4", lambda: muon.rmsnorm_act8_grad(x, x8, rstd[:2])),
            (TypeError, "up must have the type of gate", lambda: muon.swiglu_act8(x, x16)),
            (TypeError, "dup must have the type of da", lambda: muon.swiglu_act8_grad(x, x8, x8, dup=x16)),
            (TypeError, "dy must be bfloat16", lambda: muon.act8_wgrad(x, x8)),
            (ValueError, "x8 must have shape", lambda: muon.act8_wgrad(x16[:2], x8)),
            (ValueError, "out must be given", lambda: muon.act8_wgrad(x16, x8, accumulate=True)),
            (ValueError, "out must have shape", lambda: muon.act8_wgrad(x16, x8, out=x)),
            (TypeError, "ids must be int32 or int64", lambda: muon.embed(x, ids.float())),
            (ValueError, "ids must be a contiguous vector", lambda: muon.embed(x, ids[::2])),
            (ValueError, "one id per row", lambda: muon.embed_grad(x, ids[:3], 9)),
            (ValueError, "vocab must be at least 1", lambda: muon.embed_grad(x, ids, 0)),
            (ValueError, "out must be given", lambda: muon.embed_grad(x, ids, 9, accumulate=True))):
        with pytest.raises(err, match=match):
            call()
    wide = torch.zeros(2, 16400, device=DEV)
    with pytest.raises(muon.LibMuonError) as e:
        muon.rmsnorm_act8(wide)
    assert e.value.status == muon.MUON_EINVAL
    with pytest.raises(muon.LibMuonError) as e:                 # outputs over inputs
        muon.embed_grad(x, ids, 4, out=x)
    assert e.value.status == muon.MUON_EALIAS


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 bytes and 2^31 elements: their last rows."""
    rows, cols = 540_000, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-3:] = randn(1, 3, cols, dtype=torch.bfloat16).to(DEV)
    x8 = muon.act8_pack(x)
    tail = muon.Act8(x8.codes[-3:], x8.scales[-3:])
    check_pack_equal(tail, x[-3:])
    say("packed", rows, cols)
    assert torch.equal(muon.act8_unpack(x8)[-3:], muon.act8_unpack(tail))
    _, y, n8, rstd = muon.rmsnorm_act8(x)
    _, y3, n3, rstd3 = muon.rmsnorm_act8(x[-3:].contiguous())
    assert torch.equal(y[-3:], y3) and torch.equal(rstd[-3:], rstd3) and torch.equal(n8.scales[-3:], n3.scales)
    del y, n8
    say("normed")
    # the gradient's last tokens (x is zero before them), and a lookup at the table's end
    dy = x[:, :64]
    dw = muon.act8_wgrad(dy, x8)
    near(dw, np64(dy[-3:]).T @ values(tail), torch.float32, 16 * U, np.abs(np64(dy[-3:])).T @ np.abs(values(tail)))
    say("multiplied")
    ids = torch.tensor([rows - 1, 0, rows - 2], device=DEV)
    assert torch.equal(muon.embed(x, ids), x[ids])
    ids = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    ids[-2:] = 1
    assert np.allclose(np64(muon.embed_grad(x, ids, 3))[1], np64(x[-2:]).sum(0), atol=0, rtol=2 * U)

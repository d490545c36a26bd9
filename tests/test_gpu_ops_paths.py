"""The training operators on the GPU where tests/test_gpu_ops.py does not reach:
variants that only certain sizes select (tests/test_ops_launches.py names the
kernels that each size takes), rows that have to be left alone, extremes.
Tolerances as there; sums of integers have to be equal."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from oracle import ops_oracle as O
from tests.gpu_helpers import DEV
from tests.test_gpu_ops import GATE, TYPES, U, check_pack_near, embed_ids, gen, ids_of, int_case, near, np64, on_gpu, randn, values

pytestmark = pytest.mark.gpu


def bits(t):
    """The tensor's bits as integers (equal as values only where +0 is not -0)."""
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


# ------------------------------------------------- embedding, rows left alone ----
@pytest.mark.parametrize("dtype", TYPES, ids=ids_of)
@pytest.mark.parametrize("tokens,vocab,cols", [(3, 50, 40), (37, 300, 64), (37, 300, 1001), (256, 400, 520), (300, 900, 40), (300, 900, 1001)])
@pytest.mark.parametrize("kind", ["uniform", "none"])
def test_embed_gradient_leaves_rows_without_tokens(dtype, tokens, vocab, cols, kind):
    """Accumulating touches only the rows that have tokens: a table of -0, which adding zero would turn into +0, keeps its bits."""
    ids = embed_ids(kind, tokens, vocab)
    live = (ids >= 0) & (ids < vocab)
    used = torch.zeros(vocab, dtype=torch.bool)
    used[ids[live]] = True
    dy = torch.randint(1, 9, (tokens, cols), generator=gen(1)).to(dtype)
    want = torch.zeros(vocab, cols, dtype=torch.float64).index_add_(0, ids[live], dy[live].double())
    out = on_gpu(torch.full((vocab, cols), -0.0, dtype=dtype), "odd")
    before = bits(out.clone())
    muon.embed_grad(dy.to(DEV), ids.to(DEV), vocab, out=out, accumulate=True)
    after = bits(out.clone())
    assert torch.equal(after[~used.to(DEV)], before[~used.to(DEV)])
    assert torch.equal(out.cpu(), want.to(dtype))


# -------------------------------------------------- embedding, wide and short ----
# (tokens, vocab, cols): up to 256 tokens unsorted, rows of more than 512 columns a block's, in slices of 2048
WIDE = [(1, 3, 513), (37, 50, 513), (200, 9, 1001), (256, 13, 4099), (5, 3, 2049), (129, 40, 2048)]
# sorted: several slices of a row, several column blocks of a long run
WIDE_SORTED = [(700, 40, 2500), (3000, 100, 4099), (257, 700, 2056), (1300, 5, 9001)]


@pytest.mark.parametrize("kind", ["uniform", "one", "none", "skewed"])
@pytest.mark.parametrize("tokens,vocab,cols", WIDE + WIDE_SORTED)
def test_embed_gradient_of_wide_rows_is_exact_on_integers(kind, tokens, vocab, cols):
    ids = embed_ids(kind, tokens, vocab)
    dy = torch.randint(-8, 9, (tokens, cols), generator=gen(7)).float()
    live = (ids >= 0) & (ids < vocab)
    want = torch.zeros(vocab, cols, dtype=torch.float64).index_add_(0, ids[live], dy[live].double()) * 0.5
    base = torch.randint(-9, 9, (vocab, cols), generator=gen(8)).float()
    for src in TYPES:                              # every pair of types
        for dst in TYPES:
            got = muon.embed_grad(dy.to(src).to(DEV), ids.to(DEV), vocab, scale=0.5, dtype=dst)
            assert torch.equal(got.cpu(), want.float().to(dst)), (src, dst)
            out = on_gpu(base.to(dst), "odd")
            muon.embed_grad(on_gpu(dy.to(src), "odd"), ids.int().to(DEV), vocab, scale=0.5, out=out, accumulate=True)
            assert torch.equal(out.cpu(), (want + base.double()).float().to(dst)), (src, dst)


# ------------------------------------------------- weight gradient, every plan ----
# (tokens, n, k) by the tiles they take; some of the tiles whole and the last ones in token ranges, all whole, or all in ranges
WGRAD_PLANS = [(2049, 4352, 4100), (2049, 4353, 4101), (9000, 2100, 2100), (3100, 4096, 4608),         # 256 x 256
               (1000, 2048, 2304), (1001, 2047, 2301), (3000, 1104, 1296), (3001, 1101, 1303), (4000, 3000, 3000),  # 256 x 128
               (2383, 5955, 1406), (6000, 520, 264)]                                                # 128 x 128


@pytest.mark.parametrize("tokens,n,k", WGRAD_PLANS)
def test_wgrad_of_every_plan_is_exact_on_integers(tokens, n, k):
    dy, x = int_case(tokens, n, k)
    want = dy.to(DEV).double().t().contiguous() @ x.to(DEV).double()
    x8 = muon.act8_pack(x.to(DEV))
    dy = dy.to(DEV)
    assert torch.equal(muon.act8_wgrad(dy, x8).double(), want)
    assert torch.equal(muon.act8_wgrad(dy, x8, dtype=torch.bfloat16), want.float().bfloat16())
    gain = torch.exp2(torch.randint(-1, 2, (k,), generator=gen(5)).float()).to(DEV)
    base = torch.randint(-50, 50, (n, k), generator=gen(6)).float()
    for dtype in TYPES:                            # added to what is there, in a strided output
        out = on_gpu(base.to(dtype), "odd")
        muon.act8_wgrad(dy, x8, col_gain=gain, out=out, accumulate=True)
        assert torch.equal(out, (base.to(DEV).double() + want * gain).float().to(dtype))


@pytest.mark.parametrize("tokens,n,k", [(1, 80, 96), (33, 80, 96), (255, 264, 520), (4097, 24, 40), (2049, 4352, 4100), (3001, 1104, 1296)])
def test_wgrad_ends_with_the_last_token(tokens, n, k):
    """The loads reach past the last token; what lies there in the same buffers, NaN and the largest scale, must not count."""
    dy, x = int_case(tokens, n, k)
    want = dy.to(DEV).double().t().contiguous() @ x.to(DEV).double()
    x8 = muon.act8_pack(x.to(DEV))
    more = 256                                     # rows behind the last token, more than the loads run ahead
    dys = torch.full((tokens + more, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    codes = torch.full((tokens + more, -(-k // 32) * 32), 0x7F, dtype=torch.uint8, device=DEV)
    scales = torch.full((tokens + more, -(-k // 32)), 255, dtype=torch.uint8, device=DEV)
    dys[:tokens], codes[:tokens, :k], scales[:tokens] = dy.to(DEV), x8.codes.view(torch.uint8), x8.scales
    got = muon.act8_wgrad(dys[:tokens], muon.Act8(codes.view(torch.float8_e4m3fn)[:tokens, :k], scales[:tokens]))
    assert torch.equal(got.double(), want)


# ------------------------------------------------------------------ extremes ----
def near_relative(got, ref, rel):
    """fp32 results of normal size within rel of the 64-bit ones, without an absolute allowance."""
    assert np.abs(ref).min() > 2.0 ** -120
    near_ = np.abs(np64(got) - ref) <= (rel + U) * np.abs(ref)
    assert near_.all(), (np64(got)[~near_], ref[~near_])


def test_gate_of_very_negative_values():
    """1 + exp(-gate) above 2^126, where its reciprocal is subnormal, against factors that bring the results back:
    the results are normal numbers and have to be right relative to themselves."""
    g = torch.tensor([[-87.25, -87.375, -87.5, -87.75, -88.0, -88.25, -88.5, -88.625]])
    u = torch.full_like(g, 2.0 ** 100)
    a = muon.swiglu_act8(g.to(DEV), u.to(DEV), save=False)
    near_relative(a, O.swiglu(np64(g), np64(u)), GATE)
    # backward: -88 is the one value of these that 8 bits hold
    g = torch.full((1, 32), -88.0)
    u = torch.full_like(g, 2.0 ** 100)
    da = torch.full_like(g, 2.0 ** 10) * (1.0 + torch.arange(32) / 64)
    _, gate8, up8 = muon.swiglu_act8(g.to(DEV), u.to(DEV))
    assert np.array_equal(values(gate8), np64(g)) and np.array_equal(values(up8), np64(u))
    dgate, _, a8 = muon.swiglu_act8_grad(da.to(DEV), gate8, up8)
    dgo, _, ao = O.swiglu_grad(np64(da), np64(g), np64(u))
    near_relative(dgate, dgo, 2 * GATE)             # (two terms of opposite sign, the larger 88 times the smaller)
    check_pack_near(a8, ao, GATE)
    da = torch.full_like(g, 2.0 ** 100)
    _, dup, _ = muon.swiglu_act8_grad(da.to(DEV), gate8, up8)
    near_relative(dup, O.swiglu_grad(np64(da), np64(g), np64(u))[1], GATE)

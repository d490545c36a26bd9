"""The training operators on the GPU where tests/test_gpu_ops.py does not reach:
variants that only certain sizes select (tests/test_ops_launches.py names the
kernels that each size takes), rows that have to be left alone, extremes.
Tolerances as there; sums of integers have to be equal."""
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from tests.gpu_helpers import DEV
from tests.test_gpu_ops import TYPES, embed_ids, gen, ids_of, on_gpu

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

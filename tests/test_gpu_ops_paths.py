"""The training operators on the GPU where tests/test_gpu_ops.py does not reach.
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

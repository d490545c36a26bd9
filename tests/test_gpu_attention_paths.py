"""Attention's backward pass of rows that no wide load reaches, in the kernels of two launches, and outputs
in every layout.  Checks and tolerances are those of test_gpu_attention.py."""
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from tests.test_gpu_attention import BF, LAYOUTS, check, placed, starts_of, tensors
from tests.gpu_helpers import DEV
from tests.test_gpu_ops import gen

pytestmark = pytest.mark.gpu

# sequences' queries and keys, heads, key heads, columns: the steps cut into parts
PARTS = [([40], [4096], 4, 2, 64), ([3, 0, 70], [3000, 9, 2500], 2, 2, 80), ([2500], [2500], 1, 1, 64), ([2100, 30], [2100, 30], 4, 1, 128),
         ([3000], [50], 2, 1, 40), ([1500], [1400], 3, 3, 96)]


def many(count, seed):
    lengths = torch.randint(0, 9, (count,), generator=gen(seed)).tolist()
    lengths[count // 3] += 300
    lengths[-1] += 140
    return lengths


# more blocks than one launch takes, their steps whole
WHOLE = [(many(300, 1), many(300, 1), 4, 2, 64), (many(150, 2), many(150, 2), 4, 4, 80), (many(280, 3), many(280, 4), 4, 1, 128),
         ([1100], [1100], 32, 32, 64), ([700, 420], [700, 420], 32, 32, 96)]
sizes = lambda c: f"{len(c[0])}seq-{sum(c[0])}x{sum(c[1])}-{c[2]}over{c[3]}-{c[4]}"  # noqa: E731


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", PARTS + WHOLE, ids=sizes)
def test_unaligned_rows_in_two_launches(case, causal):
    nq, nk, heads, kv, dim = case
    check(*tensors(heads + dim, sum(nq), sum(nk), heads, kv, dim, "odd"), nq, nk, causal, layout="odd")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("nq,nk,heads,kv,dim", [([70, 1, 0, 130], [70, 1, 0, 130], 4, 2, 72), PARTS[3], PARTS[0]])
def test_outputs_in_every_layout(layout, nq, nk, heads, kv, dim):
    """The same bits as in new tensors, and nothing written beside them."""
    q, k, v = tensors(5, sum(nq), sum(nk), heads, kv, dim)
    st = dict(starts=starts_of(nq), k_starts=starts_of(nk))
    do = placed(torch.randn(q.shape, generator=gen(6)).to(BF), "plain")
    o, lse = muon.attention(q, k, v, **st)
    want = (o, *muon.attention_grad(do, q, k, v, o, lse, **st))
    views = [placed(torch.zeros(t.shape).to(BF), layout) for t in (q, q, k, v)]
    muon.attention(q, k, v, out=views[0], **st)
    muon.attention_grad(do, q, k, v, o, lse, dq=views[1], dk=views[2], dv=views[3], **st)
    for view, w in zip(views, want):
        assert torch.equal(view, w)
        around = torch.empty(0, device=DEV, dtype=BF).set_(view.untyped_storage())
        assert int(torch.isfinite(around).sum()) == view.numel()


@pytest.mark.parametrize("n,heads,kv", [(90, 4, 2), (2400, 4, 1), (1100, 32, 32)])
def test_lse_with_rows_of_a_wider_buffer(n, heads, kv):
    """One launch, two with parts, two without: the same bits, whatever lies behind a row."""
    q, k, v = tensors(2, n, n, heads, kv, 64)
    o, lse = muon.attention(q, k, v)
    do = placed(torch.randn(q.shape, generator=gen(1)).to(BF), "plain")
    wide = torch.full((heads, n + 13), float("nan"), device=DEV)
    wide[:, 5:5 + n] = lse
    for a, b in zip(muon.attention_grad(do, q, k, v, o, lse), muon.attention_grad(do, q, k, v, o, wide[:, 5:5 + n])):
        assert torch.equal(a, b) and torch.isfinite(a).all()

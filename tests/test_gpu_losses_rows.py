"""The losses' kernels of many rows, and of long rows that no second block shares: the checks of
test_gpu_losses.py, with their tolerances, on batches that repeat a few rows.  Every copy of a row has to
give the same bits, and the first ones are compared with the oracle."""
import pytest
import torch

import matrix_aware_optimizer_libmuon_amd as muon
from tests import test_gpu_losses as T
from tests.gpu_helpers import DEV
from tests.test_gpu_ops import TYPES, gen, ids_of, on_gpu

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
# both sides of each border of the kernels of more than 512 rows
MANY = [513, 2048, 2049, 5000, 8192, 8193, 16384, 16385, 32000, 32768, 32769, 50001, 65536]
# more rows than blocks are shared among, 1024 threads to a row: kept in registers, and read twice
LONG = [(132, 65536, F32), (132, 50001, BF), (132, 131072, BF), (132, 131073, BF), (132, 65537, F32), (132, 200003, BF), (516, 70001, F32),
        (516, 131072, BF)]
CASES = [(516, cols, dtype) for cols in MANY for dtype in (F32, BF)] + LONG
names = lambda c: f"{c[0]}x{c[1]}-{ids_of(c[2])}"  # noqa: E731


class Repeated:
    """The losses on the given rows over and over, `rows` in all; what they return for the first of them."""

    def __init__(self, rows, layout):
        self.rows, self.layout = rows, layout

    def _call(self, loss, tensors, options):
        n = len(tensors[0])
        at = torch.arange(self.rows, device=DEV) % n
        full = lambda t: on_gpu(t[at], self.layout if t.dim() == 2 else "plain") if isinstance(t, torch.Tensor) else t  # noqa: E731
        outs = loss(*(full(t) for t in tensors), **{k: full(v) for k, v in options.items()})
        for o in outs:
            assert o is None or torch.equal(o, o[:n][at])
        return tuple(None if o is None else o[:n] for o in outs)

    def distill_loss(self, *tensors, **options):
        return self._call(muon.distill_loss, tensors, options)

    def policy_loss(self, *tensors, **options):
        return self._call(muon.policy_loss, tensors, options)


@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("case", CASES, ids=names)
def test_distillation_of_many_rows(case, layout, monkeypatch):
    rows, cols, dtype = case
    monkeypatch.setattr(T, "muon", Repeated(rows, layout))
    logits = (3 * torch.randn(3, cols, generator=gen(cols))).to(dtype)
    T.check_distill(logits, T.entries(cols, 3, cols, 20, torch.int64), 2 * torch.randn(3, 20, generator=gen(cols + 1)), 1.5,
                    torch.tensor([1.0, 0.25, 0.0]))


@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("case", CASES, ids=names)
def test_policy_of_many_rows(case, layout, monkeypatch):
    rows, cols, dtype = case
    monkeypatch.setattr(T, "muon", Repeated(rows, layout))
    logits, actions, old, adv, ref = T.policy_inputs(cols, 4, cols, dtype)
    T.check_policy(logits, actions, old, adv, ref, kl=0.1, weights=torch.tensor([1.0, 0.5, 0.0, -2.0]))

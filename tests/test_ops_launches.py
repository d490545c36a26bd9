"""Which launches the training operators' entries make (CPU; launches.py)."""
import pytest

from tests.launches import record

MAX = (1 << 31) - 1                               # rows and tokens


@pytest.mark.parametrize("entry,args", [
    ("act8_pack", dict(rows=MAX, cols=40)), ("act8_unpack", dict(rows=MAX, cols=40)),
    ("rmsnorm", dict(rows=MAX, cols=40)), ("rmsnorm", dict(rows=1 << 24, cols=16384, dtype="bf16")),
    ("rmsnorm_grad", dict(rows=MAX, cols=40)), ("rmsnorm_grad", dict(rows=1 << 24, cols=16384)),
    ("swiglu", dict(rows=MAX, cols=33)), ("swiglu_grad", dict(rows=MAX, cols=33)),
    ("wgrad", dict(tokens=MAX, n=24, k=32)), ("wgrad", dict(tokens=MAX, n=23, k=33)), ("wgrad", dict(tokens=40, n=1 << 20, k=1 << 16)),
    ("embed", dict(tokens=MAX, vocab=100, cols=40)), ("embed", dict(tokens=100, vocab=MAX - 1, cols=40)),
    ("embed_grad", dict(tokens=(1 << 29) - 64, vocab=1000, cols=40)), ("embed_grad", dict(tokens=(1 << 29) - 63, vocab=1000, cols=40)),
    ("embed_grad", dict(tokens=MAX, vocab=1000, cols=16)), ("embed_grad", dict(tokens=MAX, vocab=MAX - 1, cols=520)),
    ("embed_grad", dict(tokens=100, vocab=MAX - 1, cols=40)), ("embed_grad", dict(tokens=1000, vocab=MAX - 1, cols=520)),
], ids=lambda v: v if isinstance(v, str) else "x".join(str(x) for x in v.values()))
def test_the_largest_sizes_can_be_launched(entry, args):
    """Fewer than 2^32 threads along every axis of every launch, up to the documented sizes."""
    (status, launches), = record([(entry, args)])
    assert launches
    for kernel, grid, block in launches:
        for g, b in zip(grid, block):
            assert 0 < g * b < 1 << 32, (kernel, grid, block)
    assert status == 0


def test_embedding_gradient_kernels_of_the_tested_sizes():
    from tests.test_gpu_ops_paths import WIDE, WIDE_SORTED
    got = record([("embed_grad", dict(tokens=t, vocab=v, cols=c)) for t, v, c in WIDE + WIDE_SORTED])
    for (tokens, vocab, cols), (status, launches) in zip(WIDE + WIDE_SORTED, got):
        assert status == 0
        if (tokens, vocab, cols) in WIDE:
            assert [kernel for kernel, _, _ in launches] == ["k_direct<float, float, 256>"]
        else:
            assert [kernel for kernel, _, _ in launches] == ["k_embed_buckets<4>", "k_sums<float, float, 256>", "k_join<float, 4>"]
            assert launches[2][1][1] == -(-cols // 512) > 4

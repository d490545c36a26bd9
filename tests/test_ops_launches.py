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


def wgrad_plan(tokens, n, k, launches):
    """(tile, whole: all, some or none of the tiles are made from all tokens, token ranges of the others, copies first)"""
    by_name = {kernel.split("<")[0]: (kernel, grid[0]) for kernel, grid, _ in launches}
    kernel, blocks = by_name["k_wgrad"]
    tn, tk = (int(v) for v in kernel[len("k_wgrad<"):-1].split(","))
    tiles = -(-n // tn) * -(-k // tk)
    rest = by_name["k_wgrad_join"][1] // (tn * tk // 1024) if "k_wgrad_join" in by_name else 0
    whole = tiles - rest
    ranges = (blocks - whole) // rest if rest else 1
    assert whole + rest * ranges == blocks
    return (tn, tk), "all" if rest == 0 else "some" if whole else "none", ranges, "k_wgrad_copy" in by_name


def test_weight_gradient_plans_of_the_tested_sizes():
    """The sizes that the GPU tests are exact on cover every tile with every way of dealing it; a changed estimate shows here."""
    from tests.test_gpu_ops_paths import WGRAD_PLANS
    got = record([("wgrad", dict(tokens=t, n=n, k=k)) for t, n, k in WGRAD_PLANS])
    plans = {size: wgrad_plan(*size, launches) for size, (status, launches) in zip(WGRAD_PLANS, got) if status == 0}
    assert plans == {
        (2049, 4352, 4100): ((256, 256), "some", 3, False), (2049, 4353, 4101): ((256, 256), "some", 3, True),
        (9000, 2100, 2100): ((256, 256), "none", 3, True), (3100, 4096, 4608): ((256, 256), "some", 4, False),
        (1000, 2048, 2304): ((256, 128), "all", 1, False), (1001, 2047, 2301): ((256, 128), "all", 1, True),
        (3000, 1104, 1296): ((256, 128), "none", 4, False), (3001, 1101, 1303): ((256, 128), "none", 4, True),
        (4000, 3000, 3000): ((256, 128), "some", 5, False), (2383, 5955, 1406): ((128, 128), "some", 15, True),
        (6000, 520, 264): ((128, 128), "none", 16, False)}

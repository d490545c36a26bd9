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


@pytest.mark.parametrize("entry", ["attention", "attention_grad"])
@pytest.mark.parametrize("args", [
    dict(tokens=(1 << 29) - 128 * 3, k_tokens=(1 << 29) - 128 * 3, heads_=1, kv=1, dim=64, sequences=0),
    dict(tokens=1, k_tokens=1, heads_=4, kv=4, dim=128, sequences=(1 << 20) - 2),
    dict(tokens=1 << 19, k_tokens=(1 << 19) - 5, heads_=512, kv=512, dim=104, sequences=1000),
], ids=lambda v: "x".join(str(x) for x in v.values()))
def test_the_largest_attention_can_be_launched(entry, args):
    (status, launches), = record([(entry, args)])
    assert status == 0 and len(launches) == (1 if entry == "attention" else 2)
    for kernel, grid, block in launches:
        assert 0 < grid[0] * block[0] < 1 << 32 and grid[1:] == (1, 1), (kernel, grid, block)


@pytest.mark.parametrize("entry", ["distill", "policy"])
@pytest.mark.parametrize("args", [dict(tokens=MAX, vocab=40), dict(tokens=MAX, vocab=40, dtype="bf16"), dict(tokens=1 << 20, vocab=1 << 20)],
                         ids=lambda v: "x".join(str(x) for x in v.values()))
def test_the_largest_losses_can_be_launched(entry, args):
    (status, launches), = record([(entry, args)])
    assert status == 0 and len(launches) == 1
    assert all(0 < g * b < 1 << 32 for g, b in zip(*launches[0][1:]))


def test_attention_kernels_by_columns_and_alignment():
    few, many = (dict(tokens=n, k_tokens=n, heads_=h, kv=h // 2, sequences=0) for n, h in ((300, 2), (20000, 32)))
    for dim, blocks in ((8, 2), (64, 2), (72, 3), (96, 3), (104, 4), (128, 4)):
        for odd in (False, True):
            al = "false" if odd else "true"
            got = record([(e, dict(args, dim=dim, odd=odd)) for args in (few, many) for e in ("attention", "attention_grad")])
            names = [[kernel for kernel, _, _ in launches] for _, launches in got]
            assert names == [[f"k_attn<{blocks}, {al}, true>"], [f"k_attn_grad<{blocks}, {al}>"],
                             [f"k_attn<{blocks}, {al}, true>"], [f"k_attn_dq<{blocks}, {al}>", f"k_attn_dkv<{blocks}, {al}>"]]


@pytest.mark.parametrize("heads_,kv,tokens,k_tokens,dim,one", [
    (4, 4, 74, 74, 64, True), (32, 32, 1024, 1024, 64, True), (32, 32, 1025, 1024, 64, False), (32, 32, 1024, 1025, 64, False),
    (32, 32, 1024, 1400, 128, True), (4, 4, 0, 74, 64, True), (4, 4, 74, 0, 64, True)])
def test_few_blocks_of_the_attention_gradient_take_one_launch(heads_, kv, tokens, k_tokens, dim, one):
    """Up to 512 blocks of 128 queries and 128 (past 96 columns 256) keys together."""
    (status, launches), = record([("attention_grad", dict(tokens=tokens, k_tokens=k_tokens, heads_=heads_, kv=kv, dim=dim, sequences=0))])
    assert status == 0 and [k.split("<")[0] for k, _, _ in launches] == (["k_attn_grad"] if one else ["k_attn_dq", "k_attn_dkv"])


@pytest.mark.parametrize("layout", ["side by side", "in steps", "one after the other"])
def test_attention_takes_slices_of_one_buffer(layout):
    """Heads of q, k, v, o and their gradients side by side in one buffer overlap nothing."""
    args = dict(tokens=40, k_tokens=40, heads_=4, kv=4, dim=64, sequences=0, layout=layout)
    for status, launches in record([("attention", args), ("attention_grad", args)]):
        assert status == 0 and launches


@pytest.mark.parametrize("tokens,k_tokens,heads_,kv,dim,sequences,parts", [
    (40, 4096, 4, 2, 64, 0, (8, 8, 1)), (1, 5000, 2, 1, 128, 0, (9, 9, 1)), (73, 5509, 2, 2, 80, 3, (3, 3, 1)),
    (2500, 2500, 1, 1, 64, 0, (4, 4, 4)), (2130, 2130, 4, 1, 128, 2, (2, 2, 8)), (3000, 50, 2, 1, 40, 0, (1, 1, 11)),
    (1500, 1400, 3, 3, 96, 0, (2, 2, 2)), (64, 1 << 16, 1, 1, 64, 0, (64, 16, 1)), (16384, 16384, 32, 8, 128, 4, (1, 1, 1)),
    (74, 74, 4, 4, 64, 2, (1, 1))])
def test_parts_of_attention(tokens, k_tokens, heads_, kv, dim, sequences, parts):
    """How many parts the steps of the tested sizes are cut into: forward, dq, dk and dv; each cut has its join."""
    args = dict(tokens=tokens, k_tokens=k_tokens, heads_=heads_, kv=kv, dim=dim, sequences=sequences, causal=0)
    launches = [l for _, ls in record([(e, args) for e in ("attention", "attention_grad")]) for l in ls]
    got, joins = [], 0
    for kernel, grid, _ in launches:
        if kernel == "k_attn_join":
            joins += 1
        else:
            got.append(grid[1])
    assert tuple(got) == parts and joins == sum(p > 1 for p in parts)


@pytest.mark.parametrize("tokens,k_tokens,heads_,kv,sequences,packed,grid", [
    (32, 32 * 4096, 32, 8, 32, True, (34 * 8, 2, 1)), (1, 65536, 32, 8, 0, True, (8, 64, 1)), (1, 65536, 8, 8, 0, False, (8, 64, 1)),
    (64, 64, 6, 2, 0, True, (4, 1, 1)), (65, 65, 6, 6, 0, False, (6, 1, 1)), (640, 9000, 10, 2, 10, True, (36 * 2, 1, 1)),
    (641, 9000, 10, 10, 10, False, (17 * 10, 1, 1)), (3, 3000, 4, 1, 2, True, (4, 2, 1))])
def test_heads_that_share_keys_go_together(tokens, k_tokens, heads_, kv, sequences, packed, grid):
    """Forward pass: a block has the rows of all heads of a key head."""
    (status, launches), = record([("attention", dict(tokens=tokens, k_tokens=k_tokens, heads_=heads_, kv=kv, dim=64, sequences=sequences))])
    assert status == 0 and launches[0][0] == f"k_attn<2, true, {'true' if packed else 'false'}>" and launches[0][1] == grid


@pytest.mark.parametrize("entry", ["distill", "policy"])
@pytest.mark.parametrize("tokens,vocab,dtype,share", [
    (1, 32000, "bf16", 1), (1, 32769, "bf16", 8), (1, 131072, "bf16", 16), (1, 200000, "bf16", 8), (1, 65536, "f32", 8), (1, 65537, "f32", 8),
    (16, 131072, "bf16", 16), (17, 131072, "bf16", 8), (128, 131072, "bf16", 2), (129, 131072, "bf16", 1), (128, 65536, "bf16", 2),
    (1, 16384, "bf16", 1)])
def test_blocks_that_share_a_long_row_of_few(entry, tokens, vocab, dtype, share):
    """A power of two of them, no more than the row has vectors a thread, and rows times blocks up to 256."""
    (status, ((kernel, grid, _),)), = record([(entry, dict(tokens=tokens, vocab=vocab, dtype=dtype))])
    assert status == 0 and kernel.endswith(f", {'true' if share > 1 else 'false'}>")
    assert grid == (tokens, share, 1)


def loss_shape(rows, cols, f32):
    """(threads, vectors of 8 columns a thread) of a row; 0 vectors: read twice."""
    if cols <= 512:
        return 64, 1
    if rows <= 512:
        few = [(2048, 256, 1), (8192, 1024, 1), (16384, 1024, 2), (32768, 1024, 4), (65536, 1024, 8)]
        for most, threads, vectors in few:
            if cols <= most:
                return threads, vectors
    many = [(2048, 64, 4), (8192, 256, 4), (16384, 512, 4), (32768, 512, 8)]
    many += [(65536, 1024, 8)] if f32 else [(65536, 512, 16), (131072, 1024, 16)]
    for most, threads, vectors in many:
        if cols <= most:
            return threads, vectors
    return 1024, 0


@pytest.mark.parametrize("entry", ["distill", "policy"])
def test_loss_kernels_of_the_tested_sizes(entry):
    """Every kernel that a size can take is one that tests/test_gpu_losses.py or test_gpu_losses_rows.py compares with the oracle."""
    from tests.test_gpu_losses import COLS
    from tests.test_gpu_losses_rows import CASES
    sizes = [(3, cols, t) for cols in COLS for t in ("f32", "bf16")]
    sizes += [(rows, cols, "f32" if str(t) == "torch.float32" else "bf16") for rows, cols, t in CASES]
    tested = set()
    for (rows, cols, t), (status, ((kernel, _, block),)) in zip(sizes, record([(entry, dict(tokens=r, vocab=c, dtype=t)) for r, c, t in sizes])):
        threads, vectors = loss_shape(rows, cols, t == "f32")
        name = f"k_{entry}<{'float' if t == 'f32' else 'unsigned short'}, {threads}, {vectors}, "
        assert status == 0 and kernel.startswith(name) and block == (threads, 1, 1), (rows, cols, t, kernel)
        tested.add(kernel)
    reached = set()
    grid = [(rows, cols, t) for rows in (1, 16, 100, 128, 129, 512, 513, 1 << 20) for t in ("f32", "bf16")
            for cols in (1, 512, 513, 2048, 2049, 8192, 8193, 16384, 16385, 32768, 32769, 65536, 65537, 131072, 131073, 1 << 20)]
    for _, ((kernel, _, _),) in record([(entry, dict(tokens=r, vocab=c, dtype=t)) for r, c, t in grid]):
        reached.add(kernel)
    assert reached == tested


def test_unaligned_backward_passes_of_the_tested_sizes():
    """tests/test_gpu_attention_paths.py: two launches without wide loads, cut into parts and whole."""
    from tests.test_gpu_attention_paths import PARTS, WHOLE
    for cases, cut in ((PARTS, True), (WHOLE, False)):
        for nq, nk, heads_, kv, dim in cases:
            (status, launches), = record([("attention_grad", dict(tokens=sum(nq), k_tokens=sum(nk), heads_=heads_, kv=kv, dim=dim,
                                                                  sequences=len(nq), odd=True, causal=0))])
            blocks = 2 if dim <= 64 else 3 if dim <= 96 else 4
            names = [k for k, _, _ in launches if k != "k_attn_join"]
            assert status == 0 and names == [f"k_attn_dq<{blocks}, false>", f"k_attn_dkv<{blocks}, false>"], (nq[:3], dim, launches)
            assert any(grid[1] > 1 for k, grid, _ in launches if k != "k_attn_join") == cut, (nq[:3], dim, launches)

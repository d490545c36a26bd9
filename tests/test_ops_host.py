"""Host-side checks of the training operators' C entries and of their binding
that need no GPU: bad arguments are refused before anything is launched."""
import ctypes
import os
import random

import pytest

import matrix_aware_optimizer_libmuon_amd as muon
from matrix_aware_optimizer_libmuon_amd import _lib as L

torch = pytest.importorskip("torch")
EINVAL, EALIAS, EWORKSPACE = muon.MUON_EINVAL, muon.MUON_EALIAS, muon.MUON_EWORKSPACE
BF16, F32 = muon.MUON_BF16, muon.MUON_F32
WS = ctypes.c_void_p(1 << 42)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from matrix_aware_optimizer_libmuon_amd import build
        build.build()
    return L.load()


_next = [1 << 36]


def ptr():
    """A fresh address, far from every other (never read: the calls below fail on the host)."""
    _next[0] += 1 << 28
    return _next[0]


def act8(cols=64, **kw):
    a = L.MuonAct8(ptr(), ptr(), cols, (cols + 31) // 32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def with_(s, **kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def norm(**kw):
    return with_(L.MuonRmsnorm(x=ptr(), residual=ptr(), gain=ptr(), h=ptr(), y=ptr(), n=act8(), rstd=ptr(), rows=8, cols=64,
                               ld_x=64, ld_residual=64, ld_h=64, ld_y=64, eps=1e-6, dtype=BF16), **kw)


def norm_grad(**kw):
    return with_(L.MuonRmsnormGrad(dy=ptr(), dres=ptr(), gain=ptr(), rstd=ptr(), n=act8(), dx=ptr(), dgain=ptr(), rows=4000,
                                   cols=64, ld_dy=64, ld_dres=64, ld_dx=64, dtype=BF16), **kw)


def gate(**kw):
    return with_(L.MuonSwiglu(gate=ptr(), up=ptr(), a=ptr(), gate8=act8(), up8=act8(), rows=8, cols=64, ld_gate=64, ld_up=64,
                              ld_a=64, dtype=BF16), **kw)


def gate_grad(**kw):
    return with_(L.MuonSwigluGrad(da=ptr(), gate8=act8(), up8=act8(), dgate=ptr(), dup=ptr(), a8=act8(), rows=8, cols=64,
                                  ld_da=64, ld_dgate=64, ld_dup=64, dtype=BF16), **kw)


def wgrad(**kw):
    return with_(L.MuonAct8Wgrad(dy=ptr(), x8=act8(), col_gain=ptr(), dw=ptr(), tokens=5000, n=64, k=64, ld_dy=64, ld_dw=64,
                                 dw_dtype=F32, accumulate=0), **kw)


def embed(**kw):
    return with_(L.MuonEmbed(table=ptr(), ids=ptr(), out=ptr(), tokens=9, vocab=100, cols=64, ld_table=64, ld_out=64, scale=1.0,
                             table_dtype=F32, out_dtype=BF16, id_bytes=8), **kw)


def embed_grad(**kw):
    return with_(L.MuonEmbedGrad(dy=ptr(), ids=ptr(), dtable=ptr(), tokens=900, vocab=100, cols=64, ld_dy=64, ld_dtable=64,
                                 scale=1.0, dy_dtype=BF16, table_dtype=F32, id_bytes=8), **kw)


def test_struct_layouts_match_header(lib):
    sizes = muon._marshaller().OP_BYTES
    for name, cls in (("muon_act8_t", L.MuonAct8), ("muon_rmsnorm_t", L.MuonRmsnorm),
                      ("muon_rmsnorm_grad_t", L.MuonRmsnormGrad), ("muon_swiglu_t", L.MuonSwiglu),
                      ("muon_swiglu_grad_t", L.MuonSwigluGrad), ("muon_act8_wgrad_t", L.MuonAct8Wgrad),
                      ("muon_embed_t", L.MuonEmbed), ("muon_embed_grad_t", L.MuonEmbedGrad)):
        assert sizes[name] == ctypes.sizeof(cls), name


def test_pack_and_unpack_refuse(lib):
    def pack(x=ptr(), ld=64, dtype=BF16, rows=8, cols=64, out=act8()):
        return lib.muon_act8_pack(x, ld, dtype, rows, cols, ctypes.byref(out) if out else None, None)

    def unpack(src=act8(), rows=8, cols=64, out=ptr(), ld=64, dtype=BF16):
        return lib.muon_act8_unpack(ctypes.byref(src) if src else None, rows, cols, out, ld, dtype, None)

    for bad in (dict(x=0), dict(x=ptr() + 1), dict(ld=63), dict(dtype=7), dict(rows=-1), dict(rows=1 << 31), dict(cols=0),
                dict(cols=(1 << 20) + 1), dict(out=None), dict(out=act8(codes=0)), dict(out=act8(scales=0)),
                dict(out=act8(ld_codes=63)), dict(out=act8(ld_scales=1)), dict(ld=1 << 60)):
        assert pack(**bad) == EINVAL, bad
    for bad in (dict(src=None), dict(src=act8(ld_codes=5)), dict(out=0), dict(ld=7), dict(dtype=-1), dict(cols=-3)):
        assert unpack(**bad) == EINVAL, bad
    p = ptr()
    assert pack(x=p, out=act8(codes=p + 64)) == EALIAS
    assert pack(out=act8(codes=p, scales=p + 3)) == EALIAS
    assert unpack(src=act8(codes=p), out=p + 512 - 64) == EALIAS
    # no rows: nothing is read, nothing launched
    assert pack(x=0, rows=0, out=act8(codes=0, scales=0)) == 0 and unpack(rows=0, out=0) == 0


def test_norm_refuses(lib):
    def call(**kw):
        return lib.muon_rmsnorm_act8(ctypes.byref(norm(**kw)), None)

    assert lib.muon_rmsnorm_act8(None, None) == EINVAL
    for bad in (dict(x=0), dict(dtype=3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(cols=16385),
                dict(cols=0), dict(ld_x=63), dict(ld_residual=0), dict(ld_h=1), dict(ld_y=1), dict(gain=ptr() + 2),
                dict(rstd=ptr() + 1), dict(n=act8(scales=0)), dict(n=act8(ld_codes=3)), dict(rows=-1), dict(y=ptr() + 1)):
        assert call(**bad) == EINVAL, bad
    p = ptr()
    assert call(x=p, y=p) == EALIAS and call(h=p, y=p + 2) == EALIAS and call(gain=p, rstd=p + 64) == EALIAS
    assert call(rows=0, x=0) == 0


def test_norm_gradient_refuses(lib):
    need = lib.muon_rmsnorm_act8_grad_workspace_bytes(4000, 64)
    assert need > 0 and lib.muon_rmsnorm_act8_grad_workspace_bytes(1, 64) == 0
    assert lib.muon_rmsnorm_act8_grad_workspace_bytes(10, 1 << 15) == 0 and lib.muon_rmsnorm_act8_grad_workspace_bytes(-1, 8) == 0

    def call(ws=WS, ws_bytes=need, **kw):
        return lib.muon_rmsnorm_act8_grad(ctypes.byref(norm_grad(**kw)), ws, ws_bytes, None)

    for bad in (dict(dy=0), dict(n=act8(codes=0)), dict(rstd=0), dict(dx=0), dict(reserved=1), dict(dtype=2), dict(ld_dx=9),
                dict(cols=1 << 15), dict(ld_dres=3)):
        assert call(**bad) == EINVAL, bad
    assert call(ws=None) == EWORKSPACE and call(ws_bytes=need - 1) == EWORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 42) + 8)) == EWORKSPACE
    p = ptr()
    assert call(dy=p, dx=p) == EALIAS and call(dgain=1 << 42) == EALIAS


def test_gate_refuses_and_takes_halves_of_one_buffer(lib):
    def fwd(**kw):
        return lib.muon_swiglu_act8(ctypes.byref(gate(**kw)), None)

    def bwd(**kw):
        return lib.muon_swiglu_act8_grad(ctypes.byref(gate_grad(**kw)), None)

    for bad in (dict(gate=0), dict(up=0), dict(gate8=act8(codes=0)), dict(reserved=1), dict(dtype=9), dict(ld_a=1)):
        assert fwd(**bad) == EINVAL, bad
    for bad in (dict(da=0), dict(dup=0), dict(dgate=0), dict(gate8=act8(codes=0)), dict(up8=act8(scales=0)), dict(reserved=2)):
        assert bwd(**bad) == EINVAL, bad
    p = ptr()
    # column slices that touch overlap nothing; shifted by one element they do
    assert bwd(dgate=p, dup=p + 126, ld_dgate=128, ld_dup=128) == EALIAS
    assert bwd(dgate=p + 126, dup=p, ld_dgate=128, ld_dup=128) == EALIAS
    assert bwd(dgate=p, dup=p + 130, ld_dgate=128, ld_dup=128) == EALIAS      # runs into the next row
    assert bwd(rows=1, dgate=p, dup=p + 100) == EALIAS
    assert fwd(rows=0) == 0 and bwd(rows=0) == 0


def test_wgrad_refuses(lib):
    def call(ws=WS, ws_bytes=1 << 40, **kw):
        return lib.muon_act8_wgrad(ctypes.byref(wgrad(**kw)), ws, ws_bytes, None)

    for bad in (dict(dy=0), dict(dw=0), dict(x8=act8(codes=0)), dict(n=0), dict(k=0), dict(tokens=-1), dict(n=(1 << 20) + 1),
                dict(dw_dtype=4), dict(accumulate=2), dict(ld_dy=63), dict(ld_dw=63), dict(dy=ptr() + 1), dict(dw=ptr() + 2)):
        assert call(**bad) == EINVAL, bad
    op = wgrad()
    need = lib.muon_act8_wgrad_workspace_bytes(ctypes.byref(op))
    assert need > 0 and lib.muon_act8_wgrad_workspace_bytes(ctypes.byref(wgrad(n=0))) == 0
    assert lib.muon_act8_wgrad_workspace_bytes(ctypes.byref(wgrad(ld_dy=0))) == 0
    # a single row's strides are not read
    one = [lib.muon_act8_wgrad_workspace_bytes(ctypes.byref(wgrad(tokens=1, ld_dy=ld, x8=act8(ld_codes=ld, ld_scales=ld))))
           for ld in (64, 0, -64, 1 << 50)]
    assert len(set(one)) == 1
    assert call(ws_bytes=need - 1) == EWORKSPACE and call(ws=None) == EWORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 42) + 4)) == EWORKSPACE
    p = ptr()
    assert call(dy=p, dw=p) == EALIAS and call(dw=1 << 42) == EALIAS and call(dw=p, col_gain=p) == EALIAS
    assert call(tokens=0, accumulate=1) == 0                          # nothing to add


def test_embed_refuses(lib):
    def fwd(**kw):
        return lib.muon_embed(ctypes.byref(embed(**kw)), None)

    def bwd(ws=WS, ws_bytes=1 << 40, **kw):
        return lib.muon_embed_grad(ctypes.byref(embed_grad(**kw)), ws, ws_bytes, None)

    for bad in (dict(table=0), dict(ids=0), dict(out=0), dict(vocab=0), dict(vocab=(1 << 31) - 1), dict(tokens=-1), dict(cols=0),
                dict(scale=float("nan")), dict(id_bytes=2), dict(out_dtype=5), dict(table_dtype=-1), dict(ids=ptr() + 4)):
        assert fwd(**bad) == EINVAL, bad
    for bad in (dict(dy=0), dict(ids=0), dict(dtable=0), dict(vocab=0), dict(reserved=1), dict(accumulate=-1), dict(id_bytes=1),
                dict(scale=float("inf")), dict(ld_dtable=63)):
        assert bwd(**bad) == EINVAL, bad
    need = lib.muon_embed_grad_workspace_bytes(900, 100, 64)
    assert need > 0 and lib.muon_embed_grad_workspace_bytes(900, 0, 64) == 0
    assert bwd(ws_bytes=need - 1) == EWORKSPACE and bwd(ws=None) == EWORKSPACE
    p = ptr()
    assert fwd(table=p, out=p) == EALIAS and bwd(dy=p, dtable=p) == EALIAS and bwd(dtable=1 << 42) == EALIAS
    assert fwd(tokens=0, ids=0, out=0) == 0 and bwd(tokens=0, accumulate=1) == 0


def test_workspaces_grow_with_the_work(lib):
    rng = random.Random(5)
    for _ in range(200):
        t, v, c = rng.randint(0, 1 << 20), rng.randint(1, 1 << 20), rng.randint(1, 1 << 14)
        a = lib.muon_embed_grad_workspace_bytes(t, v, c)
        assert a >= 16 * t                                            # keys and tokens, twice
        assert lib.muon_rmsnorm_act8_grad_workspace_bytes(t, c) % (4 * c) == 0


def test_binding_refuses_cpu_tensors(lib):
    x, v = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    x8 = muon.Act8(x.to(torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8))
    for call in (lambda: muon.act8_pack(x), lambda: muon.act8_unpack(x8), lambda: muon.rmsnorm_act8(x),
                 lambda: muon.rmsnorm_act8_grad(x, x8, x[:, 0]), lambda: muon.swiglu_act8(x, x),
                 lambda: muon.swiglu_act8_grad(x, x8, x8), lambda: muon.act8_wgrad(x.bfloat16(), x8),
                 lambda: muon.embed(x, v), lambda: muon.embed_grad(x, v, 9)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(AttributeError):
        muon.no_such_operator


@pytest.mark.parametrize("tokens,vocab,passes,log_buckets", [
    (256, 1000, 0, 0), (257, 1000, 1, 8), (32768, 130815, 1, 8), (32768, 130816, 1, 9), (32768, 261631, 1, 9),
    (32768, 261632, 2, 0), (32769, 511, 1, 0), (32769, 512, 2, 0), (32769, 262143, 2, 0), (32769, 262144, 3, 0), (700001, 300000, 3, 0)])
@pytest.mark.parametrize("cols", [1, 40, 4099])
def test_embedding_gradient_workspace_is_the_sum_of_its_parts(lib, tokens, vocab, passes, log_buckets, cols):
    """Keys and tokens, once per pass but at most twice; the digits' counts of a sort by digits; the rows' first places;
    two sums per 32 tokens.  Each part 256-byte aligned."""
    up = lambda n: -(-4 * n // 256) * 256  # noqa: E731
    want = 0
    if passes:
        want = min(passes, 2) * 2 * up(tokens)
        if not log_buckets:
            step = 1024 * -(-tokens // (1024 * 256))
            want += up(-(-tokens // step) * 512)
        want += up((((vocab >> log_buckets) + 1) << log_buckets) + 1) + up(-(-tokens // 32) * 2 * cols)
    assert lib.muon_embed_grad_workspace_bytes(tokens, vocab, cols) == want


def heads(n=4, dim=64, **kw):
    return with_(L.MuonHeads(ptr(), n * dim, dim), **kw)


SIZES = dict(tokens=40, k_tokens=40, heads=4, kv_heads=2, dim=64, ld_lse=40, scale=0.125, causal=1)


def attn(**kw):
    return with_(L.MuonAttention(q=heads(), k=heads(2), v=heads(2), o=heads(), lse=ptr(), **SIZES), **kw)


def attn_grad(**kw):
    return with_(L.MuonAttentionGrad(dout=heads(), q=heads(), k=heads(2), v=heads(2), o=heads(), dq=heads(), dk=heads(2), dv=heads(2),
                                     lse=ptr(), **SIZES), **kw)


def test_struct_layouts_of_attention_and_losses_match_header(lib):
    sizes = muon._marshaller().OP_BYTES
    for name, cls in (("muon_attention_t", L.MuonAttention), ("muon_attention_grad_t", L.MuonAttentionGrad),
                      ("muon_distill_t", L.MuonDistill), ("muon_policy_t", L.MuonPolicy)):
        assert sizes[name] == ctypes.sizeof(cls), name


BAD_ATTENTION = [
    dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(k_tokens=-1), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(dim=0),
    dict(dim=60), dict(dim=136), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2),
    dict(zero_rest=8), dict(zero_rest=-1), dict(reserved=1), dict(k_starts=1 << 40), dict(starts=1 << 40, sequences=-1),
    dict(starts=(1 << 40) + 2, sequences=1), dict(starts=1 << 40, sequences=1, k_tokens=39), dict(starts=1 << 40, sequences=1 << 21),
    dict(ld_lse=39), dict(lse=(1 << 41) + 1), dict(q=heads(data=0)), dict(k=heads(2, data=0)), dict(v=heads(2, data=(1 << 41) + 1)),
    dict(q=heads(ld_token=0)), dict(q=heads(ld_head=0)), dict(k=heads(2, ld_token=64)), dict(k=heads(2, ld_token=128, ld_head=65)),
    dict(q=heads(ld_token=1 << 60)), dict(q=heads(ld_head=1 << 60)), dict(q=heads(ld_token=-256))]


def test_attention_refuses(lib):
    def fwd(ws=WS, ws_bytes=1 << 40, **kw):
        return lib.muon_attention(ctypes.byref(attn(**kw)), ws, ws_bytes, None)

    assert lib.muon_attention(None, None, 0, None) == EINVAL and lib.muon_attention_workspace_bytes(None) == 0
    for bad in [*BAD_ATTENTION, dict(o=heads(data=0)), dict(zero_rest=4), dict(o=heads(ld_token=64))]:
        assert fwd(**bad) == EINVAL, bad
    p = ptr()
    assert fwd(q=heads(data=p), o=heads(data=p)) == EALIAS and fwd(o=heads(data=p), lse=p + 64) == EALIAS
    assert fwd(starts=p, sequences=3, lse=p + 12) == EALIAS
    # slices of one buffer, side by side, in steps of one stride, one after the other: shifted by 8 columns they overlap
    # (tests/test_ops_launches.py: unshifted they do not)
    wide = lambda at: heads(4, data=p + 2 * at, ld_token=10 * 64)  # noqa: E731
    mixed = lambda at: heads(4, data=p + 2 * at, ld_token=4 * 192, ld_head=192)  # noqa: E731
    first = lambda at: heads(4, data=p + 2 * at, ld_token=64, ld_head=40 * 64)  # noqa: E731
    for make, apart in ((wide, 256), (mixed, 64), (first, 4 * 40 * 64)):
        assert fwd(q=make(0), o=make(apart - 8)) == EALIAS and fwd(q=make(apart - 8), o=make(0)) == EALIAS
    # few rows over many keys are cut into parts: o and lse of each in the workspace
    long = dict(k_tokens=4096, causal=0)
    need = lib.muon_attention_workspace_bytes(ctypes.byref(attn(**long)))
    assert need == 8 * 40 * 4 * (64 + 1) * 4 and lib.muon_attention_workspace_bytes(ctypes.byref(attn())) == 0
    assert lib.muon_attention_workspace_bytes(ctypes.byref(attn(**long, dim=60))) == 0
    assert fwd(ws=None, **long) == EWORKSPACE and fwd(ws_bytes=need - 1, **long) == EWORKSPACE
    assert fwd(ws=ctypes.c_void_p((1 << 42) + 8), **long) == EWORKSPACE and fwd(lse=1 << 42, **long) == EALIAS
    # nothing to do
    assert fwd(tokens=0, q=heads(data=0), o=heads(data=0), lse=0) == 0


def test_attention_gradient_refuses(lib):
    size = lambda **kw: lib.muon_attention_grad_workspace_bytes(ctypes.byref(attn_grad(**kw)))  # noqa: E731
    long = dict(tokens=9000, k_tokens=9000, ld_lse=9000)
    need = size(**long)
    # lse and rowsum(dout o), which few blocks in one launch form for themselves; three parts of dk and dv
    assert need == 2 * 4 * 9000 * 4 + 2 * 3 * 9000 * 2 * 64 * 4 and size() == 0 and size(**dict(long, dim=60)) == 0
    assert lib.muon_attention_grad_workspace_bytes(None) == 0
    # parts of dq over many keys; parts of dk and dv over many queries
    assert size(k_tokens=4096, causal=0) == 2 * 4 * 40 * 4 + 8 * 40 * 4 * 64 * 4
    assert size(tokens=4096, ld_lse=4096, causal=0) == 2 * 4 * 4096 * 4 + 2 * 16 * 40 * 2 * 64 * 4

    def bwd(ws=WS, ws_bytes=need, **kw):
        return lib.muon_attention_grad(ctypes.byref(attn_grad(**kw)), ws, ws_bytes, None)

    assert lib.muon_attention_grad(None, WS, need, None) == EINVAL
    for bad in [*BAD_ATTENTION, dict(lse=0), dict(dout=heads(data=0)), dict(o=heads(data=0)), dict(dq=heads(data=0)),
                dict(dk=heads(2, data=0)), dict(dv=heads(2, ld_token=64))]:
        assert bwd(**bad) == EINVAL, bad
    assert bwd(ws=None, **long) == EWORKSPACE and bwd(ws_bytes=need - 1, **long) == EWORKSPACE
    assert bwd(ws=ctypes.c_void_p((1 << 42) + 8), **long) == EWORKSPACE
    p = ptr()
    assert bwd(dq=heads(data=1 << 42), **long) == EALIAS and bwd(dk=heads(2, data=p), dv=heads(2, data=p)) == EALIAS
    assert bwd(q=heads(data=p), dq=heads(data=p)) == EALIAS and bwd(lse=p, dv=heads(2, data=p)) == EALIAS
    assert bwd(tokens=0, k_tokens=0, ws=None, ws_bytes=0) == 0


def distill(**kw):
    return with_(L.MuonDistill(logits=ptr(), ids=ptr(), teacher=ptr(), weights=ptr(), loss=ptr(), dlogits=ptr(), tokens=9, vocab=50, top=4,
                               ld_logits=50, ld_ids=4, ld_teacher=4, ld_dlogits=50, temperature=1.0, dtype=F32, teacher_dtype=F32,
                               id_bytes=8), **kw)


def policy(**kw):
    return with_(L.MuonPolicy(logits=ptr(), actions=ptr(), old_logp=ptr(), advantages=ptr(), ref_logp=ptr(), weights=ptr(), loss=ptr(),
                              logp=ptr(), dlogits=ptr(), tokens=9, vocab=50, ld_logits=50, ld_dlogits=50, clip_low=0.2, clip_high=0.2,
                              kl_coef=0.1, temperature=1.0, dtype=F32, id_bytes=8), **kw)


def test_losses_refuse(lib):
    def dis(**kw):
        return lib.muon_distill(ctypes.byref(distill(**kw)), None)

    def pol(**kw):
        return lib.muon_policy(ctypes.byref(policy(**kw)), None)

    assert lib.muon_distill(None, None) == EINVAL and lib.muon_policy(None, None) == EINVAL
    nan, inf = float("nan"), float("inf")
    both = [dict(logits=0), dict(loss=0), dict(tokens=-1), dict(tokens=1 << 31), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(dtype=5),
            dict(id_bytes=2), dict(ld_logits=49), dict(ld_dlogits=49), dict(temperature=0.0), dict(temperature=-1.0),
            dict(temperature=nan), dict(temperature=inf), dict(logits=(1 << 41) + 2), dict(loss=(1 << 41) + 2),
            dict(weights=(1 << 41) + 1)]
    for bad in [*both, dict(ids=0), dict(teacher=0), dict(top=0), dict(top=1025), dict(teacher_dtype=3), dict(ld_ids=3), dict(ld_teacher=3),
                dict(ids=(1 << 41) + 4)]:
        assert dis(**bad) == EINVAL, bad
    for bad in [*both, dict(actions=0), dict(old_logp=0), dict(advantages=0), dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=nan),
                dict(clip_high=-1.0), dict(clip_high=inf), dict(kl_coef=nan), dict(kl_coef=inf), dict(logp=(1 << 41) + 2)]:
        assert pol(**bad) == EINVAL, bad
    p = ptr()
    assert dis(logits=p, dlogits=p) == EALIAS and dis(loss=p, weights=p) == EALIAS and dis(ids=p, dlogits=p + 64) == EALIAS
    assert pol(logits=p, dlogits=p) == EALIAS and pol(loss=p, logp=p + 32) == EALIAS and pol(logp=p, old_logp=p) == EALIAS
    assert dis(tokens=0, logits=0, loss=0) == 0 and pol(tokens=0, logits=0, actions=0) == 0


def test_binding_of_attention_and_losses_refuses_cpu_tensors(lib):
    q, x, v = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 64), torch.zeros(4)
    i = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: muon.attention(q, q, q), lambda: muon.attention_grad(q, q, q, q, q, x), lambda: muon.distill_loss(x, i[:, None], x),
                 lambda: muon.policy_loss(x, i, v, v)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def bytes_of(t, tokens, n, dim):
    return {t.data + 2 * (i * t.ld_token + h * t.ld_head) + b for i in range(tokens) for h in range(n) for b in range(2 * dim)}


def attention_of(q, o, n_q, n_kv, tokens, dim, lib, **kw):
    far = lambda n: heads(n, dim)  # noqa: E731
    op = with_(L.MuonAttention(q=q, k=far(n_kv), v=far(n_kv), o=o, tokens=tokens, k_tokens=tokens, heads=n_q, kv_heads=n_kv, dim=dim,
                               ld_lse=tokens, scale=1.0), **kw)
    return lib.muon_attention(ctypes.byref(op), WS, 1 << 40, None)


def test_slices_of_a_padded_buffer_do_not_overlap(lib):
    """Heads in steps whose tokens have a stride of their own: side by side in every head, padded columns, unlike numbers of heads."""
    p, tokens, n, dim = ptr(), 40, 4, 64
    for lt, lh, apart in ((3 * n * dim + dim, 3 * dim, dim), (3 * n * dim + 8, 3 * dim, 2 * dim), (3 * n * (dim + 8), dim + 8, n * (dim + 8)),
                          (3 * dim, 3 * dim * (tokens + 2), dim), (dim, dim * (3 * tokens + 1), dim * tokens)):
        one = L.MuonHeads(p, lt, lh)
        mine, seen = bytes_of(one, tokens, n, dim), set()
        for at in (apart, apart - 8, apart - 16, apart + 8, apart - dim, 0):
            other = L.MuonHeads(p + 2 * at, lt, lh)
            meet = bool(mine & bytes_of(other, tokens, n, dim))
            assert not (meet and at == apart)
            for q, o in ((one, other), (other, one)):
                got = attention_of(q, o, n, n, tokens, dim, lib)
                assert got == EALIAS if meet else got not in (EALIAS, EINVAL), (lt, lh, at)
            seen.add(meet)
        assert seen == {False, True}
    # q of 4 heads and dk, dv of 2 behind them, all in steps of padded columns
    at = lambda head: L.MuonHeads(p + 2 * head * 72, 8 * 72, 72)  # noqa: E731
    op = attn_grad(dq=at(0), dk=at(4), dv=at(6))
    assert lib.muon_attention_grad(ctypes.byref(op), WS, 1 << 40, None) not in (EALIAS, EINVAL)
    for bad in (dict(dk=at(3)), dict(dv=at(5)), dict(dq=at(1))):
        assert lib.muon_attention_grad(ctypes.byref(with_(attn_grad(dq=at(0), dk=at(4), dv=at(6)), **bad)), WS, 1 << 40, None) == EALIAS


def test_overlap_of_heads_against_sets_of_bytes(lib):
    """Random strides: a call whose output shares a byte with an input is always refused; one whose tensors have the same
    strides only then."""
    rng, apart, shared = random.Random(5), 0, 0
    for _ in range(4000):
        tokens, n, dim = rng.randint(1, 5), rng.randint(1, 4), rng.choice([8, 16])
        inner = rng.choice([dim, dim + 8, 2 * dim, 3 * dim, 3 * dim + 8])

        def strides():
            if rng.random() < 0.5:
                return rng.choice([n * inner, n * inner + 8, 3 * n * inner, (n - 1) * inner + dim]), inner
            return inner, rng.choice([tokens * inner, tokens * inner + 8, 3 * tokens * inner, (tokens - 1) * inner + dim])
        (lt, lh), p = strides(), ptr()
        other = strides() if rng.random() < 0.3 else (lt, lh)
        q, o = L.MuonHeads(p, lt, lh), L.MuonHeads(p + 2 * rng.randint(-8 * inner, 8 * inner), *other)
        got = attention_of(q, o, n, n, tokens, dim, lib)
        meet = bool(bytes_of(q, tokens, n, dim) & bytes_of(o, tokens, n, dim))
        assert got != EINVAL and (got == EALIAS if meet else True), (tokens, n, dim, lt, lh, other, o.data - p)
        if other == (lt, lh) and not meet:
            inside = max(bytes_of(q, tokens, n, dim)) >= o.data and max(bytes_of(o, tokens, n, dim)) >= p
            assert got != EALIAS, (tokens, n, dim, lt, lh, o.data - p)
            apart += inside
        shared += meet
    assert apart > 200 and shared > 500

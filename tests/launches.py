"""The launches of the training operators' C entries, noted on a machine without
a GPU (launch_recorder.cpp).

``record(calls)`` makes the calls in a child process with the recorder preloaded,
(entry, arguments) each, and returns (status, launches) for each, a launch being
(kernel with its template arguments, grid, block).  A call's matrices lie at
made-up addresses far apart, which nothing reads; its workspace has the size that
the library asks for."""
import atexit
import ctypes
import functools
import json
import os
import re
import shutil
import subprocess
import sys
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAR = 1 << 43                                    # bytes between a call's matrices, more than any of them has


@functools.lru_cache(maxsize=None)
def _recorder():
    cxx = shutil.which("g++")
    if cxx is None:
        return None
    where = tempfile.mkdtemp(prefix="launch_recorder")
    atexit.register(shutil.rmtree, where, ignore_errors=True)
    out = os.path.join(where, "recorder.so")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", os.path.join(ROOT, "tests", "launch_recorder.cpp"),
                        "-o", out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    return out


def record(calls):
    import pytest
    so = _recorder()
    if so is None:
        pytest.skip("no host C++ compiler")
    env = dict(os.environ)
    env["LD_PRELOAD"] = so + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env.pop("MUON_DEBUG", None)
    r = subprocess.run([sys.executable, "-m", "tests.launches"], cwd=ROOT, env=env, input=json.dumps(calls), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = []
    for status, log in json.loads(r.stdout):
        launches = []
        for line in log.splitlines():
            *dims, name = line.split(" ", 6)
            kernel = re.search(r"(k_\w+(?:<[^(]*>)?)", name).group(1)
            launches.append((kernel, tuple(int(d) for d in dims[:3]), tuple(int(d) for d in dims[3:])))
        out.append((status, launches))
    return out


def _child():
    from matrix_aware_optimizer_libmuon_amd import _lib as L
    lib = L.load()
    take = ctypes.CDLL(None).recorder_take
    take.restype = ctypes.c_char_p
    at = [FAR]

    def ptr():
        at[0] += FAR
        return at[0]

    def act8(cols):
        return L.MuonAct8(ptr(), ptr(), cols, -(-cols // 32))

    def heads(n, dim):
        return L.MuonHeads(ptr(), n * dim, dim)

    def attention(entry, tokens, k_tokens, heads_, kv, dim, sequences, odd=False, layout=None, causal=1):
        ends = dict(starts=ptr() if sequences else None, k_starts=ptr() if sequences else None, sequences=sequences, tokens=tokens,
                    k_tokens=k_tokens, heads=heads_, kv_heads=kv, dim=dim, ld_lse=max(tokens, 1), scale=1.0, causal=causal, zero_rest=3)
        own, shared = (lambda: heads(heads_, dim)), (lambda: heads(kv, dim))
        q, k, v = own(), shared(), shared()
        if layout:                                   # all heads of a kind in one buffer (tokens == k_tokens, heads_ == kv)
            base, places = ptr(), iter(range(9))
            own = shared = {  # noqa: E731
                "side by side": lambda: L.MuonHeads(base + 2 * next(places) * heads_ * dim, 9 * heads_ * dim, dim),
                "in steps": lambda: L.MuonHeads(base + 2 * next(places) * dim, heads_ * 9 * dim, 9 * dim),
                "one after the other": lambda: L.MuonHeads(base + 2 * next(places) * heads_ * tokens * dim, dim, tokens * dim)}[layout]
            q, k, v = own(), own(), own()
        if odd:                                      # rows on 2 bytes
            q.data += 2
            v.data += 2
        if entry == "attention":
            op = L.MuonAttention(q=q, k=k, v=v, o=own(), lse=ptr(), **ends)
            return lib.muon_attention(ctypes.byref(op), ctypes.c_void_p(1 << 60), lib.muon_attention_workspace_bytes(ctypes.byref(op)), None)
        op = L.MuonAttentionGrad(dout=own(), q=q, k=k, v=v, o=own(), dq=own(), dk=shared(), dv=shared(), lse=ptr(), **ends)
        return lib.muon_attention_grad(ctypes.byref(op), ctypes.c_void_p(1 << 60),
                                       lib.muon_attention_grad_workspace_bytes(ctypes.byref(op)), None)

    def loss(entry, tokens, vocab, dtype):
        t = L.MUON_BF16 if dtype == "bf16" else L.MUON_F32
        if entry == "distill":
            return lib.muon_distill(ctypes.byref(L.MuonDistill(
                logits=ptr(), ids=ptr(), teacher=ptr(), loss=ptr(), dlogits=ptr(), tokens=tokens, vocab=vocab, top=4, ld_logits=vocab,
                ld_ids=4, ld_teacher=4, ld_dlogits=vocab, temperature=1.0, dtype=t, teacher_dtype=L.MUON_F32, id_bytes=4)), None)
        return lib.muon_policy(ctypes.byref(L.MuonPolicy(
            logits=ptr(), actions=ptr(), old_logp=ptr(), advantages=ptr(), loss=ptr(), dlogits=ptr(), tokens=tokens, vocab=vocab,
            ld_logits=vocab, ld_dlogits=vocab, temperature=1.0, dtype=t, id_bytes=4)), None)

    def call(entry, rows=0, cols=0, tokens=0, vocab=0, n=0, k=0, dtype="f32", accumulate=0, **more):
        if entry.startswith("attention"):
            return attention(entry, tokens, **more)
        if entry in ("distill", "policy"):
            return loss(entry, tokens, vocab, dtype)
        t, ws = L.MUON_BF16 if dtype == "bf16" else L.MUON_F32, ctypes.c_void_p(1 << 60)
        ref = ctypes.byref
        if entry == "act8_pack":
            return lib.muon_act8_pack(ptr(), cols, t, rows, cols, ref(act8(cols)), None)
        if entry == "act8_unpack":
            return lib.muon_act8_unpack(ref(act8(cols)), rows, cols, ptr(), cols, t, None)
        if entry == "rmsnorm":
            return lib.muon_rmsnorm_act8(ref(L.MuonRmsnorm(x=ptr(), h=ptr(), y=ptr(), n=act8(cols), rstd=ptr(), rows=rows, cols=cols,
                                                           ld_x=cols, ld_h=cols, ld_y=cols, eps=1e-6, dtype=t)), None)
        if entry == "rmsnorm_grad":
            op = L.MuonRmsnormGrad(dy=ptr(), rstd=ptr(), n=act8(cols), dx=ptr(), dgain=ptr(), rows=rows, cols=cols, ld_dy=cols,
                                   ld_dx=cols, dtype=t)
            return lib.muon_rmsnorm_act8_grad(ref(op), ws, lib.muon_rmsnorm_act8_grad_workspace_bytes(rows, cols), None)
        if entry == "swiglu":
            return lib.muon_swiglu_act8(ref(L.MuonSwiglu(gate=ptr(), up=ptr(), a=ptr(), gate8=act8(cols), up8=act8(cols), rows=rows,
                                                         cols=cols, ld_gate=cols, ld_up=cols, ld_a=cols, dtype=t)), None)
        if entry == "swiglu_grad":
            return lib.muon_swiglu_act8_grad(ref(L.MuonSwigluGrad(da=ptr(), gate8=act8(cols), up8=act8(cols), dgate=ptr(), dup=ptr(),
                                                                  a8=act8(cols), rows=rows, cols=cols, ld_da=cols, ld_dgate=cols,
                                                                  ld_dup=cols, dtype=t)), None)
        if entry == "wgrad":        # rows padded to whole vectors and groups, as the library's own 8-bit matrices are
            x8 = L.MuonAct8(ptr(), ptr(), -(-k // 32) * 32, -(-k // 32))
            op = L.MuonAct8Wgrad(dy=ptr(), x8=x8, dw=ptr(), tokens=tokens, n=n, k=k, ld_dy=n, ld_dw=k, dw_dtype=t, accumulate=accumulate)
            return lib.muon_act8_wgrad(ref(op), ws, lib.muon_act8_wgrad_workspace_bytes(ref(op)), None)
        if entry == "embed":
            return lib.muon_embed(ref(L.MuonEmbed(table=ptr(), ids=ptr(), out=ptr(), tokens=tokens, vocab=vocab, cols=cols, ld_table=cols,
                                                  ld_out=cols, scale=1.0, table_dtype=t, out_dtype=t, id_bytes=4)), None)
        op = L.MuonEmbedGrad(dy=ptr(), ids=ptr(), dtable=ptr(), tokens=tokens, vocab=vocab, cols=cols, ld_dy=cols, ld_dtable=cols,
                             scale=1.0, dy_dtype=t, table_dtype=t, id_bytes=4, accumulate=accumulate)
        return lib.muon_embed_grad(ref(op), ws, lib.muon_embed_grad_workspace_bytes(tokens, vocab, cols), None)

    out = []
    for entry, args in json.load(sys.stdin):
        status = call(entry, **args)
        out.append((status, take().decode()))
    json.dump(out, sys.stdout)


if __name__ == "__main__":
    _child()

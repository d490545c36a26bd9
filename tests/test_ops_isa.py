"""The bounded global -> LDS loads of the weight gradient (asm statements,
outside the compiler's hazard padding) keep the gfx9 wait states after a vector
write of a scalar register they read, as the direct loads of the GEMM engine
(tests/isa_hazards.py): base descriptor, scalar offset and m0."""
import os
import re
import shutil
import subprocess

import pytest

from matrix_aware_optimizer_libmuon_amd import build
from tests import isa_hazards as H

HIPCC = build.HIPCC
_BUFFER = re.compile(r"buffer_load_(?:dwordx4|ubyte) (v\d+), (s\[\d+:\d+\]), (s\d+|0) offen lds")


def _scan(text):
    """The scanner's own form of the buffer loads: one scalar register range per operand."""
    text, n = _BUFFER.subn(r"global_load_lds_dwordx4 \1, \2, \3", text)
    assert "offen lds" not in text, "a buffer load to LDS of another form"
    return n, H.scan(text)


def test_scan_sees_descriptor_offset_and_m0():
    body = "k:\n\t%s\n\tbuffer_load_dwordx4 v2, s[8:11], s3 offen lds\n\ts_endpgm\n"
    for reg in ("s8", "s11", "s3", "m0"):
        n, bad = _scan(body % f"v_readfirstlane_b32 {reg}, v1")
        assert n == 1 and [h.wait_states for h in bad] == [0], reg
    for line in ("v_readfirstlane_b32 s4, v1", "s_mov_b32 s8, s1", "v_readfirstlane_b32 s8, v1\n\ts_nop 4"):
        assert _scan(body % line)[1] == []


@pytest.mark.skipif(not (os.path.exists(HIPCC) or shutil.which(HIPCC)), reason="hipcc not available")
def test_weight_gradient_keeps_the_wait_states(tmp_path):
    src, extra = next(s for s in build.SOURCES if s[0] == "muon_wgrad.hip")
    out = str(tmp_path / "wgrad.s")
    r = subprocess.run([HIPCC, *build.FLAGS, *extra, "--offload-device-only", "-S", "-o", out, os.path.join(build.CSRC, src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    n, bad = _scan(text)
    assert n > 20
    # and the one wait state after a scalar write of m0
    assert len(re.findall(r"s_nop 0\s+buffer_load_\w+ .* offen lds", text)) == n
    assert not bad, [(h.load, h.writer, h.wait_states) for h in bad[:5]]


@pytest.mark.skipif(not (os.path.exists(HIPCC) or shutil.which(HIPCC)), reason="hipcc not available")
def test_attention_keeps_the_wait_states(tmp_path):
    """Every load to LDS comes behind 5 wait states of its own."""
    src, extra = next(s for s in build.SOURCES if s[0] == "muon_attn.hip")
    out = str(tmp_path / "attn.s")
    r = subprocess.run([HIPCC, *build.FLAGS, *extra, "--offload-device-only", "-S", "-o", out, os.path.join(build.CSRC, src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    loads = re.findall(r"buffer_load_\w+ .* offen lds", text)
    assert len(loads) > 100 and len(re.findall(r"s_nop 4\s+buffer_load_\w+ .* offen lds", text)) == len(loads)

"""The argument checks and launch plans of the training operators under
AddressSanitizer (CPU only): as tests/test_host_asan.py, for the host tests of
those operators."""
import os
import subprocess
import sys

import pytest

from matrix_aware_optimizer_libmuon_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.timeout(600)
def test_operator_checks_are_clean_under_address_sanitizer(tmp_path):
    rt = build.asan_runtime()
    if rt is None:
        pytest.skip("no AddressSanitizer runtime in the ROCm toolchain")
    lib = build.build_asan(str(tmp_path / "asan"))
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1"
    env["MUON_LIB"] = lib
    env.pop("PYTEST_XDIST_WORKER", None)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_ops_host.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=540)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout, tail
    assert "AddressSanitizer" not in r.stderr, tail

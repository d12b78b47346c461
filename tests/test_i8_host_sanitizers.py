"""The host code of the 8-bit integer entry points under AddressSanitizer and UBSan (no GPU).

As test_host_sanitizers.py does for the other entry points: the host tests test_i8_host.py and
test_i8_limits_host.py run in a child interpreter on a build whose host code is sanitized (the
device code is that of the product build). A sanitizer report, or a check that returns another
status than the documented one, fails the test.
"""
import os
import subprocess
import sys

import pytest

from mxfp4_mixture_experts_route_amd import build as moe_build

san = pytest.importorskip("test_host_sanitizers")   # (its flags and runtime; host trees only)

FILES = ("test_i8_host.py", "test_i8_limits_host.py")


@pytest.mark.timeout(900)
def test_i8_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    rt = san.asan_runtime()
    if not rt:
        pytest.skip("no AddressSanitizer runtime next to hipcc")
    so = moe_build.build(extra=san.SAN, out_path=str(tmp_path / "libmoe_mx4_san.so"),
                         build_dir=str(tmp_path / "obj"), link_extra=san.SAN)
    env = dict(os.environ)
    env.update(MOE_MX4_LIB=so, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    cmd = [sys.executable, "-m", "pytest", *(os.path.join(san.ROOT, "tests", f) for f in FILES), "-q",
           "-s", "-p", "no:cacheprovider", "-m", "not gpu"]
    r = subprocess.run(cmd, cwd=san.ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout, out[-2000:]

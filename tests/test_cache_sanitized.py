"""The host side of the calls that fill and read a cache and attend prompts under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only; csrc/vts_cache_api.hip holds no kernels, and stand-ins take
the place of the launches): tests/sanitize/cache_battery.cpp runs clean over shapes from the smallest
to the limits."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_cache_host_side_under_asan_and_ubsan(tmp_path):
    exe = tmp_path / "cache_battery"
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined"]
    b = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", *san,
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                        os.path.join(ROOT, "varlen_top_select_amd", "csrc", "vts_cache_api.hip"),
                        os.path.join(ROOT, "tests", "sanitize", "cache_battery.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "runtime error" not in r.stderr and "cache battery clean" in r.stdout

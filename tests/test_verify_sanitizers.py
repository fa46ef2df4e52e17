"""The host layer of the verification of drafted tokens (argument checks and
workspace sizes) under AddressSanitizer and UndefinedBehaviorSanitizer, on the
CPU: its sources with the sanitizers on the host code, driven by
tests/sanitize/verify_checks.cpp. Every call returns before any launch."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from rl_policy_gradient_amd.build import CSRC, FUSED, HIPCC, ROOT
from tests.test_operators_sanitizers import SAN, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_verify_host_layer_clean_under_asan_and_ubsan(tmp_path):
    common = ["-x", "hip", "-O1", "-g", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    dev = ["--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    jobs = [[HIPCC, *dev, *common, *SAN, "-c", os.path.join(CSRC, s), "-o", str(tmp_path / (s + ".o"))]
            for s in (*FUSED, "verify_api.cpp", "verify.hip")]  # FUSED: errors and the workspace's checks
    jobs.append([HIPCC, "--cuda-host-only", *common, *SAN, "-c",
                 os.path.join(ROOT, "tests", "sanitize", "verify_checks.cpp"), "-o", str(tmp_path / "checks.o")])
    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        list(ex.map(_run, jobs))
    exe = tmp_path / "checks"
    _run([HIPCC, "--offload-arch=gfx950", *SAN, *sorted(str(p) for p in tmp_path.glob("*.o")), "-o", str(exe)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:exitcode=24")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
    assert "verify checks passed" in r.stdout

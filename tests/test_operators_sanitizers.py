"""The host layer of the operators around the fused loss (argument checks,
workspace sizes, the launch tables' bounds) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: every source of the library with the
sanitizers on its host code, driven by tests/sanitize/operator_checks.cpp.
Every call returns before any launch."""
import concurrent.futures as cf
import os
import subprocess

import pytest

from rl_policy_gradient_amd.build import CSRC, HIPCC, ROOT, SOURCES

# sanitizers on the host code only, each flag right after -Xarch_host
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all"]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, "\n".join(l for l in r.stderr.splitlines() if "recognized feature" not in l)[-4000:]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_operators_host_layer_clean_under_asan_and_ubsan(tmp_path):
    common = ["-x", "hip", "-O1", "-g", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    dev = ["--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    jobs = [[HIPCC, *dev, *common, *SAN, "-c", os.path.join(CSRC, s), "-o", str(tmp_path / (s + ".o"))]
            for s in SOURCES]
    jobs.append([HIPCC, "--cuda-host-only", *common, *SAN, "-c",
                 os.path.join(ROOT, "tests", "sanitize", "operator_checks.cpp"), "-o", str(tmp_path / "checks.o")])
    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        list(ex.map(_run, jobs))
    exe = tmp_path / "checks"
    _run([HIPCC, "--offload-arch=gfx950", *SAN, *sorted(str(p) for p in tmp_path.glob("*.o")), "-o", str(exe)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1:exitcode=24")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
    assert "operator checks passed" in r.stdout

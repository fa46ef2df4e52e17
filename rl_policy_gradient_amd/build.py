"""Build libplp.so (HIP, gfx950) in-tree with hipcc.

Usage: python -m rl_policy_gradient_amd.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libplp.so")
BUILD = os.path.join(ROOT, "_build")

# The fused path's own sources, then those of the operators around it: every
# other file of csrc that is compiled by itself.
FUSED = ["lmhead_fwd.hip", "lmhead_fwd_o.hip", "lmhead_mfma.hip", "lmhead_generic.hip", "loss_stage.hip",
         "plp_api.cpp"]
SOURCES = FUSED + sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")) and f not in FUSED)

# Per-source compiler options. Both two-role sweeps are faster without the
# scheduler's unclustered high-register-pressure rescheduling stage (measured
# on MI355X: weight gradient about 1 % at 512 to 16384 tokens, forward 1-2 %
# at 512 and 4096 tokens, with and without a bias; same results bit for bit).
EXTRA = {
    "lmhead_mfma.hip": ["-mllvm", "-amdgpu-disable-unclustered-high-rp-reschedule"],
    "lmhead_fwd_o.hip": ["-mllvm", "-amdgpu-disable-unclustered-high-rp-reschedule"],
}

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
COMMON = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    # packed fp32 instructions are kept out of the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    "-Wno-unused-command-line-argument",
]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON, *EXTRA.get(src, []), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Rpass-analysis=kernel-resource-usage")
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if verbose and err:
        print(err, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))

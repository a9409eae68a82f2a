"""Builds libnaju.so (hipcc, gfx950) in-tree.

    python -m selective_state_space_naju_amd.build [--verbose]

Every HIP source is compiled with packed-fp32 instruction selection turned
off (``-Xclang -target-feature -Xclang -packed-fp32-ops``) and without the
atomic optimizer's wave aggregation.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnaju.so")
SOURCES = ["naju_api.hip", "naju_fwd.hip", "naju_fwd_mfma.hip", "naju_fwd_mfma64.hip", "naju_bwd.hip",
           "naju_bwd_mfma.hip",
           "naju_step.hip", "naju_mixer.hip", "naju_embed.hip",
           "naju_distill.hip", "naju_logits.hip", "naju_w4.hip"]
ARCH = os.environ.get("NAJU_OFFLOAD_ARCH", "gfx950")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         # single-lane counter atomics stay plain: the wave-aggregating rewrite
         # reads the result back at once, which would wait out the round trip
         "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
         # the iterative instruction scheduler aimed at occupancy: the chunk kernels
         # are held at two waves per SIMD by their launch bounds, and within that it
         # interleaves their long dependency chains better than the default (block
         # forward 99.6 -> 94.8 us, block backward 254.3 -> 251.6 us at 8 x 2048 x
         # 1536; the other workloads within 1 %)
         "-mllvm", "-amdgpu-sched-strategy=iterative-maxocc",
         "-I" + os.path.join(ROOT, "include"), "-Wno-unused-command-line-argument"]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(CSRC, src.replace(".hip", ".o"))
    cmd = [HIPCC] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Rpass-analysis=kernel-resource-usage")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libnaju.so.  Returns the library path."""
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    # (hipBLASLt runs the mixer layer's projections)
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs + [
        "-L/opt/rocm/lib", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr)
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))

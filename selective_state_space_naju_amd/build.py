"""Builds libnaju.so (hipcc, gfx950) and the binding's _tensors.so (g++) in-tree.

    python -m selective_state_space_naju_amd.build [--verbose]

Every HIP source is compiled with packed-fp32 instruction selection turned
off (``-Xclang -target-feature -Xclang -packed-fp32-ops``) and without the
atomic optimizer's wave aggregation.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnaju.so")
TENSORS = os.path.join(HERE, "_tensors.so")
SOURCES = ["naju_api.hip", "naju_fwd.hip", "naju_fwd_mfma.hip", "naju_fwd_mfma64.hip", "naju_bwd.hip",
           "naju_bwd_mfma.hip",
           "naju_step.hip", "naju_mixer.hip", "naju_embed.hip",
           "naju_distill.hip", "naju_logits.hip", "naju_w4.hip",
           "naju_norm.hip", "naju_adamw.hip", "naju_linattn.hip"]
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


def _compile_tensors() -> None:
    """The binding's helper for lists of tensors: host code on torch's headers."""
    import torch
    from torch.utils import cpp_extension
    tmp = TENSORS + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    cmd += ["-I" + d for d in cpp_extension.include_paths()]
    cmd += ["-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "naju_tensors.cpp"),
            "-o", tmp]
    cmd += ["-L" + d for d in cpp_extension.library_paths()]
    r = subprocess.run(cmd + ["-ltorch_python", "-ltorch_cpu", "-lc10"], capture_output=True,
                       text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for naju_tensors.cpp:\n%s" % r.stderr)
    os.replace(tmp, TENSORS)


def build(verbose: bool = False) -> str:
    """Compile every HIP source, link libnaju.so, and compile _tensors.so.  Returns the path of
    libnaju.so, which is there also where _tensors.so fails (that error is raised behind it)."""
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        tensors = ex.submit(_compile_tensors)
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
        tensors.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))

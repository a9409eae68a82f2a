"""Host code of the entry points around the mixer layer under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only): their HIP sources and the file that
holds the shared checks are built with the sanitizers on the host compilation
only, and tests/sanitize/lm_driver.cpp drives argument checks, workspace sizing
and empty problems.  Leak checking is off: the HIP runtime keeps allocations
until exit."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_naju_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANGXX = "/opt/rocm/llvm/bin/clang++"


def run(cmd, env=None):
    r = subprocess.run(cmd, capture_output=True, text=True, env=env, timeout=600)
    return r.returncode, r.stdout + r.stderr


def test_lm_entry_points_host_side_under_asan_ubsan(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)):
        pytest.skip("hipcc / clang++ not found")
    from selective_state_space_naju_amd import build
    flags = ["--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I" + os.path.join(ROOT, "include"), "-Wno-unused-command-line-argument",
             "-Wno-inline-asm",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        return run([HIPCC] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]) + (obj,)
    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, build.SOURCES))
    for rc, out, _ in results:
        assert rc == 0, "hipcc failed:\n" + out[-3000:]
    lib = str(tmp_path / "libnaju_lm_san.so")
    rc, out = run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib] +
                  [o for _, _, o in results] +
                  ["-L/opt/rocm/lib", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"])
    assert rc == 0, "link failed:\n" + out[-3000:]
    exe = str(tmp_path / "lm_driver")
    cmd = [CLANGXX, "-O1", "-g", "-std=c++17"]
    cmd += ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    cmd += ["-fno-omit-frame-pointer", "-I" + os.path.join(ROOT, "include"),
            os.path.join(ROOT, "tests", "sanitize", "lm_driver.cpp"), "-o", exe,
            "-L" + str(tmp_path), "-lnaju_lm_san", "-Wl,-rpath," + str(tmp_path),
            "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    rc, out = run(cmd)
    assert rc == 0, "driver build failed:\n" + out[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    rc, out = run([exe], env=env)
    assert rc == 0 and "lm driver: ok" in out, out[-5000:]

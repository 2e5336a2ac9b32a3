"""The host code of the 8-bit activation path (validation, workspace sizes, launch arithmetic) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: the whole library is built with the sanitizers on host code only and driven
through the C ABI with fake device pointers and extreme sizes (tests/sanitize/mx8_driver.c)."""
import concurrent.futures
import os
import subprocess

import pytest

from nvfp4_quantized_gemm_amd import build

HERE = os.path.join(build.ROOT, "tests", "sanitize")
INCLUDE = "-I" + os.path.join(build.ROOT, "include")


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd[:3])} ...: rc {r.returncode}\n{r.stdout[-3000:]}\n{r.stderr[-6000:]}"
    return r


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not installed")
def test_mx8_host_code_under_asan_ubsan(tmp_path):
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-g"]
    common = [build.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-ffp-contract=off",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", INCLUDE] + san

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        _run(common + ["-c"] + (["-x", "hip"] if src.endswith(".cpp") else []) + [os.path.join(build.CSRC, src), "-o", obj])
        return obj

    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as pool:
        objs = list(pool.map(compile_one, build.SOURCES))
    _run([build.HIPCC, "-O1", "-g", INCLUDE] + san +
         ["-x", "c", "-c", os.path.join(HERE, "mx8_driver.c"), "-o", drv])
    _run([build.HIPCC, "--offload-arch=gfx950"] + san + [drv] + objs + ["-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = _run([exe], env=env, timeout=300)
    assert "mx8 driver ok" in r.stdout
    assert "runtime error" not in r.stderr

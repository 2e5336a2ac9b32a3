"""The host code of the attention calls (validation, workspace sizes, launch arithmetic), and the index arithmetic that their
kernels take device data through, under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: the sources are
built with the sanitizers on host code only and driven through the C ABI with fake device pointers and extreme sizes
(tests/sanitize/attention_driver.c); the index arithmetic with any offsets, lengths and page tables
(tests/sanitize/sequence_index_driver.cpp)."""
import concurrent.futures
import os
import subprocess

import pytest

from nvfp4_quantized_gemm_amd import build

HERE = os.path.join(build.ROOT, "tests", "sanitize")
INCLUDE = "-I" + os.path.join(build.ROOT, "include")
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
SOURCES = ["attention.hip", "attention_backward.hip", "paged_attention.hip", "debug_check.hip", "nvfp4_attention_api.cpp"]


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd[:3])} ...: rc {r.returncode}\n{r.stdout[-3000:]}\n{r.stderr[-6000:]}"
    return r


def test_index_arithmetic_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "driver")
    _run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", build.CSRC,
          os.path.join(HERE, "sequence_index_driver.cpp"), "-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert "sequence index driver ok" in r.stdout


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not installed")
def test_attention_host_code_under_asan_ubsan(tmp_path):
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-g"]
    common = [build.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-ffp-contract=off",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", INCLUDE] + san

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        _run(common + ["-c"] + (["-x", "hip"] if src.endswith(".cpp") else []) + [os.path.join(build.CSRC, src), "-o", obj])
        return obj

    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    with concurrent.futures.ThreadPoolExecutor(max_workers=5) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    _run([build.HIPCC, "-O1", "-g", INCLUDE] + san + ["-x", "c", "-c", os.path.join(HERE, "attention_driver.c"), "-o", drv])
    _run([build.HIPCC, "--offload-arch=gfx950"] + san + [drv] + objs + ["-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert "attention driver ok" in r.stdout
    assert "runtime error" not in r.stderr

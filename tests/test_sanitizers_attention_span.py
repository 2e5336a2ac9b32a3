"""The rows that joining kernels may take, under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU
(tests/sanitize/sequence_span_driver.cpp)."""
import os
import subprocess

from nvfp4_quantized_gemm_amd import build

HERE = os.path.join(build.ROOT, "tests", "sanitize")
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")


def test_rows_of_sequences_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", build.CSRC,
                        os.path.join(HERE, "sequence_span_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], env=ENV, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    assert "sequence span driver ok" in r.stdout

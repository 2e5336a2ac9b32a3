"""The package imports on a torch without its device bindings (a CPU-only build): only calls need them."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_device_bindings():
    code = ("import torch\n"
            "for name in dir(torch._C):\n"
            "    if name.startswith('_cuda_'):\n"
            "        delattr(torch._C, name)\n"
            "import nvfp4_quantized_gemm_amd as nv\n"
            "print(nv.rope_inv_freq((8,), device='cpu').shape[0])\n"
            "try:\n"
            "    nv.nvfp4_mx8_quantize(torch.zeros(2, 32))\n"
            "except ValueError as e:\n"
            "    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[:2] == ["4", "the operands must be device tensors"]

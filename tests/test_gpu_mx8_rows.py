"""RMS norm rows at the ends of the number range, and equal calls giving equal bits.

Tolerances as in the norm's own tests (u = 2^-24): 60 u of |y| and 55 u of inv_rms, plus, where the sum of squares leaves
fp32 and the row is scaled first, one more product and an inv_rms down to 2^-128, where a subnormal's half unit is 4 u:
68 u and 60 u."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_mx8 import check_mx8_of, grad_ref, rnd

pytestmark = pytest.mark.gpu
DEV, U, V = "cuda", 2.0 ** -24, 2.0 ** -8
F32, BF = torch.float32, torch.bfloat16
WIDTHS = [32, 2048, 2080, 8192, 8224, 32768]  # one wave, 256 and 1024 threads a row, with and without rows ahead


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("M", [9, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_with_a_non_finite_value_is_non_finite(M, K, bad):
    x, r = rnd(M, K, seed=K, dtype=BF), rnd(M, K, seed=K + 1, dtype=BF)
    clean = nv.nvfp4_rmsnorm(x.to(DEV), r.to(DEV), y_dtype=F32, save_inv_rms=True)
    x[1, K - 1], r[M - 1, 3] = bad, bad
    out = nv.nvfp4_rmsnorm(x.to(DEV), r.to(DEV), y_dtype=F32, save_inv_rms=True)
    rows = torch.zeros(M, dtype=torch.bool)
    rows[1] = rows[M - 1] = True
    assert (out.scales.cpu()[rows] == 255).all() and ((out.codes.cpu()[rows] & 0x7F) == 0x7F).all()
    assert torch.isnan(out.y.cpu()[rows]).all() and torch.isnan(out.inv_rms.cpu()[rows]).all()
    for a, b in ((out.y, clean.y), (out.codes, clean.codes), (out.scales, clean.scales), (out.inv_rms, clean.inv_rms)):
        assert torch.equal(a.cpu()[~rows], b.cpu()[~rows])
    assert torch.equal(out.h.cpu().isfinite(), (x.float() + r.float()).isfinite())
    fq = nv.nvfp4_rmsnorm(x.to(DEV), r.to(DEV), mx8=False, y_dtype=BF, fake_quantize=True).y.cpu()
    assert torch.isnan(fq[rows]).all() and torch.isfinite(fq[~rows]).all()


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("M", [9, 300])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_whose_squares_leave_fp32(M, K, dtype):
    x = rnd(M, K, seed=K, wide=False).double()
    x = x / x.abs().amax(1, keepdim=True)
    for i, e in ((0, 63.5), (2, 64.5), (3, 80.0), (4, 100.0), (5, 126.0), (M - 1, 127.9)):
        x[i] *= 2.0 ** e
    x[6, :] = 0
    x[6, K // 2] = 2.0 ** 120  # one value alone
    x[7, ::2] *= 2.0 ** 90
    x = x.to(dtype)
    w = (1 + 0.2 * rnd(K, seed=7, wide=False))
    out = nv.nvfp4_rmsnorm(x.to(DEV), None, w.to(DEV), 1e-5, y_dtype=F32, save_inv_rms=True)
    s = x.double()
    inv = 1 / (s.square().mean(1) + 1e-5).sqrt()
    y = (s * inv[:, None] * w.double()).numpy()
    assert (np.abs(out.inv_rms.cpu().double().numpy() - inv.numpy()) <= 60 * U * inv.numpy()).all()
    assert (np.abs(out.y.cpu().double().numpy() - y) <= 68 * U * np.abs(y) + 2.0 ** -149).all()
    top = np.abs(y).reshape(M, -1, 32).max(2).min(1) > 2.0 ** -100  # rows without blocks of subnormals
    t = torch.from_numpy(top)
    check_mx8_of(out.codes.cpu()[t], out.scales.cpu()[t], y[top], 68 * U)
    dy = rnd(M, K, seed=3, dtype=dtype, wide=False)
    dx, dw = nv.nvfp4_rmsnorm_backward(dy.to(DEV), x.to(DEV), out.inv_rms, w.to(DEV))
    rx, tol, rw, aw = grad_ref(dy, x, out.inv_rms.cpu(), w, None)
    tol = tol + 2.0 ** -148 + (V * rx.abs() + 2.0 ** -133 if dtype == BF else 0)
    assert ((dx.cpu().double() - rx).abs() <= tol).all()
    assert ((dw.cpu().double() - rw).abs() <= (M / 256 + 80) * U * aw + 1e-30).all()


def test_a_large_eps_counts_beside_squares_past_fp32():
    x = torch.full((3, 64), 2.0 ** 70)
    x[1] = 2.0 ** 63.5
    x[2] = 1.0
    out = nv.nvfp4_rmsnorm(x.to(DEV), None, None, 3e38, y_dtype=F32, save_inv_rms=True)
    inv = 1 / (x.double().square().mean(1) + float(np.float32(3e38))).sqrt()
    assert ((out.inv_rms.cpu().double() - inv).abs() <= 60 * U * inv).all()


@pytest.mark.parametrize("M,K,dtype", [(16384, 8192, BF), (1003, 2592, F32), (1, 4608, BF)])
def test_equal_calls_give_equal_bits(M, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r = (torch.randn(M, K, generator=g, device=DEV).to(dtype) for _ in range(2))
    x[:, :: 97] *= 20
    w = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(dtype)
    first = nv.nvfp4_rmsnorm(x, r, w, y_dtype=dtype, save_inv_rms=True)
    for i in range(8):
        again = nv.nvfp4_rmsnorm(x, r, w, y_dtype=dtype, save_inv_rms=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again)), i
    at = torch.arange(0, M, max(1, M // 64), device=DEV)  # and they are the norm's
    s = (x[at].double() + r[at].double()).cpu()
    y = (s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double().cpu()).numpy()
    check_mx8_of(first.codes[at], first.scales[at], y, 60 * U)

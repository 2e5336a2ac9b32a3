"""Arrays that the 8-bit path's calls write in place of an input, at another pitch: rows would be overwritten before others
are read, so the calls refuse them on the host (fake device pointers, no GPU is needed)."""
import ctypes

import pytest

import nvfp4_quantized_gemm_amd as nv

S = nv.Status
P = [0x1000000 * (i + 1) for i in range(8)]
STOPS = (S.ERR_HIP, S.ERR_DEVICE)  # past validation: without a GPU the device check ends the call


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def norm(L, x=P[0], ldx=64, r=P[1], ldr=64, dt=nv.BF16, M=4, K=64, h=P[2], ldh=64, y=P[3], ydt=nv.BF16, ldy=64):
    return L.nvfp4_rmsnorm(x, ldx, r, ldr, dt, M, K, None, 0, 1e-6, h, ldh, P[4], P[5], y, ydt, ldy, 0, None, None)


def test_norm_refuses_h_or_y_in_an_inputs_place_at_another_pitch(L):
    for kw in (dict(h=P[0], ldh=72), dict(h=P[0], ldx=72), dict(h=P[1], ldh=72), dict(h=P[1], ldr=72),
               dict(y=P[0], ldy=72), dict(y=P[1], ldr=72), dict(y=P[0], ydt=nv.F32), dict(y=P[1], ydt=nv.F32, M=1)):
        assert norm(L, **kw) == S.ERR_STRIDE, kw


@pytest.mark.skipif(not no_gpu(), reason="fake pointers")
def test_norm_takes_h_or_y_in_an_inputs_place_at_its_pitch(L):
    for kw in (dict(h=P[0]), dict(h=P[1]), dict(h=P[0], ldx=72, ldh=72), dict(y=P[0]), dict(y=P[1]),
               dict(h=P[0], ldh=72, M=1), dict(r=None, h=P[0])):
        assert norm(L, **kw) in STOPS, kw


def backward(L, dy=P[0], ldy=64, h=P[1], ldh=64, dh=P[2], ldd=64, M=4, dx=P[3], ldx=64):
    return L.nvfp4_rmsnorm_backward(dy, ldy, h, ldh, dh, ldd, nv.BF16, M, 64, None, 0, P[4], dx, ldx, None, None, 0, None)


def test_backward_refuses_dx_in_an_inputs_place_at_another_pitch(L):
    for kw in (dict(dx=P[0], ldx=72), dict(dx=P[0], ldy=72), dict(dx=P[1], ldh=72), dict(dx=P[2], ldd=72),
               dict(dx=P[2], ldx=72)):
        assert backward(L, **kw) == S.ERR_STRIDE, kw


@pytest.mark.skipif(not no_gpu(), reason="fake pointers")
def test_backward_takes_dx_in_an_inputs_place_at_its_pitch(L):
    for kw in (dict(dx=P[0]), dict(dx=P[1]), dict(dx=P[2]), dict(dx=P[0], ldx=72, M=1), dict(dx=P[2], ldd=72, ldx=72)):
        assert backward(L, **kw) in STOPS, kw


def test_rope_refuses_y_in_xs_place_at_another_pitch(L):
    dims = (ctypes.c_int32 * 1)(32)
    for lt, lh, yt, yh in ((192, 64, 256, 64), (256, 64, 192, 64), (192, 64, 64, 256)):
        assert L.nvfp4_rope_axes(P[0], nv.BF16, 4, 3, 64, lt, lh, P[1], 1, dims, P[2], 0, 0, P[0], yt, yh, None) == S.ERR_STRIDE

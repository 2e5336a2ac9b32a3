"""What the calls of the 8-bit activation path refuse, on the host: no GPU is needed (fake device pointers are never
dereferenced, because validation fails first)."""
import ctypes

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

S = nv.Status
P, P8, PODD = 0x10000, 0x10008, 0x10001


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def test_quantize(L):
    def q(x=P, dt=nv.BF16, M=4, K=64, ld=64, c=P, s=P):
        return L.nvfp4_mx8_quantize(x, dt, M, K, ld, c, s, None)
    assert q(dt=9) == S.ERR_DTYPE
    for kw in (dict(M=-1), dict(K=0), dict(K=16), dict(K=48), dict(M=1 << 41)):
        assert q(**kw) == S.ERR_SHAPE, kw
    for name in ("x", "c", "s"):
        assert q(**{name: None}) == S.ERR_NULL
    assert q(ld=56) == S.ERR_STRIDE and q(ld=1 << 62) == S.ERR_SHAPE
    assert q(x=P8) == S.ERR_ALIGN and q(ld=68) == S.ERR_ALIGN and q(c=P8) == S.ERR_ALIGN
    assert q(M=0, x=None, c=None, s=None) == S.OK


def norm(L, x=P, ldx=64, r=P, ldr=64, dt=nv.BF16, M=4, K=64, w=P, wdt=nv.F32, eps=1e-6, h=P, ldh=64, c=P, s=P, y=P,
         ydt=nv.F32, ldy=64, inv=P):
    return L.nvfp4_rmsnorm(x, ldx, r, ldr, dt, M, K, w, wdt, eps, h, ldh, c, s, y, ydt, ldy, 0, inv, None)


def test_rmsnorm(L):
    for kw in (dict(dt=2), dict(wdt=-1), dict(ydt=5)):
        assert norm(L, **kw) == S.ERR_DTYPE, kw
    for kw in (dict(K=40), dict(M=-2), dict(K=32800, ldx=40000, ldr=40000, ldh=40000, ldy=40000)):
        assert norm(L, **kw) == S.ERR_SHAPE, kw
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(L, eps=eps) == S.ERR_MODE, eps
    for kw in (dict(x=None), dict(c=None), dict(s=None), dict(c=None, s=None, y=None)):
        assert norm(L, **kw) == S.ERR_NULL, kw
    for kw in (dict(ldx=32), dict(ldr=56), dict(ldh=8), dict(ldy=63)):
        assert norm(L, **kw) == S.ERR_STRIDE, kw
    for kw in (dict(x=P8), dict(r=PODD), dict(h=P8), dict(y=P8), dict(w=P8), dict(c=P8), dict(inv=PODD), dict(ldx=68),
               dict(ldy=65)):
        assert norm(L, **kw) == S.ERR_ALIGN, kw
    assert norm(L, M=0, x=None, r=None, h=None, c=None, s=None, y=None) == S.OK


def test_rmsnorm_backward(L):
    need = L.nvfp4_rmsnorm_backward_workspace_bytes(300, 64)
    assert need > 0 and L.nvfp4_rmsnorm_backward_workspace_bytes(300, 65) == 0

    def b(dy=P, h=P, dh=P, ldy=64, ldh=64, lddh=64, dt=nv.F32, M=300, K=64, w=P, wdt=nv.F32, inv=P, dx=P, ldx=64, dw=P,
          ws=P, n=need):
        return L.nvfp4_rmsnorm_backward(dy, ldy, h, ldh, dh, lddh, dt, M, K, w, wdt, inv, dx, ldx, dw, ws, n, None)
    assert b(dt=3) == S.ERR_DTYPE and b(wdt=3) == S.ERR_DTYPE and b(K=33) == S.ERR_SHAPE
    for name in ("dy", "h", "inv", "dx"):
        assert b(**{name: None}) == S.ERR_NULL, name
    for name in ("ldy", "ldh", "lddh", "ldx"):
        assert b(**{name: 32}) == S.ERR_STRIDE and b(**{name: 66}) == S.ERR_ALIGN, name
    assert b(ws=None) == S.ERR_WORKSPACE and b(n=need - 1) == S.ERR_WORKSPACE
    assert b(ws=P8) == S.ERR_ALIGN and b(dw=P8) == S.ERR_ALIGN and b(dh=P8) == S.ERR_ALIGN
    assert b(M=0, dw=None) == S.OK


def test_w4a8(L):
    def g(a=P, sa=P, b=P, sb=P, M=4, N=8, K=64, c=P, dt=nv.F32, ldc=8):
        return L.nvfp4_mx_gemm_w4a8(a, sa, b, sb, M, N, K, c, dt, ldc, None)
    assert g(dt=4) == S.ERR_DTYPE
    for kw in (dict(M=-1), dict(N=-1), dict(K=16), dict(K=80), dict(M=1 << 30, K=32), dict(N=1 << 30, K=32, ldc=1 << 30)):
        assert g(**kw) == S.ERR_SHAPE, kw
    for name in ("a", "sa", "b", "sb", "c"):
        assert g(**{name: None}) == S.ERR_NULL, name
    for kw in (dict(a=P8), dict(b=P8), dict(sa=PODD), dict(sb=PODD), dict(c=P8)):
        assert g(**kw) == S.ERR_ALIGN, kw
    assert g(ldc=7) == S.ERR_STRIDE
    assert g(M=0, a=None) == S.OK and g(N=0, c=None) == S.OK


def test_rope(L):
    def r(x=P, dt=nv.BF16, T=4, H=3, D=64, lt=192, lh=64, pos=P, dims=(32, 16), f=P, layout=0, y=P + 0x100000, yt=192,
          yh=64, n=None, no_dims=False):
        arr = None if no_dims else (ctypes.c_int32 * max(1, len(dims)))(*dims)
        return L.nvfp4_rope_axes(x, dt, T, H, D, lt, lh, pos, len(dims) if n is None else n, arr, f, layout, 0, y, yt, yh,
                                 None)
    assert r(dt=2) == S.ERR_DTYPE and r(layout=2) == S.ERR_MODE
    for kw in (dict(T=-1), dict(H=-1), dict(D=0), dict(D=60), dict(D=1032), dict(n=0), dict(n=5), dict(dims=(31,)),
               dict(dims=(-2,)), dict(dims=(40, 32)), dict(H=(1 << 20) + 1), dict(T=1 << 31)):
        assert r(**kw) == S.ERR_SHAPE, kw
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(f=None), dict(no_dims=True)):
        assert r(**kw) == S.ERR_NULL, kw
    for kw in (dict(yt=64), dict(yh=56), dict(yh=0), dict(lt=-8), dict(lt=1 << 50), dict(y=P, yt=256), dict(y=P, lh=72)):
        assert r(**kw) == S.ERR_STRIDE, kw
    for kw in (dict(x=P8), dict(y=P8), dict(lt=196), dict(yt=196), dict(pos=PODD), dict(f=PODD)):
        assert r(**kw) == S.ERR_ALIGN, kw
    assert r(T=0, x=None) == S.OK and r(H=0, y=None) == S.OK


def test_python_refuses_host_tensors_and_wrong_forms():
    x = torch.zeros(4, 64)
    u = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nv.nvfp4_mx8_quantize(x)
    with pytest.raises(ValueError):
        nv.nvfp4_mx8_quantize(x.t())
    with pytest.raises(ValueError):
        nv.nvfp4_rmsnorm(x, torch.zeros(4, 32))
    with pytest.raises(ValueError):
        nv.nvfp4_rmsnorm(x, x.bfloat16())
    with pytest.raises(ValueError):
        nv.nvfp4_rmsnorm(x[0])
    with pytest.raises(ValueError):
        nv.nvfp4_rmsnorm_backward(x, x, torch.zeros(3))
    with pytest.raises(ValueError):
        nv.nvfp4_mx_gemm_w4a8(u, u[:, :3], u[:, :32], u[:, :2])
    with pytest.raises(ValueError):
        nv.nvfp4_mx_gemm_w4a8(u[:, ::2], u, u, u)
    with pytest.raises(ValueError):
        nv.nvfp4_rope_axes(x.view(4, 2, 32), torch.zeros(4, 2), (32,), torch.zeros(16))
    with pytest.raises(ValueError):
        nv.nvfp4_rope_axes(x.view(4, 2, 32), torch.zeros(4, 1), (32,), torch.zeros(15))
    with pytest.raises(ValueError):
        nv.nvfp4_rope_axes(x, torch.zeros(4, 1), (32,), torch.zeros(16))

"""The differentiable entry points of the 8-bit activation path on the CPU: the library's calls are replaced by plain torch
stand-ins that take only what the C ABI takes (16-byte aligned rows at a pitch of at least K and of whole 16 bytes), so
every gradient and every input that autograd can hand over has to arrive in that form."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

EPS = 1e-6


def takes_rows(t, K):
    assert t.dim() == 2 and t.shape[1] == K and t.stride(1) == 1 and t.data_ptr() % 16 == 0
    if t.shape[0] > 1:
        assert t.stride(0) >= K and t.stride(0) * t.element_size() % 16 == 0


def takes_heads(t):
    es = t.element_size()
    assert t.dim() == 3 and t.stride(2) == 1 and t.data_ptr() % 16 == 0
    for dim in (0, 1):
        assert t.shape[dim] == 1 or (t.stride(dim) >= 0 and t.stride(dim) * es % 16 == 0)


def plain_rmsnorm(x, residual=None, weight=None, eps=EPS, *, mx8=True, y_dtype=None, fake_quantize=False,
                  save_inv_rms=False, h=None, stream=None):
    takes_rows(x, x.shape[1])
    s = x
    if residual is not None:
        takes_rows(residual, x.shape[1])
        s = h = x + residual
    if weight is not None:
        assert weight.is_contiguous() and weight.data_ptr() % 16 == 0
    inv = torch.rsqrt(s.square().mean(1) + eps)
    y = s * inv[:, None] * (1 if weight is None else weight)
    return nv.RMSNormOutput(h, None, None, y, inv)


def plain_backward(dy, h, inv_rms, weight=None, dh=None, *, dweight=True, dx=None, workspace=None, stream=None):
    for t in (dy, h) if dh is None else (dy, h, dh):
        takes_rows(t, h.shape[1])
    if weight is not None:
        assert weight.is_contiguous() and weight.data_ptr() % 16 == 0
    n, g = h * inv_rms[:, None], dy * (1 if weight is None else weight)
    out = inv_rms[:, None] * (g - n * (g * n).mean(1, keepdim=True)) + (0 if dh is None else dh)
    return out, (dy * n).sum(0) if dweight else None


def plain_rope(x, positions, axis_dims, inv_freq, *, layout=nv.ROPE_PAIRS, inverse=False, out=None, stream=None):
    takes_heads(x)
    d = sum(axis_dims)
    axis = torch.repeat_interleave(torch.arange(len(axis_dims)), torch.tensor(axis_dims) // 2)
    ang = (positions[:, axis] * inv_freq)[:, None] * (-1 if inverse else 1)
    y = x.clone()
    x1, x2 = x[..., 0:d:2], x[..., 1:d:2]
    y[..., 0:d:2], y[..., 1:d:2] = x1 * ang.cos() - x2 * ang.sin(), x2 * ang.cos() + x1 * ang.sin()
    return y


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    monkeypatch.setattr(nv, "nvfp4_rmsnorm", plain_rmsnorm)
    monkeypatch.setattr(nv, "nvfp4_rmsnorm_backward", plain_backward)
    monkeypatch.setattr(nv, "nvfp4_rope_axes", plain_rope)


def reference(x, r, w):
    s = x if r is None else x + r
    return s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * w, s


LOSSES = {
    "sum over tokens": lambda y, h, u: (y.sum(0) * u).sum(),
    "sum over tokens of both": lambda y, h, u: (y.sum(0) * u).sum() + (h.sum(0) * u.square()).sum(),
    "mean of all": lambda y, h, u: (y * u).mean(),
    "behind three values": lambda y, h, u: torch.cat([u[:3], y.flatten(), h.flatten()]).square().sum(),
    "behind one row": lambda y, h, u: torch.cat([u[None], y, h]).square().sum(),
    "one row": lambda y, h, u: (y[2] * u).sum(),
}


@pytest.mark.parametrize("name", LOSSES)
@pytest.mark.parametrize("form", ["dense", "expanded", "overlapping", "offset", "transposed"])
def test_rmsnorm_takes_every_gradient_and_input(name, form):
    M, K = 5, 64
    torch.manual_seed(1)
    leaf = {"dense": lambda: torch.randn(M, K), "expanded": lambda: torch.randn(1, K),
            "overlapping": lambda: torch.randn(K + 8 * (M - 1)), "offset": lambda: torch.randn(M * K + 3),
            "transposed": lambda: torch.randn(K, M)}[form]
    view = {"dense": lambda t: t, "expanded": lambda t: t.expand(M, K),
            "overlapping": lambda t: t.as_strided((M, K), (8, 1)), "offset": lambda t: t[3:].view(M, K),
            "transposed": lambda t: t.t()}[form]
    a, b, w, u = leaf().requires_grad_(), leaf().requires_grad_(), torch.rand(K).requires_grad_(), torch.randn(K)
    grads = []
    for f in (lambda x, r: nv.rmsnorm(x, r, w, EPS), lambda x, r: reference(x, r, w)):
        y, h = f(view(a), view(b))
        LOSSES[name](y, h, u).backward()
        grads.append([t.grad for t in (a, b, w)])
        a.grad = b.grad = w.grad = None
    for got, want in zip(*grads):
        if want is None:
            want = torch.zeros_like(got)
        assert torch.allclose(got, want, rtol=1e-4, atol=1e-5 * float(want.abs().max()))


@pytest.mark.parametrize("form", ["offset", "expanded", "strided"])
def test_rmsnorm_takes_every_weight(form):
    K = 64
    torch.manual_seed(2)
    x = torch.randn(3, K)
    leaf = {"offset": torch.rand(K + 1), "expanded": torch.rand(1), "strided": torch.rand(2 * K)}[form].requires_grad_()
    w = {"offset": lambda: leaf[1:], "expanded": lambda: leaf.expand(K), "strided": lambda: leaf[::2]}[form]
    grads = []
    for f in (lambda: nv.rmsnorm(x, None, w(), EPS)[0], lambda: reference(x, None, w())[0]):
        f().square().sum().backward()
        grads.append(leaf.grad)
        leaf.grad = None
    assert torch.allclose(*grads, rtol=1e-4, atol=1e-5 * float(grads[1].abs().max()))


@pytest.mark.parametrize("form", ["dense", "expanded", "offset", "strided", "odd pitch", "heads first"])
def test_rope_takes_every_gradient_and_input(form):
    T, H, D, dims = 3, 4, 16, (8, 4)
    torch.manual_seed(3)
    leaf = {"dense": (T, H, D), "expanded": (T, 1, D), "offset": (T * H * D + 3,), "strided": (T, H, 2 * D),
            "odd pitch": (T, H, D + 1), "heads first": (H, T, D)}[form]
    view = {"dense": lambda t: t, "expanded": lambda t: t.expand(T, H, D), "offset": lambda t: t[3:].view(T, H, D),
            "strided": lambda t: t[..., ::2], "odd pitch": lambda t: t[..., :D],
            "heads first": lambda t: t.transpose(0, 1)}[form]
    pos, f, u = torch.rand(T, 2) * 9, nv.rope_inv_freq(dims, device="cpu"), torch.randn(T, H, D)
    x = torch.randn(leaf).requires_grad_()
    back = plain_rope(u, pos, dims, f, inverse=True)
    for loss in (lambda y: (y * u).sum(), lambda y: torch.cat([u[0, 0, :3], (y * u).flatten()]).sum(),
                 lambda y: (torch.cat([u[0, 0, :3], y.flatten()]) * torch.cat([u[0, 0, :3], u.flatten()])).sum()):
        loss(nv.rope_axes(view(x), pos, dims, f)).backward()
        want = x.detach().clone().requires_grad_()
        (view(want) * back).sum().backward()
        assert torch.allclose(x.grad, want.grad, rtol=1e-4, atol=1e-5)
        x.grad = None
    total = nv.rope_axes(view(x), pos, dims, f).sum(0)  # a gradient of stride 0 along the tokens
    (total * u[0]).sum().backward()
    assert x.grad is not None and torch.isfinite(x.grad).all()

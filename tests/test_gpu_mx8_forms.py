"""The differentiable entry points of the 8-bit activation path on tensors as autograd and models hand them over: expanded,
overlapping, strided and off 16 bytes.  A copy changes no bits, so what the kernels give for the given form has to equal
what they give for a dense copy of it."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


def rnd(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def off16(t):
    """A contiguous copy of t that starts 3 elements into its memory."""
    big = torch.empty(t.numel() + 3, dtype=t.dtype, device=t.device)
    big[3:] = t.flatten()
    return big[3:].view(t.shape)


ROWS = {"dense": lambda t: t, "expanded": lambda t: t[:1].expand(t.shape), "off 16 bytes": off16,
        "overlapping": lambda t: t.flatten().as_strided(t.shape, (16, 1)), "columns": lambda t: t.t().contiguous().t()}


@pytest.mark.parametrize("M,K", [(1, 96), (7, 96), (130, 2304)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form", ROWS)
def test_rmsnorm(M, K, dtype, form):
    x, r, dy, dh = (ROWS[form](rnd(M, K, seed=i, dtype=dtype)) for i in range(4))
    w = 1 + 0.1 * rnd(K, seed=5)
    xs, rs, ws = (t.detach().requires_grad_() for t in (x, r, w))
    y, h = nv.rmsnorm(xs, rs, ws)
    dense = [t.clone(memory_format=torch.contiguous_format) for t in (x, r, w, dy, dh)]
    want = nv.nvfp4_rmsnorm(*dense[:3], mx8=False, y_dtype=dtype, save_inv_rms=True)
    assert torch.equal(y, want.y) and torch.equal(h, want.h)
    dx, dw = nv.nvfp4_rmsnorm_backward(dense[3], want.h, want.inv_rms, dense[2], dense[4])
    gx, gr, gw = torch.autograd.grad((y, h), (xs, rs, ws), (dy, dh))
    assert torch.equal(gx, dx) and torch.equal(gr, dx) and torch.equal(gw, dw)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rmsnorm_under_sums_over_tokens_and_behind_other_values(dtype):
    x, u = rnd(2, 9, 96, seed=1, dtype=dtype).requires_grad_(), rnd(2, 96, seed=2, dtype=dtype)
    w = torch.ones(96, device=DEV, requires_grad=True)
    want = torch.autograd.grad(nv.rmsnorm(x, None, w)[0], (x, w), u[:, None].expand(2, 9, 96).contiguous())
    got = torch.autograd.grad((nv.rmsnorm(x, None, w)[0].sum(1) * u).sum(), (x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    v = rnd(3 + 2 * 9 * 96, seed=3, dtype=dtype)
    want = torch.autograd.grad(nv.rmsnorm(x, None, w)[0], (x, w), v[3:].clone().view(2, 9, 96))
    got = torch.autograd.grad((torch.cat([v[:3], nv.rmsnorm(x, None, w)[0].flatten()]) * v).sum(), (x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form", ["off 16 bytes", "expanded", "strided"])
def test_rmsnorm_weight(dtype, form):
    M, K = 7, 96
    w = {"off 16 bytes": lambda t: off16(t), "expanded": lambda t: t[:1].expand(K),
         "strided": lambda t: t.repeat_interleave(2)[::2]}[form](1 + 0.1 * rnd(K, seed=5, dtype=dtype))
    x, dy = rnd(M, K, seed=1, dtype=dtype), rnd(M, K, seed=2, dtype=dtype)
    xs, ws, wd = (t.detach().requires_grad_() for t in (x, w, w.clone(memory_format=torch.contiguous_format)))
    y, want = nv.rmsnorm(xs, None, ws)[0], nv.rmsnorm(xs, None, wd)[0]
    assert torch.equal(y, want)
    for a, b in zip(torch.autograd.grad(y, (xs, ws), dy), torch.autograd.grad(want, (xs, wd), dy)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K", [(3, 96), (3000, 96), (300, 4608), (5, 32768)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradients_in_an_input_s_place(M, K, dtype):
    dy, h, dh = (rnd(M, K, seed=i, dtype=dtype) for i in range(3))
    inv, w = 1 / h.float().square().mean(1).sqrt(), 1 + 0.1 * rnd(K, seed=5)
    dx, dw = nv.nvfp4_rmsnorm_backward(dy, h, inv, w, dh)
    for i in range(3):
        t = [dy.clone(), h.clone(), dh.clone()]
        got, gw = nv.nvfp4_rmsnorm_backward(t[0], t[1], inv, w, t[2], dx=t[i])
        assert got is t[i] and torch.equal(got, dx) and torch.equal(gw, dw), i


HEADS = {"dense": lambda t: t, "expanded heads": lambda t: t[:, :1].expand(t.shape), "off 16 bytes": off16,
         "expanded tokens": lambda t: t[:1].expand(t.shape), "heads first": lambda t: t.transpose(0, 1).contiguous().transpose(0, 1),
         "strided": lambda t: t.repeat_interleave(2, 2)[..., ::2],
         "odd pitches": lambda t: torch.cat([t, t[..., :1]], 2)[..., : t.shape[2]]}


@pytest.mark.parametrize("T,H", [(1, 1), (1, 5), (6, 1), (6, 5)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", [nv.ROPE_PAIRS, nv.ROPE_HALVES])
@pytest.mark.parametrize("form", HEADS)
def test_rope(T, H, dtype, layout, form):
    D, dims = 72, (24, 20, 16)
    x, dy = (HEADS[form](rnd(T, H, D, seed=i, dtype=dtype)) for i in range(2))
    pos, f = torch.arange(3 * T, device=DEV).view(T, 3).float(), nv.rope_inv_freq(dims)
    xs = x.detach().requires_grad_()
    y = nv.rope_axes(xs, pos, dims, f, layout)
    dense = [t.clone(memory_format=torch.contiguous_format) for t in (x, dy)]
    assert torch.equal(y, nv.nvfp4_rope_axes(dense[0], pos, dims, f, layout=layout))
    dx, = torch.autograd.grad(y, xs, dy)
    assert torch.equal(dx, nv.nvfp4_rope_axes(dense[1], pos, dims, f, layout=layout, inverse=True))

@pytest.mark.parametrize("T,H", [(1, 1), (1, 5), (6, 1)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rope_of_one_token_or_one_head_at_any_pitch(T, H, dtype):
    """The pitch of a dimension of one element is never used, whatever it is."""
    D, dims, odd = 72, (24, 20, 16), 72 * H * T + 13
    x = rnd(T, H, D, seed=1, dtype=dtype)
    pos, f = torch.arange(3 * T, device=DEV).view(T, 3).float(), nv.rope_inv_freq(dims)
    want = nv.nvfp4_rope_axes(x, pos, dims, f)
    big = torch.zeros(2 * odd, dtype=dtype, device=DEV)
    strides = (odd if T == 1 else D * H, odd if H == 1 else D, 1)
    view = big.as_strided((T, H, D), strides)
    view.copy_(x)
    assert torch.equal(nv.nvfp4_rope_axes(view, pos, dims, f), want)
    assert nv.nvfp4_rope_axes(view, pos, dims, f, out=view) is view and torch.equal(view, want)

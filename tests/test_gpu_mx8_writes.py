"""Tensors that the 8-bit path's calls write into count as written: autograd sees it, and one whose gradient is being
recorded is refused, because the call itself records none."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def rows(seed, dtype=BF, K=96):
    return torch.randn(4, K, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def test_a_saved_sum_that_a_later_norm_overwrites_is_noticed():
    x, r, z = (rows(i) for i in range(3))
    w = torch.ones(96, device=DEV, requires_grad=True)
    y, h = nv.rmsnorm(x.requires_grad_(), r, w)
    with torch.no_grad():
        nv.nvfp4_rmsnorm(z, h, h=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_saved_input_that_a_rotation_overwrites_is_noticed():
    x = rows(1, torch.float32).requires_grad_()
    s = x.exp()  # saves its result
    with torch.no_grad():
        heads = s.view(4, 3, 32)
        nv.nvfp4_rope_axes(heads, torch.ones(4, 1, device=DEV), (32,), nv.rope_inv_freq((32,)), out=heads)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        s.sum().backward()


def calls():
    """Every call with a tensor to write into: name, the call with it, a maker of that tensor."""
    x, r, pos, f = rows(1), rows(2), torch.ones(4, 1, device=DEV), nv.rope_inv_freq((32,))
    inv, w = torch.ones(4, device=DEV), torch.ones(96, device=DEV)
    c, s = nv.nvfp4_mx8_quantize(x)
    b, sb = nv.nvfp4_mx_quantize(rows(3))
    return [("norm", lambda t: nv.nvfp4_rmsnorm(x, r, h=t), lambda: r.clone()),
            ("backward", lambda t: nv.nvfp4_rmsnorm_backward(x, r, inv, w, dx=t), lambda: r.clone()),
            ("product", lambda t: nv.nvfp4_mx_gemm_w4a8(c, s, b, sb, out=t), lambda: torch.empty(4, 4, device=DEV)),
            ("rope", lambda t: nv.nvfp4_rope_axes(x.view(4, 3, 32), pos, (32,), f, out=t), lambda: x.view(4, 3, 32).clone()),
            ("codes", lambda t: nv.nvfp4_mx8_quantize(x, codes=t), lambda: c.clone()),
            ("scales", lambda t: nv.nvfp4_mx8_quantize(x, scales=t), lambda: s.clone())]


@pytest.mark.parametrize("name", ["norm", "backward", "product", "rope", "codes", "scales"])
def test_written_tensors_count_as_written(name):
    call, make = {n: (f, m) for n, f, m in calls()}[name]
    t = make()
    before = t._version
    call(t)
    assert t._version > before
    with torch.inference_mode():
        call(make())
    torch.cuda.synchronize()
    if t.dtype is torch.uint8:
        return
    t = make().requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        call(t)
    with torch.no_grad():
        call(t)
    torch.cuda.synchronize()


def test_the_example_s_serving_calls_write_without_gradients():
    x, r = rows(1), rows(2)
    n = nv.nvfp4_rmsnorm(x, r)
    assert nv.nvfp4_rmsnorm(x, n.h, h=n.h).h is n.h

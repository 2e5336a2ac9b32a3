"""The example's training block rounds what its serving block rounds, to the same formats: MXFP4 weights, MXFP8 inputs of
both products.  All values are compared for equality."""
import os
import sys

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_mx8 import dequantized

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import w4a8_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_training_multiplies_what_serving_multiplies(monkeypatch):
    grid, heads, head_dim, dims = (2, 5, 7), 4, 72, (24, 24, 24)
    hidden, tokens = heads * head_dim, 70
    x, r, w_qkv, w_out, nw, _ = ex.make_inputs(tokens, hidden, seed=5)
    pos, inv_freq = ex.grid_positions(*grid, x.device), nv.rope_inv_freq(dims)
    seen, linear = [], ex.F.linear
    monkeypatch.setattr(ex.F, "linear", lambda a, w: seen.append((a.detach(), w.detach())) or linear(a, w))
    params = [t.clone().requires_grad_() for t in (w_qkv, w_out, nw)]
    out, _ = ex.training_block(x, r, pos, dims, inv_freq, heads, *params)
    (qkv_in, qkv_w), (out_in, out_w) = seen
    for got, w in ((qkv_w, w_qkv), (out_w, w_out)):
        assert torch.equal(got, nv.nvfp4_mx_dequantize(*nv.nvfp4_mx_quantize(w), w.dtype))
    n = nv.nvfp4_rmsnorm(x, r, nw)
    assert (qkv_in.cpu().double().numpy() == dequantized(n.codes, n.scales)).all()
    assert (out_in.cpu().double().numpy() == dequantized(*nv.nvfp4_mx8_quantize(out_in))).all()
    out.float().square().mean().backward()
    assert all(bool((p.grad != 0).any()) and bool(torch.isfinite(p.grad).all()) for p in params)


def test_straight_through_gradients():
    w = (0.02 * torch.randn(64, 96, device="cuda")).to(torch.bfloat16).requires_grad_()
    g = torch.randn(64, 96, device="cuda").to(torch.bfloat16)
    assert torch.equal(torch.autograd.grad(ex.mx4_weight(w), w, g)[0], g)
    t = torch.randn(64, 96, device="cuda", requires_grad=True)
    y = ex.mx8_activation(t, torch.bfloat16)
    assert (y.detach().cpu().double().numpy() == dequantized(*nv.nvfp4_mx8_quantize(t.detach()))).all()
    assert torch.equal(torch.autograd.grad(y, t, g)[0], g.float())

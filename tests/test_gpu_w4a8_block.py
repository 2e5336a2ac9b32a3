"""The example block (examples/w4a8_block.py): the serving path against the same path in 64 bits with the same quantized
operands, and the training path's gradients against a plain fp32 block.

Tolerances: every step of the serving path is compared on the operands that the step before really produced, so only its
own rounding counts: the norms as in their own tests, the products 1e-5 sum|a b| + bf16's rounding."""
import os
import sys

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_mx8 import check_mx8_of, check_product, mx_values, U

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import w4a8_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grid,heads,head_dim,dims", [((2, 5, 7), 4, 72, (24, 24, 24)), ((1, 1, 1), 2, 64, (24, 20, 20)),
                                                      ((3, 8, 16), 3, 128, (44, 42, 42))])
def test_serving_block_steps(grid, heads, head_dim, dims):
    hidden, tokens = heads * head_dim, grid[0] * grid[1] * grid[2]
    x, r, w_qkv, w_out, nw, nw2 = ex.make_inputs(tokens, hidden, seed=tokens)
    pos = ex.grid_positions(*grid, x.device)
    block = ex.ServingBlock(hidden, heads, dims, w_qkv, w_out, nw, nw2)
    codes, scales, h = block(x, r, pos)
    # the same calls, one by one, each against its definition
    n = nv.nvfp4_rmsnorm(x, r, nw)
    s = x.cpu().double() + r.cpu().double()
    y = s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * nw.cpu().double()
    check_mx8_of(n.codes, n.scales, y.numpy(), 60 * U)
    qkv = nv.nvfp4_mx_gemm_w4a8(n.codes, n.scales, *block.qkv)
    check_product(qkv, *mx_values(*(t.cpu() for t in (n.codes, n.scales, *block.qkv))))
    qkv = qkv.view(tokens, 3 * heads, head_dim)
    turned = nv.nvfp4_rope_axes(qkv[:, : 2 * heads], pos, dims, block.inv_freq)
    att = ex.attention(turned[:, :heads], turned[:, heads:], qkv[:, 2 * heads:])
    a, sa = nv.nvfp4_mx8_quantize(att)
    out = nv.nvfp4_mx_gemm_w4a8(a, sa, *block.out)
    check_product(out, *mx_values(*(t.cpu() for t in (a, sa, *block.out))))
    after = nv.nvfp4_rmsnorm(out, n.h, nw2)
    assert torch.equal(after.h, h) and torch.equal(after.codes, codes) and torch.equal(after.scales, scales)


def test_training_block_learns_and_matches_the_plain_block_where_nothing_is_quantized():
    grid, heads, head_dim, dims = (2, 4, 8), 2, 64, (24, 20, 20)
    hidden, tokens = heads * head_dim, 64
    x, r, w_qkv, w_out, nw, _ = ex.make_inputs(tokens, hidden, seed=3)
    pos, inv_freq = ex.grid_positions(*grid, x.device), nv.rope_inv_freq(dims)
    target = 0.1 * torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).to(x)
    params = [t.clone().requires_grad_() for t in (w_qkv, w_out, nw)]
    losses = []
    for _ in range(6):
        out, _ = ex.training_block(x, r, pos, dims, inv_freq, heads, *params)
        loss = (out.float() - target.float()).square().mean()
        loss.backward()
        assert all(torch.isfinite(p.grad).all() for p in params)
        with torch.no_grad():
            for p in params:
                p -= 0.5 * p.grad
                p.grad = None
        losses.append(float(loss.detach()))
    assert losses[-1] < losses[0]
    # norm and rotation together, fp32, against torch's own autograd in 64 bits
    xs, rs, ws = (t.float().clone().requires_grad_() for t in (x, r, nw))
    y, h = nv.rmsnorm(xs, rs, ws)
    z = nv.rope_axes(y.view(tokens, heads, head_dim), pos, dims, inv_freq)
    u, p = torch.randn_like(z), torch.randn_like(h)
    ((z * u).sum() + (h * p).sum()).backward()
    xd, rd, wd = (t.detach().double().requires_grad_() for t in (xs, rs, ws))
    s = xd + rd
    yd = (s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * wd).view(tokens, heads, head_dim)
    zd, at, q = yd.clone(), 0, 0
    for a, d in enumerate(dims):
        ang = (pos[:, a, None] * inv_freq[q: q + d // 2]).double()[:, None]
        x1, x2 = yd[..., at: at + d: 2], yd[..., at + 1: at + d: 2]
        zd[..., at: at + d: 2] = x1 * ang.cos() - x2 * ang.sin()
        zd[..., at + 1: at + d: 2] = x2 * ang.cos() + x1 * ang.sin()
        at, q = at + d, q + d // 2
    ((zd * u.double()).sum() + (s * p.double()).sum()).backward()
    for got, want in ((xs.grad, xd.grad), (rs.grad, rd.grad), (ws.grad, wd.grad)):
        assert (got.double() - want).abs().max() <= (300 * U + 3e-6) * want.abs().max()

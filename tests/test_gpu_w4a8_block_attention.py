"""The example block on the library's attention (examples/w4a8_block.py): serving and training calls, and a causal model's
prompts and tokens over a paged cache, step by step on the operands that the steps before really produced."""
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import check, definition
from test_gpu_paged_attention import values

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import w4a8_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def block(heads, head_dim, dims, seed=0):
    _, _, w_qkv, w_out, nw, nw2 = ex.make_inputs(1, heads * head_dim, seed=seed)
    return ex.ServingBlock(heads * head_dim, heads, dims, w_qkv, w_out, nw, nw2, ex.library_attention)


@pytest.mark.parametrize("grid,heads,head_dim,dims", [((2, 5, 7), 4, 72, (24, 24, 24)), ((3, 8, 16), 3, 128, (44, 42, 42))])
def test_serving(grid, heads, head_dim, dims):
    tokens = grid[0] * grid[1] * grid[2]
    x, r = ex.make_inputs(tokens, heads * head_dim, seed=tokens)[:2]
    pos, b = ex.grid_positions(*grid, x.device), block(heads, head_dim, dims)
    codes, scales, h = b(x, r, pos)
    (q, k, v), res = b.before(x, r, pos)
    att = ex.library_attention(q, k, v)
    check(att.view(tokens, heads, head_dim), None, definition(q, k, v, [tokens], [tokens], False, head_dim ** -0.5))
    want = b.after(att, res)
    assert all(torch.equal(a, c) for a, c in zip((codes, scales, h), want))


def test_prompts_and_tokens():
    heads, head_dim, dims, prompts, steps = 4, 72, (72, 0, 0), [40, 1, 77], 6
    hidden, b = heads * head_dim, block(heads, head_dim, dims)
    dev = b.inv_freq.device
    pages, table = ex.sequence_pages([n + steps for n in prompts], 16, dev)
    cache = nv.paged_cache(pages, 16, heads, head_dim, mx8=True)
    lengths = torch.tensor(prompts, dtype=torch.int32, device=dev)
    cu = torch.tensor([0] + prompts, device=dev).cumsum(0).int()
    place = lambda t: torch.stack([t, 0 * t, 0 * t], 1).float()  # noqa: E731
    x, r = ex.make_inputs(sum(prompts), hidden, seed=1)[:2]
    pos = place(torch.cat([torch.arange(n, device=dev) for n in prompts]))
    got = b.prompts(x, r, pos, cu, cache, table, lengths)
    (q, k, v), h = b.before(x, r, pos)
    att = nv.nvfp4_attention(q, k, v, causal=True, cu_q=cu, cu_k=cu)[0]
    check(att, None, definition(q, k, v, prompts, prompts, True, head_dim ** -0.5))
    assert all(torch.equal(a, c) for a, c in zip(got, b.after(att.flatten(1), h)))
    for s in range(steps):
        x, r = ex.make_inputs(3, hidden, seed=2 + s)[:2]
        lengths += 1
        got = b.tokens(x, r, place(lengths - 1), cache, table, lengths)
        (q, k, v), h = b.before(x, r, place(lengths - 1))
        att = nv.nvfp4_paged_attention(q, cache, table, lengths)
        keys, vals = values(cache, table, lengths.tolist(), head_dim)
        check(att, None, definition(q, keys, vals, [1] * 3, lengths.tolist(), False, head_dim ** -0.5))
        last = lengths.cumsum(0).long() - 1  # the new tokens' own rows are in the cache, rounded as quantize does
        for cached, mine in ((keys, k), (vals, v)):
            assert bool(((cached[last] - mine.double()).abs() <= mine.double().abs() / 16 + 2.0 ** -9 * mine.double().abs().amax(2, keepdim=True)
                         + mine.double().abs().amax(2, keepdim=True) / 8).all())
        assert all(torch.equal(a, c) for a, c in zip(got, b.after(att.flatten(1), h)))


def test_training_gradients_run():
    grid, heads, head_dim, dims = (2, 4, 8), 2, 64, (24, 20, 20)
    x, r, w_qkv, w_out, nw, _ = ex.make_inputs(64, heads * head_dim, seed=3)
    params = [t.clone().requires_grad_() for t in (w_qkv, w_out, nw)]
    out, _ = ex.training_block(x, r, ex.grid_positions(*grid, x.device), dims, nv.rope_inv_freq(dims), heads, *params,
                               ex.library_attention)
    out.float().square().mean().backward()
    assert all(bool(torch.isfinite(p.grad).all()) and bool((p.grad != 0).any()) for p in params)


def test_command():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "w4a8_block.py"), "--grid", "2,4,8", "--heads", "4", "--steps", "1",
                        "--attention", "library", "--prompts", "30,1,100", "--tokens", "3"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr
    assert "decoding: 3 prompts, 3 tokens each, lengths [33, 4, 103]" in r.stdout and "training: step 0" in r.stdout

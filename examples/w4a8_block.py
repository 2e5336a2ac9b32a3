"""The attention half of a transformer block on the 8-bit activation path, as a video or image model runs it:

  serving   residual + RMS norm -> MXFP8 -> QKV product with an MXFP4 weight -> rotary positions of time, height and
            width on q and k, in place in the QKV output -> attention (torch in fp32, or the library's on q, k and v
            where they lie) -> MXFP8 -> output projection -> the next norm with the residual's addition
  decoding  the same block in a causal model: prompts of different lengths packed together, their keys and values into
            a paged MXFP8 cache, then one token per sequence and step over that cache
  training  the same block with bf16 weights in quantization-aware training: what serving rounds is rounded to the
            same values (MXFP8 inputs of both products, MXFP4 weights), straight-through gradients, a few steps of
            gradient descent

  python examples/w4a8_block.py [--grid 4,32,32] [--heads 16] [--head-dim 72] [--steps 3] [--attention torch|library]
                                [--prompts 300,17,1000] [--tokens 8]
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_quantized_gemm_amd as nv  # noqa: E402


def grid_positions(frames: int, height: int, width: int, device) -> torch.Tensor:
    """fp32 [frames * height * width, 3]: the coordinates of every token."""
    axes = [torch.arange(n, device=device, dtype=torch.float32) for n in (frames, height, width)]
    return torch.stack(torch.meshgrid(*axes, indexing="ij"), -1).reshape(-1, 3).contiguous()


def attention(q, k, v):
    """[T, H, D] each -> [T, H * D], in fp32."""
    q, k, v = (t.float().transpose(0, 1).contiguous() for t in (q, k, v))
    out = F.scaled_dot_product_attention(q.unsqueeze(0), k.unsqueeze(0), v.unsqueeze(0))
    return out[0].transpose(0, 1).reshape(q.shape[1], -1)


def library_attention(q, k, v):
    """The same on the library's kernels, bf16: no copies, differentiable."""
    return nv.attention(q, k, v).flatten(1)


class ServingBlock:
    """MXFP4 weights, MXFP8 activations."""

    def __init__(self, hidden: int, heads: int, axis_dims, w_qkv, w_out, norm_weight, next_norm_weight, attend=attention):
        self.attend = attend
        self.heads, self.head_dim, self.axis_dims = heads, hidden // heads, axis_dims
        self.qkv, self.out = nv.nvfp4_mx_quantize(w_qkv), nv.nvfp4_mx_quantize(w_out)  # once per weight
        self.norm_weight, self.next_norm_weight = norm_weight, next_norm_weight
        self.inv_freq = nv.rope_inv_freq(axis_dims, device=w_qkv.device)

    def before(self, x, residual, positions):
        """(q, k, v [T, heads, head_dim] as views of the QKV output, q and k turned; the residual stream)."""
        n = nv.nvfp4_rmsnorm(x, residual, self.norm_weight)
        qkv = nv.nvfp4_mx_gemm_w4a8(n.codes, n.scales, *self.qkv).view(x.shape[0], 3 * self.heads, self.head_dim)
        qk = qkv[:, : 2 * self.heads]
        nv.nvfp4_rope_axes(qk, positions, self.axis_dims, self.inv_freq, out=qk)
        return qkv.split(self.heads, 1), n.h

    def after(self, att, h):
        y = nv.nvfp4_mx_gemm_w4a8(*nv.nvfp4_mx8_quantize(att), *self.out)
        after = nv.nvfp4_rmsnorm(y, h, self.next_norm_weight, h=h)
        return after.codes, after.scales, after.h

    def __call__(self, x, residual, positions):
        """x, residual [T, hidden] bf16 -> (the next linear's MXFP8 codes and scales, the residual stream)."""
        qkv, h = self.before(x, residual, positions)
        return self.after(self.attend(*qkv), h)

    def prompts(self, x, residual, positions, cu, cache, page_table, lengths):
        """The same, causal, for the packed prompts that cu names; their keys and values go into the cache."""
        (q, k, v), h = self.before(x, residual, positions)
        nv.nvfp4_cache_append(k, v, cache, page_table, lengths, cu)
        return self.after(nv.nvfp4_attention(q, k, v, causal=True, cu_q=cu, cu_k=cu)[0].flatten(1), h)

    def tokens(self, x, residual, positions, cache, page_table, lengths):
        """The same for one new token of each sequence, which lengths counts already."""
        (q, k, v), h = self.before(x, residual, positions)
        nv.nvfp4_cache_append(k, v, cache, page_table, lengths)
        return self.after(nv.nvfp4_paged_attention(q, cache, page_table, lengths).flatten(1), h)


def sequence_pages(tokens, page_size: int, device):
    """(pages of a cache, page table) for sequences of up to so many tokens each."""
    need = [-(-n // page_size) for n in tokens]
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    return at, table.to(device)


class StraightThrough(torch.autograd.Function):
    """Takes the quantized values of x forward and their gradient back to x."""

    @staticmethod
    def forward(ctx, x, quantized):
        ctx.dtype = x.dtype
        return quantized.view_as(quantized)

    @staticmethod
    def backward(ctx, grad):
        return grad.to(ctx.dtype), None


def mx4_weight(w):
    """The values of w's MXFP4 codes (exact in bf16)."""
    return StraightThrough.apply(w, nv.nvfp4_mx_dequantize(*nv.nvfp4_mx_quantize(w.detach()), w.dtype))


def mx8_activation(t, dtype):
    """The values of t's MXFP8 codes (exact in bf16)."""
    codes, scales = nv.nvfp4_mx8_quantize(t.detach())
    blocks = codes.view(torch.float8_e4m3fn).float().view(*scales.shape, 32)
    values = blocks * scales.view(torch.float8_e8m0fnu).float().unsqueeze(-1)
    return StraightThrough.apply(t, values.view(t.shape).to(dtype))


def training_block(x, residual, positions, axis_dims, inv_freq, heads, w_qkv, w_out, norm_weight, attend=attention):
    """The block for quantization-aware training: (output, residual stream), differentiable."""
    T, hidden = x.shape
    y, h = nv.rmsnorm(x, residual, norm_weight, fake_quantize=True)
    qkv = F.linear(y, mx4_weight(w_qkv)).view(T, 3 * heads, hidden // heads)
    q, k, v = qkv.split(heads, 1)
    q, k = (nv.rope_axes(t, positions, axis_dims, inv_freq) for t in (q, k))
    return F.linear(mx8_activation(attend(q, k, v), x.dtype), mx4_weight(w_out)), h


def make_inputs(tokens: int, hidden: int, device="cuda", seed: int = 0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    bf = torch.bfloat16
    return (draw(tokens, hidden).to(bf), draw(tokens, hidden).to(bf), (0.02 * draw(3 * hidden, hidden)).to(bf),
            (0.02 * draw(hidden, hidden)).to(bf), (1 + 0.1 * draw(hidden)).to(bf), (1 + 0.1 * draw(hidden)).to(bf))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--grid", default="4,32,32", help="frames, height, width in tokens")
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--head-dim", type=int, default=72)
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--attention", choices=("torch", "library"), default="torch")
    ap.add_argument("--prompts", default="", help="lengths of packed prompts, to decode from")
    ap.add_argument("--tokens", type=int, default=8, help="tokens to decode after each prompt")
    a = ap.parse_args()
    attend = library_attention if a.attention == "library" else attention
    grid = [int(n) for n in a.grid.split(",")]
    hidden, tokens = a.heads * a.head_dim, grid[0] * grid[1] * grid[2]
    third = a.head_dim // 6 * 2
    axis_dims = (a.head_dim - 2 * third, third, third)
    x, residual, w_qkv, w_out, nw, nw2 = make_inputs(tokens, hidden)
    positions = grid_positions(*grid, x.device)

    block = ServingBlock(hidden, a.heads, axis_dims, w_qkv, w_out, nw, nw2, attend)
    codes, scales, h = block(x, residual, positions)
    torch.cuda.synchronize()
    print(f"serving: {tokens} tokens, hidden {hidden}: codes {tuple(codes.shape)}, scales {tuple(scales.shape)}, "
          f"residual rms {h.float().square().mean().sqrt().item():.4f}")

    if a.prompts:
        lens = [int(n) for n in a.prompts.split(",")]
        pages, table = sequence_pages([n + a.tokens for n in lens], 16, x.device)
        cache = nv.paged_cache(pages, 16, a.heads, a.head_dim, mx8=True)
        lengths = torch.tensor(lens, dtype=torch.int32, device=x.device)
        cu = torch.tensor([0] + lens, device=x.device).cumsum(0).int()
        place = lambda t: torch.stack([t, 0 * t, 0 * t], 1).float()  # noqa: E731
        p = make_inputs(sum(lens), hidden, seed=1)
        block.prompts(p[0], p[1], place(torch.cat([torch.arange(n, device=x.device) for n in lens])), cu, cache, table, lengths)
        for step in range(a.tokens):
            t = make_inputs(len(lens), hidden, seed=2 + step)
            lengths += 1
            _, _, h = block.tokens(t[0], t[1], place(lengths - 1), cache, table, lengths)
        torch.cuda.synchronize()
        print(f"decoding: {len(lens)} prompts, {a.tokens} tokens each, lengths {lengths.tolist()}, residual rms "
              f"{h.float().square().mean().sqrt().item():.4f}")

    params = [t.clone().requires_grad_() for t in (w_qkv, w_out, nw)]
    target = 0.1 * torch.randn_like(x)
    inv_freq = nv.rope_inv_freq(axis_dims, device=x.device)
    optimizer = torch.optim.Adam(params, lr=1e-3)
    for step in range(a.steps):
        optimizer.zero_grad()
        out, _ = training_block(x, residual, positions, axis_dims, inv_freq, a.heads, *params, attend)
        loss = (out.float() - target.float()).square().mean()
        loss.backward()
        optimizer.step()
        print(f"training: step {step}, loss {loss.item():.6f}")


if __name__ == "__main__":
    main()

"""attention() takes tensors in any strides: token pitches past what the kernels' tiles address (2^23 elements), at the border
and one step below it."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import BF, DEV, rnd

pytestmark = pytest.mark.gpu


def far(t, pitch):
    """t's values with tokens `pitch` elements apart."""
    T, H, D = t.shape
    memory = torch.zeros((T - 1) * pitch + H * D, dtype=BF, device=DEV)
    view = memory.as_strided((T, H, D), (pitch, D, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("pitch", [(1 << 23) - 8, 1 << 23, (1 << 23) + 64, 1 << 25])
def test_far_tokens(pitch):
    T, H, D = 6, 2, 64
    q, k, v, u = (rnd(T, H, D, seed=i) for i in range(4))
    leaves = [far(t, pitch).detach().requires_grad_() for t in (q, k, v)]
    out = nv.attention(*leaves, causal=True)
    want, lse = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True)
    assert torch.equal(out, want)
    grads = nv.nvfp4_attention_backward(u, q, k, v, want, lse, causal=True)
    for a, b in zip(torch.autograd.grad(out, leaves, far(u, pitch)), grads):
        assert torch.equal(a, b)


def test_the_plain_calls_refuse_them():
    q = far(rnd(3, 2, 64, seed=0), 1 << 23)
    k = rnd(3, 2, 64, seed=1)
    for args in ((q, k, k), (k, q, k), (k, k, q)):
        with pytest.raises(nv.NVFP4Error):
            nv.nvfp4_attention(*args)
    out, lse = nv.nvfp4_attention(k, k, k, save_lse=True)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_attention_backward(q, k, k, k, out, lse)


@pytest.mark.parametrize("D", [64, 72, 128])
def test_whole_tiles_of_far_tokens(D):
    """The widest pitch that the calls take, over tiles of 128 rows: the last lies 2 GiB from the first."""
    T, pitch = 260, (1 << 23) - 8
    wide = torch.zeros(T * pitch, dtype=BF, device=DEV).view(T, pitch)
    dense = [rnd(T, 1, D, seed=i) for i in range(4)]
    q, k, v, u = (wide[:, 128 * i: 128 * i + D].unsqueeze(1) for i in range(4))
    for a, b in zip((q, k, v, u), dense):
        a.copy_(b)
    want, lse = nv.nvfp4_attention(*dense[:3], causal=True, save_lse=True)
    out, sums = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True)
    assert torch.equal(out, want) and torch.equal(sums, lse)
    grads = nv.nvfp4_attention_backward(dense[3], *dense[:3], want, lse, causal=True)
    far_out, far_grads = wide[:, 1024: 1024 + D].unsqueeze(1), [wide[:, 1152 + 128 * i: 1152 + 128 * i + D].unsqueeze(1) for i in range(3)]
    nv.nvfp4_attention(q, k, v, causal=True, out=far_out)
    nv.nvfp4_attention_backward(u, q, k, v, far_out, lse, causal=True, dq=far_grads[0], dk=far_grads[1], dv=far_grads[2])
    assert torch.equal(far_out, want) and all(torch.equal(a, b) for a, b in zip(far_grads, grads))

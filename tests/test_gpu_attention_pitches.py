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

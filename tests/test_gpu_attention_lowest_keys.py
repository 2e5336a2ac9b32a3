"""Gradients of a key that no query weighs (its scores are -inf): its own are 0 at any number of queries, the other keys' are
those without it.  (The queries' are 0 times infinity there: NaN in that place of a head and nowhere else.)"""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import offsets, qkv, rnd
from test_gpu_attention_backward import check, gradients

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nk", [(64, 64), (128, 100), (150, 150), (1, 5), (63, 300), (65, 700), (40, 3000), (2000, 70)])
@pytest.mark.parametrize("D", [16, 64, 72, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 1)])
def test_gradients(nq, nk, D, Hq, Hkv):
    q, k, v = qkv([nq], [nk], Hq, Hkv, D)
    u, j = rnd(nq, Hq, D, seed=9), nk // 2
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    k[j, :, 3] = -math.inf
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True)
    dq, dk, dv = nv.nvfp4_attention_backward(u, q, k, v, out, lse)
    assert bool((dk[j] == 0).all()) and bool((dv[j] == 0).all())
    rest = torch.arange(nk, device=k.device) != j
    wq, wk, wv = gradients(u, q, k[rest], v[rest], [nq], [nk - 1], False, D ** -0.5)
    place = torch.arange(D, device=k.device) != 3
    check((dq[..., place], dk[rest], dv[rest]), ([t[..., place] for t in wq], wk, wv))


def test_packed_and_causal():
    nq, nk, D = [50, 130], [80, 200], 64
    q, k, v = qkv(nq, nk, 4, 2, D)
    u, cu = rnd(180, 4, D, seed=9), dict(cu_q=offsets(nq), cu_k=offsets(nk), causal=True)
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    gone = [20, 100]  # one of each sequence, which every query attends with others
    k[gone, :, 3] = -math.inf
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    dq, dk, dv = nv.nvfp4_attention_backward(u, q, k, v, out, lse, **cu)
    assert bool((dk[gone] == 0).all()) and bool((dv[gone] == 0).all())
    rest = torch.ones(280, dtype=torch.bool, device=k.device)
    rest[gone] = False
    _, wk, wv = gradients(u, q, k[rest], v[rest], nq, [79, 199], True, D ** -0.5)
    check((dk[rest], dv[rest]), (wk, wv), ("dk", "dv"))

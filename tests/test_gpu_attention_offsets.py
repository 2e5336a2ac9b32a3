"""Rows of no sequence where several workgroups share a block of queries or of keys and a second launch joins their sums:
those before the first offset (the offsets of some sequences of a packed batch), behind the last one, and rows of offsets
that descend.  Workspaces are full of NaN and the outputs given, so that a row which no workgroup computed shows."""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import DEV, check, definition, qkv, rnd
from test_gpu_attention_backward import check as check_gradients
from test_gpu_attention_backward import gradients

pytestmark = pytest.mark.gpu
U8 = torch.uint8

# (rows before, lengths of queries, of keys, rows behind, Hq, Hkv, D)
CASES = [(529, [17], [4096], 9, 4, 2, 64), (40, [100, 0, 33], [3000, 20, 2500], 0, 3, 1, 72), (1, [200, 64], [1500, 900], 130, 2, 1, 128),
         (1000, [1000], [1000], 40, 4, 2, 128), (300, [129, 500], [200, 1003], 7, 12, 4, 64)]


def ints(x):
    return torch.tensor(x, dtype=torch.int64).to(torch.int32).to(DEV)


def offsets_from(first, lens):
    return ints([first + sum(lens[:i]) for i in range(len(lens) + 1)])


def full_of_nan(n):
    return torch.full((max(n, 16),), 0xFF, dtype=U8, device=DEV)


def problem(case, seed=0):
    before, nq, nk, tail, Hq, Hkv, D = case
    Tq, Tk = before + sum(nq) + tail, before + sum(nk) + tail
    q, k, v = qkv([Tq], [Tk], Hq, Hkv, D, seed=seed)
    cu = dict(cu_q=offsets_from(before, nq), cu_k=offsets_from(before, nk), causal=True)
    return q, k, v, rnd(Tq, Hq, D, seed=seed + 9), cu, (Tq, Tk, Hq, Hkv, D, len(nq))


def test_the_cases_are_shared():
    for c in CASES:
        Tq, Tk, Hq, Hkv, D, B = sizes = problem(c)[5]
        assert nv.nvfp4_attention_workspace_bytes(*sizes) > 0, c  # keys of queries, forward and for dq
        if c != CASES[1]:  # queries of keys
            assert nv.nvfp4_attention_backward_workspace_bytes(*sizes) >= 8 * Tq * Hq + 2 * 2 * 4 * Tk * Hkv * D, c


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    before, nq, nk, _, Hq, _, D = case
    q, k, v, _, cu, sizes = problem(case)
    a, b = before + sum(nq), before + sum(nk)
    out, lse = torch.full_like(q, 3.0), torch.full((Hq, q.shape[0]), 5.0, device=DEV)
    nv.nvfp4_attention(q, k, v, out=out, lse=lse, workspace=full_of_nan(nv.nvfp4_attention_workspace_bytes(*sizes)), **cu)
    check(out[before:a], lse[:, before:a], definition(q[before:a], k[before:b], v[before:b], nq, nk, True, D ** -0.5))
    for rows in (slice(0, before), slice(a, None)):
        assert bool((out[rows] == 3).all()) and bool((lse[:, rows] == 5).all())
    new, sums = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    assert torch.equal(new[before:a], out[before:a]) and torch.equal(sums[:, before:a], lse[:, before:a])
    for rows in (slice(0, before), slice(a, None)):
        assert bool((new[rows] == 0).all()) and bool((sums[:, rows] == -math.inf).all())


@pytest.mark.parametrize("case", CASES)
def test_gradients(case):
    before, nq, nk, _, Hq, _, D = case
    q, k, v, u, cu, sizes = problem(case)
    a, b = before + sum(nq), before + sum(nk)
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    given = [torch.full_like(t, 3.0) for t in (q, k, v)]
    ws = full_of_nan(nv.nvfp4_attention_backward_workspace_bytes(*sizes))
    nv.nvfp4_attention_backward(u, q, k, v, out, lse, dq=given[0], dk=given[1], dv=given[2], workspace=ws, **cu)
    want = gradients(u[before:a], q[before:a], k[before:b], v[before:b], nq, nk, True, D ** -0.5)
    check_gradients((given[0][before:a], given[1][before:b], given[2][before:b]), want)
    for t, end in zip(given, (a, b, b)):
        assert bool((t[:before] == 3).all()) and bool((t[end:] == 3).all())
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    for t, g, end in zip(given, torch.autograd.grad(nv.attention(*leaves, **cu), leaves, u), (a, b, b)):
        assert torch.equal(g[before:end], t[before:end]) and bool((g[:before] == 0).all()) and bool((g[end:] == 0).all())


def test_a_packed_batch_in_two_calls():
    """The second call's rows do not touch the first one's."""
    lens, Hq, Hkv, D = [300, 41, 700, 90], 4, 2, 64
    q, k, v = qkv(lens, lens, Hq, Hkv, D)
    u, cu, n = rnd(sum(lens), Hq, D, seed=9), offsets_from(0, lens), sum(lens)
    out, lse = torch.full_like(q, 3.0), torch.full((Hq, n), 5.0, device=DEV)
    grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
    sizes = (n, n, Hq, Hkv, D, 2)
    for part in (cu[:3], cu[2:]):
        how = dict(cu_q=part, cu_k=part, causal=True)
        nv.nvfp4_attention(q, k, v, out=out, lse=lse, workspace=full_of_nan(nv.nvfp4_attention_workspace_bytes(*sizes)), **how)
    for part in (cu[:3], cu[2:]):
        how = dict(cu_q=part, cu_k=part, causal=True)
        nv.nvfp4_attention_backward(u, q, k, v, out, lse, dq=grads[0], dk=grads[1], dv=grads[2],
                                    workspace=full_of_nan(nv.nvfp4_attention_backward_workspace_bytes(*sizes)), **how)
    check(out, lse, definition(q, k, v, lens, lens, True, D ** -0.5))
    check_gradients(grads, gradients(u, q, k, v, lens, lens, True, D ** -0.5))


@pytest.mark.parametrize("cu", [[0, 2900, 40, 3000], [500, 20, 2700], [2900, 100], [0, 5000, -3, 2 ** 31 - 1]])
def test_shared_blocks_of_offsets_that_descend_write_nothing(cu):
    """(The arrays lie between rows of other memory, which must not change either.)"""
    T, Hq, Hkv, D = 3000, 2, 1, 64
    c = ints(cu)
    sizes = (T, T, Hq, Hkv, D, len(cu) - 1)
    assert nv.nvfp4_attention_workspace_bytes(*sizes) > 0
    q, k, v = qkv([T], [T], Hq, Hkv, D)
    u, lse = rnd(T, Hq, D, seed=9), torch.full((Hq, T), 5.0, device=DEV)
    big = [torch.full((3 * T, h, D), 9.0, dtype=q.dtype, device=DEV) for h in (Hq, Hq, Hkv, Hkv)]
    out, dq, dk, dv = (t[T: 2 * T] for t in big)
    for _ in range(2):
        nv.nvfp4_attention(q, k, v, causal=True, cu_q=c, cu_k=c, out=out, lse=lse,
                           workspace=full_of_nan(nv.nvfp4_attention_workspace_bytes(*sizes)))
        nv.nvfp4_attention_backward(u, q, k, v, out, lse, causal=True, cu_q=c, cu_k=c, dq=dq, dk=dk, dv=dv,
                                    workspace=full_of_nan(nv.nvfp4_attention_backward_workspace_bytes(*sizes)))
    assert all(bool((t == 9).all()) for t in big) and bool((lse == 5).all())

"""Infinities in queries and keys.  A query whose every attended score is -inf has 0 / 0 for its weights: its output is NaN (its
log sum of exponentials is log 0 = -inf), and so is what its gradients reach.  One that attends nothing gives 0 as ever.  What
does not attend an infinity keeps its bits."""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import DEV, check, definition, offsets, qkv, rnd
from test_gpu_paged_attention import filled, values

pytestmark = pytest.mark.gpu


def lowest(q, k, at):
    """Query `at`'s score is -inf with every key: -inf in a place where all keys are above 0."""
    q, k = q.clone(), k.clone()
    k[:, :, 3] = k[:, :, 3].abs() + 1
    plain = q.clone()
    q[at, 0, 3] = -math.inf
    return plain, q, k


@pytest.mark.parametrize("n,m,D", [(200, 200, 64), (200, 200, 72), (130, 130, 128), (50, 3000, 64), (17, 4096, 128), (300, 1, 16)])
@pytest.mark.parametrize("causal", [False, True])
def test_all_scores_lowest(n, m, D, causal):
    q, k, v = qkv([n], [m], 2, 1, D)
    u, at = rnd(n, 2, D, seed=5), n - 1
    plain, q, k = lowest(q, k, at)
    want, wl = nv.nvfp4_attention(plain, k, v, causal=causal, save_lse=True)
    out, lse = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True)
    check(want, wl, definition(plain, k, v, [n], [m], causal, D ** -0.5))
    assert bool(out[at, 0].isnan().all()) and float(lse[0, at]) == -math.inf
    same = torch.ones(n, 2, dtype=torch.bool, device=DEV)
    same[at, 0] = False
    assert torch.equal(out[same], want[same]) and torch.equal(lse.t()[same], wl.t()[same])
    dq, dk, dv = nv.nvfp4_attention_backward(u, q, k, v, out, lse, causal=causal)
    wq, _, _ = nv.nvfp4_attention_backward(u, plain, k, v, want, wl, causal=causal)
    assert bool(dq[at, 0].isnan().all()) and torch.equal(dq[same], wq[same])
    assert bool(dk.isnan().all()) and bool(dv.isnan().all())  # the last query attends all keys


@pytest.mark.parametrize("D", [64, 128])
def test_a_lowest_key(D):
    """Key 0 is -inf for queries above 0: the one that attends it alone is NaN, for the others its weight is 0."""
    n = 150
    q, k, v = qkv([n], [n], 2, 2, D)
    q[:, :, 3] = q[:, :, 3].abs() + 1
    k[0, :, 3] = -math.inf
    out, lse = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True)
    assert bool(out[0].isnan().all()) and bool((lse[:, 0] == -math.inf).all())
    want = definition(q[1:], k[1:], v[1:], [n - 1], [n - 1], True, D ** -0.5)
    check(out[1:], lse[:, 1:], want)


def test_queries_without_keys_beside_queries_of_lowest_scores():
    """Causal, more queries than keys: the first ones attend nothing, whatever they hold."""
    nq, nk, D = [100, 40], [30, 0], 64
    q, k, v = qkv(nq, nk, 2, 1, D)
    k[:, :, 3] = k[:, :, 3].abs() + 1
    q[5, :, 3] = q[80, :, 3] = q[110, :, 3] = -math.inf
    out, lse = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True, cu_q=offsets(nq), cu_k=offsets(nk))
    assert bool((out[:70] == 0).all()) and bool((out[100:] == 0).all()) and bool((lse[:, :70] == -math.inf).all())
    assert bool(out[80].isnan().all()) and bool(torch.isfinite(out[70:80]).all()) and bool(torch.isfinite(out[81:100]).all())
    assert bool((lse[:, 80] == -math.inf).all())


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("lens,D", [([100, 33], 64), ([1, 16], 128), ([3000, 700], 72), ([1300, 5], 128)])
@pytest.mark.parametrize("Hq", [2, 40])
def test_single_tokens(mx8, lens, D, Hq):
    cache, table, lengths = filled(lens, 16, 2, D, mx8)
    (cache.k[..., 3].fill_(0x38) if mx8 else cache.k[..., 3].fill_(1.0))  # 1, times the block's scale: above 0 in all keys
    q = rnd(2, Hq, D, seed=5)
    want = nv.nvfp4_paged_attention(q, cache, table, lengths)
    keys, vals = values(cache, table, lens, D)
    check(want, None, definition(q, keys, vals, [1, 1], lens, False, D ** -0.5))
    low = q.clone()
    low[0, Hq - 1, 3] = -math.inf
    out = nv.nvfp4_paged_attention(low, cache, table, lengths)
    assert bool(out[0, Hq - 1].isnan().all())
    assert torch.equal(out[1], want[1]) and torch.equal(out[0, : Hq - 1], want[0, : Hq - 1])
    none = nv.nvfp4_paged_attention(low, cache, torch.full_like(table, -1), lengths)  # no page: no tokens
    assert bool((none == 0).all())
    assert bool((nv.nvfp4_paged_attention(low, cache, table, torch.zeros_like(lengths)) == 0).all())


@pytest.mark.parametrize("lens", [[40], [2000]])
def test_single_tokens_over_a_lowest_key(lens):
    """The one token's key is -inf: NaN; a longer sequence only leaves it out."""
    D = 64
    cache, table, lengths = filled(lens, 16, 1, D, False)
    cache.k[..., 3].fill_(1.0)
    q = rnd(1, 3, D, seed=5).abs()
    first = int(table[0, 0])
    cache.k[first, 0, 0, 3] = -math.inf
    one = torch.ones_like(lengths)
    assert bool(nv.nvfp4_paged_attention(q, cache, table, one).isnan().all())
    keys, vals = values(cache, table, lens, D)
    out = nv.nvfp4_paged_attention(q, cache, table, lengths)
    check(out, None, definition(q, keys[1:], vals[1:], [1], [lens[0] - 1], False, D ** -0.5))

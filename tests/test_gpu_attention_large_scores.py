"""Scores so large that an exponent's product with the scale leaves fp32's digits behind.  A single place of a head is not 0, so
that scores are exact in fp32, and the largest ones are equal or lie far above the others: the weights are 1 / n for the n
largest and 0 (below 2^-1000) else, and nothing but the outputs' rounding and the sums' (2^-8 |o| + 2^-8 A, see
test_gpu_attention.py) is off."""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import BF, DEV, HALF, offsets, rnd
from test_gpu_paged_attention import filled, values

pytestmark = pytest.mark.gpu

# |score| is 2^e .. 2^(e + 1), neighbours 2^(e - 7) apart (fp32's largest is 2^128); times the scale
SIZES = [(18, 1.0), (20, 1.0), (24, 1.0), (28, 1.0), (31, 0.7), (32, 1.0), (40, 0.125), (100, 1.0), (120, 0.3), (90, 2.0 ** 20),
         (100, 2.0 ** 60)]


def steps(n):
    return (1 + torch.arange(n, device=DEV) % 128 / 128).to(BF)


def problem(nq, nk, H, D, e, sign, at=3):
    """Queries of sign * 2^(e / 2), keys of 2^(e - e / 2) (1 .. 2 in 128 steps, over and over)."""
    q, k = torch.zeros(nq, H, D, dtype=BF, device=DEV), torch.zeros(nk, H, D, dtype=BF, device=DEV)
    q[:, :, at] = sign * 2.0 ** (e // 2)
    k[:, :, at] = (steps(nk) * 2.0 ** (e - e // 2))[:, None]
    return q, k


def wanted(q, k, v, causal, scale, at=3):
    """(out, A, largest score) in 64 bits from the exact scores, query by query [nq, H, ..]."""
    s = q[:, None, :, at].double() * k[None, :, :, at].double()
    nq, nk = s.shape[:2]
    if causal:
        i, j = torch.arange(nq, device=DEV)[:, None], torch.arange(nk, device=DEV)[None]
        s = torch.where((j - i <= nk - nq)[..., None], s, -math.inf)
    top = s.amax(1, keepdim=True)
    p = torch.exp((s - top) * scale)
    n = p.sum(1, keepdim=True)
    p = p / n
    out, A = (torch.stack([p[:, :, h] @ x[:, h] for h in range(q.shape[1])], 1) for x in (v.double(), v.double().abs()))
    return out, A, top[:, 0] * scale + n[:, 0].log()


def close(out, want, A):
    err, tol = (out.double() - want).abs(), HALF * (A + want.abs()) + 2.0 ** -15 * A
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("e,scale", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("nq,nk,D,causal", [(150, 150, 64, True), (150, 300, 72, False), (40, 70, 128, True), (17, 4096, 64, False),
                                            (33, 3000, 128, True)])
def test_attention(e, scale, sign, nq, nk, D, causal):
    q, k = problem(nq, nk, 2, D, e, sign)
    v = rnd(nk, 2, D, seed=2)
    out, lse = nv.nvfp4_attention(q, k, v, causal=causal, scale=scale, save_lse=True)
    want, A, sums = wanted(q, k, v, causal, scale)
    close(out, want, A)
    fits = sums.abs() < 2.0 ** 127
    assert bool(((lse.t().double() - sums)[fits].abs() <= 2.0 ** -21 * sums[fits].abs() + 2.0 ** -20).all())


def test_neighbours_keep_their_bits():
    """Queries of ordinary scores beside others of large ones, in one tile and in one sequence's shared blocks."""
    for nq, nk in ((100, 300), (20, 5000)):
        q, k = problem(nq, nk, 2, 64, 40, 1)
        k[:, :, 8:] = rnd(nk, 2, 56, seed=3)
        v, plain = rnd(nk, 2, 64, seed=2), q.clone()
        plain[:, :, 3] = 0
        plain[:, :, 8:] = rnd(nq, 2, 56, seed=4)
        mixed = plain.clone()
        mixed[::3, :, 3] = q[::3, :, 3]
        want, wl = nv.nvfp4_attention(plain, k, v, causal=True, save_lse=True)
        out, lse = nv.nvfp4_attention(mixed, k, v, causal=True, save_lse=True)
        rest = torch.arange(nq, device=DEV) % 3 != 0
        assert torch.equal(out[rest], want[rest]) and torch.equal(lse[:, rest], wl[:, rest])
        assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("e,scale", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,Hq", [(100, 2), (4096, 2), (3000, 40)])
def test_single_tokens(e, scale, sign, n, Hq):
    D, page = 64, 16
    cache, table, lengths = filled([n], page, 1, D, False)
    pages = table[0, : -(-n // page)].long()
    rows = torch.zeros(len(pages) * page, D, dtype=BF, device=DEV)
    rows[:, 3] = steps(len(pages) * page) * 2.0 ** (e - e // 2)
    cache.k[pages, 0] = rows.view(len(pages), page, D)
    q = torch.zeros(1, Hq, D, dtype=BF, device=DEV)
    q[..., 3] = sign * 2.0 ** (e // 2)
    out = nv.nvfp4_paged_attention(q, cache, table, lengths, scale=scale)
    k, v = values(cache, table, [n], D)
    want, A, _ = wanted(q[:, :1], k, v, False, scale)
    close(out, want.expand(1, Hq, D), A.expand(1, Hq, D))


def test_single_tokens_keep_their_bits_beside_large_scores():
    D = 64
    cache, table, lengths = filled([2000], 16, 1, D, True)
    q = rnd(1, 8, D, seed=4)
    want = nv.nvfp4_paged_attention(q, cache, table, lengths)
    large = q.clone()
    large[0, 5] *= 2.0 ** 40
    out = nv.nvfp4_paged_attention(large, cache, table, lengths)
    rest = torch.arange(8, device=DEV) != 5
    assert torch.equal(out[0, rest], want[0, rest]) and bool(torch.isfinite(out).all())


def test_a_key_of_the_lowest_value():
    """A key filled with the type's lowest value stands for one that is left out: where its scores are below all others it is,
    and where they are above it has all the weight."""
    n, D = 100, 64
    q, k, v = rnd(n, 2, D, seed=0), rnd(n, 2, D, seed=1), rnd(n, 2, D, seed=2)
    q[:, :, 1:] *= 2.0 ** -10  # the sum of a query's values has the sign of the first, and its score stays finite
    q[:, :, 0] = torch.where(q[:, :, 0] >= 0, 0.25, -0.25)
    k[0] = torch.finfo(BF).min
    out, lse = nv.nvfp4_attention(q, k, v)
    up = (q.double().sum(2) < 0)
    assert bool(up.any()) and not bool(up.all())
    assert torch.equal(out[up], v[:1].expand(n, 2, D)[up])
    less, _ = nv.nvfp4_attention(q, k[1:], v[1:])  # both off by 2^-8 (A + |o|), each at most the largest value
    err = (out.double() - less.double()).abs()[~up]
    assert bool((err <= 2.0 ** -6 * v.abs().max()).all()) and bool(torch.isfinite(out).all())

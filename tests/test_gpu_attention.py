"""Attention of whole sequences (nvfp4_attention) against its definition in 64 bits.

Tolerances, per element, with A = sum_j p_ij |v_j| of the row (p the softmax):
  out   the exponentials are rounded to bf16, 2^-8 of each at most, and so is the result: 2^-8 (A + |o|).  What fp32 adds:
        a score's products are exact, its sum of D terms is off by (D + 2) 2^-24 sum |q k| scale at most; the exponent's
        multiply-add, 2^x and the sum of exponentials by another 2^-20.  Together E (below), relative to A, twice (numerator
        and denominator).
  lse   E, and the sum's logarithm, 2^-21 of the value.
"""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
HALF = 2.0 ** -8  # half a step of bf16


def rnd(*shape, seed, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(BF).to(DEV)


def offsets(lens):
    return torch.tensor([0] + list(lens), device=DEV).cumsum(0).int()


def qkv(nq, nk, Hq, Hkv, D, seed=0, tail=0, scale=1.0):
    return (rnd(sum(nq) + tail, Hq, D, seed=seed, scale=scale), rnd(sum(nk) + tail, Hkv, D, seed=seed + 1, scale=scale),
            rnd(sum(nk) + tail, Hkv, D, seed=seed + 2))


def sees(m, n, causal):
    i, j = torch.arange(m, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
    return (j - i <= n - m) if causal else torch.ones(m, n, dtype=torch.bool, device=DEV)


def definition(q, k, v, nq, nk, causal, scale):
    """(out, lse [Tq, Hq], A, E) in 64 bits."""
    Tq, Hq, D = q.shape
    group = Hq // k.shape[1]
    out = torch.zeros(Tq, Hq, D, dtype=torch.float64, device=DEV)
    A, lse = out.clone(), torch.full((Tq, Hq), -math.inf, dtype=torch.float64, device=DEV)
    E, a, b = 0.0, 0, 0
    for m, n in zip(nq, nk):
        if m and n:
            mask = sees(m, n, causal)
            some = mask.any(1)
            for h in range(Hq):
                Q, K, V = q[a: a + m, h].double(), k[b: b + n, h // group].double(), v[b: b + n, h // group].double()
                s = torch.where(mask, Q @ K.t() * scale, -math.inf)
                E = max(E, float((Q.abs() @ K.abs().t()).max()) * scale * (D + 2) * 2.0 ** -24)
                l = torch.logsumexp(torch.where(some[:, None], s, 0.0), 1)
                p = torch.where(mask, torch.exp(s - l[:, None]), 0.0)
                out[a: a + m, h], A[a: a + m, h] = p @ V, p @ V.abs()
                lse[a: a + m, h] = torch.where(some, l, -math.inf)
        a, b = a + m, b + n
    return out, lse, A, E + 2.0 ** -20


def check(out, lse, want, rows=None):
    o, l, A, E = want
    rows = o.shape[0] if rows is None else rows
    err = (out[:rows].double() - o[:rows]).abs()
    tol = HALF * (A + o.abs()) + (2 * E + HALF * HALF) * A + 1e-37
    assert bool((err <= tol[:rows]).all()), float((err / tol[:rows]).max())
    if lse is not None:
        got, l = lse.t()[:rows].double(), l[:rows]
        assert torch.equal(got == -math.inf, l == -math.inf)
        fine = l > -math.inf
        assert bool(((got - l)[fine].abs() <= E + 2.0 ** -21 * (1 + l[fine].abs())).all())


def run(nq, nk, Hq, Hkv, D, causal, packed=True, seed=0, scale=None, size=1.0):
    q, k, v = qkv(nq, nk, Hq, Hkv, D, seed=seed, scale=size)
    cu = dict(cu_q=offsets(nq), cu_k=offsets(nk)) if packed else dict(batch=len(nq))
    out, lse = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True, scale=scale, **cu)
    check(out, lse, definition(q, k, v, nq, nk, causal, D ** -0.5 if scale is None else scale))


@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 72, 80, 88, 96, 104, 112, 120, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_head_sizes(D, causal):
    run([77, 200], [130, 200], 3, 1, D, causal, seed=D)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1003])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(n, causal):
    run([n], [n], 2, 2, 64, causal, packed=False, seed=n)


@pytest.mark.parametrize("m,n", [(1, 1), (1, 300), (300, 1), (5, 1000), (1000, 5), (64, 65), (130, 64), (200, 0), (3, 4097)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [72, 128])
def test_queries_and_keys_of_different_numbers(m, n, causal, D):
    """Causal with more queries than keys: the first ones attend nothing."""
    run([m], [n], 4, 2, D, causal, packed=m > 100, seed=m + n)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 1), (12, 4), (24, 3), (5, 5), (16, 8)])
@pytest.mark.parametrize("causal", [False, True])
def test_grouped_heads(Hq, Hkv, causal):
    run([100, 0, 1, 333], [100, 7, 1, 400], Hq, Hkv, 80, causal, seed=Hq)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1] * 70, [0, 5, 0, 0, 64, 0, 1, 129, 0], list(range(200)), [3] * 5000])
def test_packed_lengths(lens):
    run(lens, lens, 1, 1, 16, True, seed=len(lens))


def test_equal_batches_are_the_same_as_packed_ones():
    q, k, v = qkv([77] * 5, [130] * 5, 4, 2, 72)
    for causal in (False, True):
        a = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True, batch=5)
        b = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True, cu_q=offsets([77] * 5), cu_k=offsets([130] * 5))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("size,scale", [(1.0, 0.001), (1.0, 1.0), (6.0, 0.3), (0.01, 100.0), (30.0, 0.01)])
def test_scales(size, scale):
    """Flat and peaked softmaxes (the sharpest have all weight on a key), maxima that rise late."""
    run([150], [500], 2, 1, 64, True, seed=3, scale=scale, size=size)


def test_a_maximum_that_rises_in_every_tile():
    n, D = 1000, 64
    q, v = rnd(64, 1, D, seed=1).abs(), rnd(n, 1, D, seed=2)
    k = (torch.arange(n, device=DEV)[:, None, None] / 40 * torch.ones(1, 1, D, device=DEV)).to(BF)
    for keys, vals in ((k, v), (k.flip(0).contiguous(), v)):
        out, lse = nv.nvfp4_attention(q, keys, vals, save_lse=True)
        check(out, lse, definition(q, keys, vals, [64], [n], False, D ** -0.5))


def test_views_of_a_qkv_output_and_other_pitches():
    T, H, D = 150, 4, 72
    rows = rnd(T, 3 * H + 2, D, seed=1)
    q, k, v = rows[:, :H], rows[:, H: 2 * H], rows[:, 2 * H: 3 * H]
    want = nv.nvfp4_attention(q.contiguous(), k.contiguous(), v.contiguous(), causal=True, save_lse=True)
    got = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]  # heads outermost
    out = torch.full((H, T, D), 7.0, dtype=BF, device=DEV).transpose(0, 1)
    got = nv.nvfp4_attention(*first, causal=True, out=out)
    assert got[0] is out and torch.equal(out, want[0])
    same = q.clone()
    assert torch.equal(nv.nvfp4_attention(same, k, v, causal=True, out=same)[0], want[0]) and torch.equal(same, want[0])
    # one key and one value head in the place of all
    k1, v1 = k[:, :1].expand(T, H, D), v[:, :1].expand(T, H, D)
    a = nv.nvfp4_attention(q, k1, v1)[0]
    assert torch.equal(a, nv.nvfp4_attention(q, k1.contiguous(), v1.contiguous())[0])


@pytest.mark.parametrize("tail", [1, 40, 300])
def test_rows_behind_the_last_sequence_are_left(tail):
    nq, nk = [33, 100], [64, 50]
    q, k, v = qkv(nq, nk, 4, 2, 64, tail=tail)
    for t in (q, k, v):
        t[-tail:] = math.nan
    out, lse = torch.full_like(q, 3.0), torch.full((4, sum(nq) + tail), 5.0, device=DEV)
    want = definition(q[: sum(nq)], k[: sum(nk)], v[: sum(nk)], nq, nk, True, 0.125)
    cu = dict(cu_q=offsets(nq), cu_k=offsets(nk))
    nv.nvfp4_attention(q, k, v, causal=True, out=out, lse=lse, **cu)
    check(out, lse, want, sum(nq))
    assert bool((out[sum(nq):] == 3).all()) and bool((lse[:, sum(nq):] == 5).all())
    new, sums = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True, **cu)
    assert torch.equal(new[: sum(nq)], out[: sum(nq)]) and bool((new[sum(nq):] == 0).all())
    assert bool((sums[:, sum(nq):] == -math.inf).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("at", [0, 40, 63, 64, 130, 199])
def test_values_that_are_not_finite_reach_only_who_attends_them(bad, D, at):
    n = 200
    q, k, v = qkv([n, 50], [n, 50], 2, 1, D)
    cu = dict(cu_q=offsets([n, 50]), cu_k=offsets([n, 50]))
    want, wl = nv.nvfp4_attention(q, k, v, causal=True, save_lse=True, **cu)
    v2 = v.clone()
    v2[at, 0, 3] = bad
    got, gl = nv.nvfp4_attention(q, k, v2, causal=True, save_lse=True, **cu)
    assert torch.equal(gl, wl)
    assert torch.equal(got[:at], want[:at]) and torch.equal(got[n:], want[n:])
    assert not bool(torch.isfinite(got[at:n, :, 3]).any())
    assert torch.equal(torch.cat([got[..., :3], got[..., 4:]], 2), torch.cat([want[..., :3], want[..., 4:]], 2))
    k2 = k.clone()
    k2[at, 0, 3] = math.nan
    got, gl = nv.nvfp4_attention(q, k2, v, causal=True, save_lse=True, **cu)
    assert torch.equal(got[:at], want[:at]) and torch.equal(got[n:], want[n:]) and bool(got[at:n].isnan().all())
    assert torch.equal(gl[:, :at], wl[:, :at]) and bool(gl[:, at:n].isnan().all())
    q2 = q.clone()
    q2[at, 1, 5] = math.nan
    got, _ = nv.nvfp4_attention(q2, k, v, causal=True, **cu)
    assert bool(got[at, 1].isnan().all())
    got[at, 1] = want[at, 1]
    assert torch.equal(got, want)


def test_long_sequences_past_32_bits_of_bytes():
    """Rows 2^21 elements apart: the last lie 4 GiB from the first."""
    T, D = 1100, 64
    wide = torch.zeros(T, 1 << 21, dtype=BF, device=DEV)
    q, k, v = (rnd(T, 1, D, seed=i) for i in range(3))
    views = []
    for i, t in enumerate((q, k, v)):
        views.append(wide[:, 64 * i: 64 * i + 64].unsqueeze(1))
        views[-1].copy_(t)
    assert torch.equal(nv.nvfp4_attention(*views, causal=True)[0], nv.nvfp4_attention(q, k, v, causal=True)[0])


@pytest.mark.parametrize("cu", [[0, 5000], [-3, 100], [50, 20], [0, 90, 40, 100], [7, 7, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1]])
def test_offsets_that_say_nothing_sensible_stay_inside_the_arrays(cu):
    """The arrays lie between rows of other memory, which must not change."""
    T = 100
    c = torch.tensor(cu, dtype=torch.int64).to(torch.int32).to(DEV)
    big = torch.full((3 * T, 2, 64), 9.0, dtype=BF, device=DEV)
    q, k, v = qkv([T], [T], 2, 2, 64)
    nv.nvfp4_attention(q, k, v, causal=True, cu_q=c, cu_k=c, out=big[T: 2 * T])
    assert bool((big[:T] == 9).all()) and bool((big[2 * T:] == 9).all())
    inside = big[T: 2 * T]
    assert bool(torch.isfinite(inside).all())

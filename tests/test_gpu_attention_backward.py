"""Gradients of attention (nvfp4_attention_backward, attention) against the formulas in 64 bits, against differences of the
64-bit definition, and under autograd.

Tolerances, per element.  P and dS are rounded to bf16 before their products and each gradient once more: 2^-8 each of
sum |p dout|, scale sum |ds k|, scale sum |ds q|, and of the value.  dS itself is off by what its inputs are: delta is
formed with the bf16 out, off by 2^-8 |o| + 2^-8 A in each element, so delta by 2^-8 sum_d |dout| (|o| + A) (A = sum_j p |v|
of the row), and dP and P by fp32's sums, (D + 2) 2^-24 of sum |dout v| and E (of the scores) relative: ds is off by
p (d_delta + E' (sum |dout v| + |delta|)).  Those enter dq and dk through p |k| and p |q|.  Below fp32's and bf16's least
normal number, 2^-126, P and dS may become 0: P is off by 2^-126 more, and dS by that times its factor and by 2^-126 itself
(at scores of hundreds whole keys have only such weights: dk of 1.6e-37 in place of 0 there)."""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import BF, DEV, HALF, definition, offsets, qkv, rnd, sees

pytestmark = pytest.mark.gpu


def gradients(dout, q, k, v, nq, nk, causal, scale):
    """((value, tolerance) of dq, dk, dv) in 64 bits."""
    Tq, Hq, D = q.shape
    group = Hq // k.shape[1]
    o, l, A, E = definition(q, k, v, nq, nk, causal, scale)
    new = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=DEV)  # noqa: E731
    dq, dk, dv, tq, tk, tv = new(q), new(k), new(k), new(q), new(k), new(k)
    a = b = 0
    for m, n in zip(nq, nk):
        if m and n:
            mask = sees(m, n, causal)
            for h in range(Hq):
                i, j = slice(a, a + m), slice(b, b + n)
                Q, K, V, dO = q[i, h].double(), k[j, h // group].double(), v[j, h // group].double(), dout[i, h].double()
                lse = torch.where(l[i, h] == -math.inf, 0.0, l[i, h])
                p = torch.where(mask, torch.exp(Q @ K.t() * scale - lse[:, None]), 0.0)
                dP, delta = dO @ V.t(), (dO * o[i, h]).sum(1, keepdim=True)
                ds = p * (dP - delta)
                size = dO.abs() @ V.abs().t() + (dO * o[i, h]).abs().sum(1, keepdim=True)
                off = HALF * (dO.abs() * (o[i, h].abs() + A[i, h])).sum(1, keepdim=True)
                off = p * (off + ((D + 2) * 2.0 ** -24 + 3 * E) * size)
                dq[i, h] += scale * ds @ K
                dk[j, h // group] += scale * ds.t() @ Q
                dv[j, h // group] += p.t() @ dO
                tiny = mask * 2.0 ** -126
                r = off + HALF * 1.01 * ds.abs() + tiny * (size + 1)
                tq[i, h] += scale * r @ K.abs()
                tk[j, h // group] += scale * r.t() @ Q.abs()
                tv[j, h // group] += ((HALF * 1.01 + 3 * E) * p + tiny).t() @ dO.abs()
        a, b = a + m, b + n
    return [(x, t * 1.01 + HALF * x.abs() + 1e-37) for x, t in ((dq, tq), (dk, tk), (dv, tv))]


def check(got, want, names=("dq", "dk", "dv")):
    for g, (x, tol), name in zip(got, want, names):
        err = (g.double() - x).abs()
        assert bool((err <= tol).all()), (name, float((err / tol).max()))


def run(nq, nk, Hq, Hkv, D, causal, packed=True, seed=0, scale=None, size=1.0):
    q, k, v = qkv(nq, nk, Hq, Hkv, D, seed=seed, scale=size)
    dout = rnd(sum(nq), Hq, D, seed=seed + 7)
    cu = dict(cu_q=offsets(nq), cu_k=offsets(nk)) if packed else dict(batch=len(nq))
    out, lse = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True, scale=scale, **cu)
    got = nv.nvfp4_attention_backward(dout, q, k, v, out, lse, causal=causal, scale=scale, **cu)
    check(got, gradients(dout, q, k, v, nq, nk, causal, D ** -0.5 if scale is None else scale))
    again = nv.nvfp4_attention_backward(dout, q, k, v, out, lse, causal=causal, scale=scale, **cu)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 72, 80, 88, 96, 104, 112, 120, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_head_sizes(D, causal):
    run([77, 200], [130, 200], 3, 1, D, causal, seed=D)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1003])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(n, causal):
    run([n], [n], 2, 2, 64, causal, packed=False, seed=n)


@pytest.mark.parametrize("m,n", [(1, 1), (1, 300), (300, 1), (5, 1000), (1000, 5), (64, 65), (130, 64), (200, 0), (0, 200),
                                 (3, 2049)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [72, 128])
def test_queries_and_keys_of_different_numbers(m, n, causal, D):
    run([m], [n], 4, 2, D, causal, packed=m > 100, seed=m + n)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 1), (12, 4), (24, 3), (5, 5), (16, 8)])
@pytest.mark.parametrize("causal", [False, True])
def test_grouped_heads(Hq, Hkv, causal):
    run([100, 0, 1, 333], [100, 7, 1, 400], Hq, Hkv, 80, causal, seed=Hq)


@pytest.mark.parametrize("lens", [[0], [1] * 70, [0, 5, 0, 0, 64, 0, 1, 129, 0], list(range(150))])
def test_packed_lengths(lens):
    run(lens, lens, 1, 1, 16, True, seed=len(lens))


@pytest.mark.parametrize("size,scale", [(1.0, 0.001), (1.0, 1.0), (6.0, 0.3)])
def test_scales(size, scale):
    run([150], [500], 2, 1, 64, True, seed=3, scale=scale, size=size)


@pytest.mark.parametrize("tail", [1, 200])
def test_rows_behind_the_last_sequence_are_left(tail):
    nq, nk = [33, 100], [64, 50]
    q, k, v = qkv(nq, nk, 4, 2, 64, tail=tail)
    dout = rnd(sum(nq) + tail, 4, 64, seed=9)
    for t in (q, k, v, dout):
        t[-tail:] = math.nan
    cu = dict(cu_q=offsets(nq), cu_k=offsets(nk), causal=True)
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    given = [torch.full_like(t, 3.0) for t in (q, k, v)]
    nv.nvfp4_attention_backward(dout, q, k, v, out, lse, dq=given[0], dk=given[1], dv=given[2], **cu)
    a, b = sum(nq), sum(nk)
    want = gradients(dout[:a], q[:a], k[:b], v[:b], nq, nk, True, 0.125)
    check((given[0][:a], given[1][:b], given[2][:b]), want)
    assert all(bool((t[-tail:] == 3).all()) for t in given)
    new = nv.nvfp4_attention_backward(dout, q, k, v, out, lse, **cu)
    for x, y in zip(new, given):
        assert torch.equal(x[:-tail], y[:-tail]) and bool((x[-tail:] == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("at", [0, 40, 63, 64, 130, 199])
def test_values_that_are_not_finite_reach_only_what_they_touch(bad, D, at):
    """Causal: query `at` touches keys up to `at`; key `at` touches queries from `at` on (and through them all keys)."""
    n = 200
    q, k, v = qkv([n, 50], [n, 50], 2, 1, D)
    dout = rnd(n + 50, 2, D, seed=5)
    cu = dict(cu_q=offsets([n, 50]), cu_k=offsets([n, 50]), causal=True)
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    want = nv.nvfp4_attention_backward(dout, q, k, v, out, lse, **cu)
    d2 = dout.clone()
    d2[at, 1, 3] = bad
    dq, dk, dv = nv.nvfp4_attention_backward(d2, q, k, v, out, lse, **cu)
    assert torch.equal(dk[at + 1:], want[1][at + 1:]) and torch.equal(dv[at + 1:], want[2][at + 1:])
    assert not bool(torch.isfinite(dv[: at + 1, 0, 3]).any())
    assert torch.equal(dv[..., :3], want[2][..., :3]) and torch.equal(dv[..., 4:], want[2][..., 4:])
    rows = torch.arange(n + 50, device=DEV) != at
    assert torch.equal(dq[rows], want[0][rows]) and torch.equal(dq[at, 0], want[0][at, 0])
    k2 = k.clone()
    k2[at, 0, 3] = bad
    o2, l2 = nv.nvfp4_attention(q, k2, v, save_lse=True, **cu)
    dq, dk, dv = nv.nvfp4_attention_backward(dout, q, k2, v, o2, l2, **cu)
    assert torch.equal(dq[:at], want[0][:at]) and torch.equal(dq[n:], want[0][n:])
    assert torch.equal(dk[n:], want[1][n:]) and torch.equal(dv[n:], want[2][n:])
    q2 = q.clone()
    q2[at, 0, 3] = bad
    o2, l2 = nv.nvfp4_attention(q2, k, v, save_lse=True, **cu)
    dq, dk, dv = nv.nvfp4_attention_backward(dout, q2, k, v, o2, l2, **cu)
    assert torch.equal(dk[at + 1:], want[1][at + 1:]) and torch.equal(dv[at + 1:], want[2][at + 1:])
    assert torch.equal(dq[rows], want[0][rows]) and torch.equal(dq[at, 1], want[0][at, 1])


def test_differences_of_the_definition():
    """Along random directions, central differences of the 64-bit definition; the gradients' own rounding, 2^-7 of the sum of
    products' magnitudes at the most, is the bar."""
    nq, nk, Hq, Hkv, D = [37, 64], [50, 64], 4, 2, 40
    q, k, v = qkv(nq, nk, Hq, Hkv, D)
    u = rnd(sum(nq), Hq, D, seed=5)
    cu = dict(cu_q=offsets(nq), cu_k=offsets(nk), causal=True)
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    grads = nv.nvfp4_attention_backward(u, q, k, v, out, lse, **cu)
    at = [t.double() for t in (q, k, v)]
    f = lambda *x: float((definition(*x, nq, nk, True, D ** -0.5)[0] * u.double()).sum())  # noqa: E731
    want = gradients(u, q, k, v, nq, nk, True, D ** -0.5)
    for n in range(3):
        g = torch.Generator().manual_seed(n)
        d = torch.randn(at[n].shape, generator=g, dtype=torch.float64).to(DEV)
        step = 1e-4
        plus, minus = list(at), list(at)
        plus[n], minus[n] = at[n] + step * d, at[n] - step * d
        slope = (f(*plus) - f(*minus)) / (2 * step)
        got = float((grads[n].double() * d).sum())
        assert abs(got - slope) <= float((want[n][1] * d.abs()).sum()) + 1e-5 * abs(slope)


def off16(t):
    big = torch.empty(t.numel() + 3, dtype=t.dtype, device=t.device)
    big[3:] = t.flatten()
    return big[3:].view(t.shape)


FORMS = {"dense": lambda t: t, "expanded heads": lambda t: t[:, :1].expand(t.shape), "off 16 bytes": off16,
         "expanded tokens": lambda t: t[:1].expand(t.shape), "heads first": lambda t: t.transpose(0, 1).contiguous().transpose(0, 1),
         "strided": lambda t: t.repeat_interleave(2, 2)[..., ::2]}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 4), (70, 4)])
def test_autograd_takes_tensors_as_they_come(form, T, H):
    D = 72
    q, k, v, u = (FORMS[form](rnd(T, H, D, seed=i)) for i in range(4))
    leaves = [t.detach().requires_grad_() for t in (q, k, v)]
    out = nv.attention(*leaves, causal=True)
    dense = [t.clone(memory_format=torch.contiguous_format) for t in (q, k, v, u)]
    want, lse = nv.nvfp4_attention(*dense[:3], causal=True, save_lse=True)
    assert torch.equal(out, want)
    grads = nv.nvfp4_attention_backward(dense[3], *dense[:3], want, lse, causal=True)
    for a, b in zip(torch.autograd.grad(out, leaves, u), grads):
        assert torch.equal(a, b)


def test_autograd_through_a_qkv_output_with_padding():
    """One leaf in three places, a sum over tokens behind it (an expanded gradient), rows past the last sequence."""
    nq, H, D = [30, 41], 2, 64
    rows = rnd(sum(nq) + 5, 3 * H, D, seed=1).requires_grad_()
    cu = offsets(nq)
    out = nv.attention(*rows.split(H, 1), causal=True, cu_q=cu, cu_k=cu)
    g, = torch.autograd.grad(out.sum(), rows)
    q, k, v = rows.detach().split(H, 1)
    n = sum(nq)
    want = gradients(torch.ones(n, H, D, dtype=BF, device=DEV), q[:n], k[:n], v[:n], nq, nq, True, 0.125)
    check(g[:n].split(H, 1), want)
    assert bool((g[n:] == 0).all()) and bool((out[n:] == 0).all())


def test_written_tensors_and_saved_ones():
    q, k, v = (t.requires_grad_() for t in qkv([20], [20], 2, 2, 64))
    with pytest.raises(ValueError):
        nv.nvfp4_attention(q, k, v, out=q)
    out = nv.attention(q, k, v)
    with torch.no_grad():
        k.mul_(2)
    with pytest.raises(RuntimeError):
        out.sum().backward()
    x = torch.zeros(20, 2, 64, dtype=BF, device=DEV)
    y = nv.attention(q, k, v) * x  # x is saved
    nv.nvfp4_attention(q.detach(), k.detach(), v.detach(), out=x)
    with pytest.raises(RuntimeError):
        y.sum().backward()

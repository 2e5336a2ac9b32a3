"""The paged cache: appending (bit for bit) and the attention of one new token, against the definition in 64 bits over the
values that the cache holds.  Tolerances: those of test_gpu_attention.py; joining the splits adds roundings of fp32 that
its 2^-20 holds."""
import math

import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import BF, DEV, check, definition, offsets, qkv, rnd

pytestmark = pytest.mark.gpu
U8, I32 = torch.uint8, torch.int32


def tables(lens, page, seed=0, spare=2, extra=1):
    """(pages, page table with -1 where a sequence has no page, lengths)."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(lens), max(need + [0]) + extra), -1, dtype=I32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    return pages, table.to(DEV), torch.tensor(lens, dtype=I32, device=DEV)


def new_cache(pages, page, Hkv, D, mx8, fill=0xAB):
    cache = nv.paged_cache(pages, page, Hkv, D, mx8=mx8)
    for t in cache:
        if t is not None:
            t.view(U8).fill_(fill)
    return cache


def quantized(x):
    """nvfp4_mx8_quantize of rows of D values, padded to whole blocks: (codes, scales)."""
    D, blocks = x.shape[-1], -(-x.shape[-1] // 32)
    wide = torch.zeros(*x.shape[:-1], 32 * blocks, dtype=BF, device=DEV)
    wide[..., :D] = x
    codes, scales = nv.nvfp4_mx8_quantize(wide.view(-1, 32 * blocks))
    return codes.view(*x.shape[:-1], -1)[..., :D], scales.view(*x.shape[:-1], -1)


def place(cache, k, v, where, at):
    """Token t of k, v to row at[t] of page where[t], plainly."""
    want = [None if t is None else t.clone() for t in cache]
    for i, x in ((0, k), (1, v)):
        if cache.k_scales is None:
            want[i][where, :, at] = x
        else:
            want[i][where, :, at], want[2 + i][where, :, at] = quantized(x)
    return want


def same(cache, want):
    return all(a is None if b is None else torch.equal(a.view(U8), b.view(U8)) for a, b in zip(cache, want))


@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 104, 128])
@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_append(D, mx8, page):
    lens, new = [70, 5, 0, 33, 130], [70, 2, 0, 1, 64]
    pages, table, lengths = tables(lens, page)
    k, v = rnd(sum(new) + 3, 3, D, seed=1, scale=9), rnd(sum(new) + 3, 3, D, seed=2)
    where, at = [], []
    for b, n in enumerate(new):
        for p in range(lens[b] - n, lens[b]):
            where.append(int(table[b, p // page]))
            at.append(p % page)
    cache = new_cache(pages, page, 3, D, mx8)
    n = sum(new)
    want = place(cache, k[:n], v[:n], torch.tensor(where, device=DEV), torch.tensor(at, device=DEV))
    nv.nvfp4_cache_append(k, v, cache, table, lengths, offsets(new))  # the last 3 tokens are nobody's
    assert same(cache, want)
    # one token per sequence, out of a wider row
    lens = [70, 5, 1, 33, 130]
    pages, table, lengths = tables(lens, page, seed=3)
    cache = new_cache(pages, page, 3, D, mx8)
    rows = rnd(5, 8, D, seed=4)
    k, v = rows[:, 1:4], rows[:, 5:]
    b = torch.arange(5, device=DEV)
    want = place(cache, k, v, table[b, (lengths - 1).long() // page].long(), (lengths - 1).long() % page)
    nv.nvfp4_cache_append(k, v, cache, table, lengths)
    assert same(cache, want)


@pytest.mark.parametrize("mx8", [False, True])
def test_append_leaves_out_what_has_no_place(mx8):
    page, D = 16, 64
    table = torch.tensor([[0, 7, -1], [99, 2, -5], [3, 4, 5], [6, 1, 2 ** 31 - 1], [-2 ** 31, 5, 6]], dtype=I32, device=DEV)
    # a page outside, none, a position past the table, lengths of zero and below
    lengths = torch.tensor([40, 10, 49, 0, -7], dtype=I32, device=DEV)
    k, v = rnd(5, 2, D, seed=1), rnd(5, 2, D, seed=2)
    cache = new_cache(8, page, 2, D, mx8)
    want = [None if t is None else t.clone() for t in cache]
    nv.nvfp4_cache_append(k, v, cache, table, lengths)
    assert same(cache, want)
    # offsets that say nothing sensible
    for cu in ([5, 4, 3, 2, 1, 0], [-9, 2, 2 ** 31 - 1, -2 ** 31, 7, 90], [0, 0, 0, 0, 0, 0]):
        nv.nvfp4_cache_append(k, v, cache, torch.full_like(table, 8), lengths, torch.tensor(cu, device=DEV).to(I32))
        assert same(cache, want)


def test_append_of_values_that_are_not_finite():
    page, D = 16, 72
    pages, table, lengths = tables([1, 1], page)
    k, v = rnd(2, 1, D, seed=1), rnd(2, 1, D, seed=2)
    k[0, 0, 3], v[1, 0, 71] = math.nan, -math.inf
    cache = new_cache(pages, page, 1, D, True)
    want = place(cache, k, v, table[:, 0].long(), torch.zeros(2, dtype=torch.long, device=DEV))
    nv.nvfp4_cache_append(k, v, cache, table, lengths)
    assert same(cache, want)


def values(cache, table, lens, D):
    """k, v [sum(lens), Hkv, D] that the cache holds, float64."""
    out = []
    page = cache.k.shape[2]
    for i in range(2):
        x = cache[i]
        if cache.k_scales is not None:
            s = cache[2 + i].view(torch.float8_e8m0fnu).double().repeat_interleave(32, -1)[..., :D]
            x = x.view(torch.float8_e4m3fn).double() * s
        x = x.double()
        rows = [x[table[b, : -(-n // page)].long()].transpose(1, 2).flatten(0, 1)[:n] for b, n in enumerate(lens)]
        out.append(torch.cat(rows))
    return out


def filled(lens, page, Hkv, D, mx8, seed=0):
    pages, table, lengths = tables(lens, page, seed)
    cache = new_cache(pages, page, Hkv, D, mx8, fill=0xFF)  # NaN wherever nothing is written
    k, v = rnd(sum(lens), Hkv, D, seed=seed + 1), rnd(sum(lens), Hkv, D, seed=seed + 2)
    if lens:
        nv.nvfp4_cache_append(k, v, cache, table, lengths, offsets(lens))
    return cache, table, lengths


def run(lens, Hq, Hkv, D, page, mx8, seed=0, scale=None):
    cache, table, lengths = filled(lens, page, Hkv, D, mx8, seed)
    q = rnd(len(lens), Hq, D, seed=seed + 5)
    out = nv.nvfp4_paged_attention(q, cache, table, lengths, scale=scale)
    k, v = values(cache, table, lens, D)
    check(out, None, definition(q, k, v, [1] * len(lens), lens, False, D ** -0.5 if scale is None else scale))
    assert torch.equal(out, nv.nvfp4_paged_attention(q, cache, table, lengths, scale=scale))


@pytest.mark.parametrize("D", [8, 16, 32, 40, 64, 72, 80, 96, 104, 112, 128])
@pytest.mark.parametrize("mx8", [False, True])
def test_head_sizes(D, mx8):
    run([1, 200, 33], 4, 2, D, 16, mx8, seed=D)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 1000, 4097])
@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_lengths(n, mx8, page):
    run([n], 4, 1, 64, page, mx8, seed=n)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 1), (12, 4), (24, 3), (32, 1), (33, 1), (70, 2)])
@pytest.mark.parametrize("mx8", [False, True])
def test_grouped_heads(Hq, Hkv, mx8):
    run([100, 0, 1, 333], Hq, Hkv, 72, 32, mx8, seed=Hq)


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("lens", [[0, 0], [1] * 300, list(range(100)), [5000, 1, 0, 70], [20000]])
def test_batches(lens, mx8):
    run(lens, 4, 2, 64, 64, mx8, seed=len(lens))


@pytest.mark.parametrize("scale", [0.001, 1.0, 3.0])
def test_scales(scale):
    run([600, 40], 4, 2, 64, 16, True, seed=3, scale=scale)


def test_pages_outside_the_cache_hold_no_keys():
    page, D = 16, 64
    cache, table, lengths = filled([100, 60], page, 2, D, False)
    q = rnd(2, 4, D, seed=9)
    bad = table.clone()
    bad[0, 1], bad[0, 4], bad[1, 3] = 10 ** 6, -2 ** 31, cache.k.shape[0]
    out = nv.nvfp4_paged_attention(q, cache, bad, lengths)
    k, v = values(cache, table, [100, 60], D)
    keep = torch.ones(160, dtype=torch.bool, device=DEV)
    keep[16:32] = keep[64:80] = keep[148:160] = False
    check(out, None, definition(q, k[keep], v[keep], [1, 1], [68, 48], False, 0.125))
    none = nv.nvfp4_paged_attention(q, cache, torch.full_like(table, -1), lengths)
    assert bool((none == 0).all())
    # lengths past the table end there, negative ones at zero
    most = torch.tensor([2 ** 31 - 1, -5], dtype=I32, device=DEV)
    out = nv.nvfp4_paged_attention(q, cache, table[:, :6].contiguous(), most)
    check(out[:1], None, definition(q[:1], k[:96], v[:96], [1], [96], False, 0.125))
    assert bool((out[1] == 0).all())


@pytest.mark.parametrize("mx8", [False, True])
def test_a_cache_past_4_gib(mx8):
    page, D, Hkv = 1024, 128, 8
    pages = 5000 if mx8 else 2500  # 5.2 GB each
    cache = nv.paged_cache(pages, page, Hkv, D, mx8=mx8)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=I32, device=DEV)
    n = 2 * page + 70
    lengths = torch.tensor([n], dtype=I32, device=DEV)
    k, v, q = rnd(n, Hkv, D, seed=1), rnd(n, Hkv, D, seed=2), rnd(1, 32, D, seed=3)
    nv.nvfp4_cache_append(k, v, cache, table, lengths, offsets([n]))
    small = nv.paged_cache(3, page, Hkv, D, mx8=mx8)
    t = torch.tensor([[2, 0, 1]], dtype=I32, device=DEV)
    nv.nvfp4_cache_append(k, v, small, t, lengths, offsets([n]))
    assert torch.equal(nv.nvfp4_paged_attention(q, cache, table, lengths), nv.nvfp4_paged_attention(q, small, t, lengths))
    assert torch.equal(cache.k[pages - 1], small.k[2]) and torch.equal(cache.v[pages - 2, :, :70], small.v[1, :, :70])


def test_views_and_given_tensors():
    cache, table, lengths = filled([100, 60, 3], 16, 2, 72, True)
    rows = rnd(3, 9, 72, seed=1)
    q = rows[:, 2:6]
    want = nv.nvfp4_paged_attention(q.contiguous(), cache, table, lengths)
    out = torch.full((4, 3, 72), 5.0, dtype=BF, device=DEV).transpose(0, 1)
    assert nv.nvfp4_paged_attention(q, cache, table, lengths, out=out) is out and torch.equal(out, want)
    own = q.clone()
    assert torch.equal(nv.nvfp4_paged_attention(own, cache, table, lengths, out=own), want)
    wide = torch.full((3, 40), -1, dtype=I32, device=DEV)
    wide[:, : table.shape[1]] = table
    assert torch.equal(nv.nvfp4_paged_attention(q, cache, wide[:, : table.shape[1]], lengths), want)
    n = nv.nvfp4_paged_attention_workspace_bytes(3, 4, 2, 72, table.shape[1] * 16)
    ws = torch.empty(n, dtype=U8, device=DEV)
    assert torch.equal(nv.nvfp4_paged_attention(q, cache, table, lengths, workspace=ws), want)


@pytest.mark.parametrize("mx8", [False, True])
def test_prompt_then_tokens(mx8):
    """A run as it would be used: prompts of different lengths through attention and into the cache, then tokens one by one.
    Every token's output is the causal attention's over all its sequence (over the cache's values)."""
    D, Hq, Hkv, page = 72, 6, 2, 16
    prompt, steps = [40, 1, 77], 20
    total = [n + steps for n in prompt]
    q, k, v = qkv(total, total, Hq, Hkv, D)
    pages, table, _ = tables(total, page)
    cache = new_cache(pages, page, Hkv, D, mx8, fill=0xFF)
    begin = [0, total[0], total[0] + total[1]]
    first = torch.cat([torch.arange(b, b + n) for b, n in zip(begin, prompt)]).to(DEV)
    cu = offsets(prompt)
    out = nv.nvfp4_attention(q[first], k[first], v[first], causal=True, cu_q=cu, cu_k=cu)[0]
    want = definition(q[first], k[first], v[first], prompt, prompt, True, D ** -0.5)
    check(out, None, want)
    lengths = torch.tensor(prompt, dtype=I32, device=DEV)
    nv.nvfp4_cache_append(k[first], v[first], cache, table, lengths, cu)
    outs = []
    for s in range(steps):
        at = torch.tensor([b + n + s for b, n in zip(begin, prompt)], device=DEV)
        lengths += 1
        nv.nvfp4_cache_append(k[at], v[at], cache, table, lengths)
        outs.append(nv.nvfp4_paged_attention(q[at], cache, table, lengths))
    hk, hv = values(cache, table, total, D)
    if not mx8:
        assert torch.equal(hk, k.double()) and torch.equal(hv, v.double())
    whole = definition(q, hk, hv, total, total, True, D ** -0.5)
    for s in range(steps):
        at = torch.tensor([b + n + s for b, n in zip(begin, prompt)], device=DEV)
        check(outs[s], None, (whole[0][at], whole[1][at], whole[2][at], whole[3]))

"""Attention and the paged cache as programs run them: captured in graphs and replayed, on streams, two calls at once, with
given workspaces, under autograd in a graph.  Every replay is compared bit for bit with the eager call."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import BF, DEV, check, definition, offsets, qkv, rnd
from test_gpu_paged_attention import filled, new_cache, same, tables

pytestmark = pytest.mark.gpu

SHAPES = [([300], [300], 4, 2, 72), ([17], [5000], 4, 1, 128), ([40, 0, 333], [100, 7, 333], 6, 3, 64)]


def call(shape, seed=0):
    nq, nk, Hq, Hkv, D = shape
    q, k, v = qkv(nq, nk, Hq, Hkv, D, seed=seed)
    cu = dict(cu_q=offsets(nq), cu_k=offsets(nk), causal=True)
    return q, k, v, rnd(sum(nq), Hq, D, seed=seed + 9), cu


def step(q, k, v, u, cu):
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    return (out, lse, *nv.nvfp4_attention_backward(u, q, k, v, out, lse, **cu))


@pytest.mark.parametrize("shape", SHAPES)
def test_graph_replays(shape):
    q, k, v, u, cu = call(shape)
    fresh = [call(shape, seed=s)[:4] for s in (20, 30, 40)]
    step(q, k, v, u, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(q, k, v, u, cu)
    for new in fresh + fresh[:1]:
        want = step(*new, cu)
        for t, x in zip((q, k, v, u), new):
            t.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        junk = torch.randn(1 << 20, device=DEV).sum()  # the program's own work between replays
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and bool(torch.isfinite(junk))


@pytest.mark.parametrize("mx8", [False, True])
def test_decoding_graph_replays(mx8):
    """A decode step captured once; lengths and page tables change between the replays."""
    D, Hq, Hkv, page, B, steps = 128, 8, 2, 16, 3, 40
    total = [600, 40, 77]
    pages, table, _ = tables(total, page)
    cache, plain = new_cache(pages, page, Hkv, D, mx8), new_cache(pages, page, Hkv, D, mx8)
    q, k, v = (rnd(B * steps, h, D, seed=i) for i, h in enumerate((Hq, Hkv, Hkv)))
    lengths = torch.tensor([n - steps for n in total], dtype=torch.int32, device=DEV)
    qs, ks, vs, at = q[:B].clone(), k[:B].clone(), v[:B].clone(), lengths.clone()

    def one(c):
        nv.nvfp4_cache_append(ks, vs, c, table, at)
        return nv.nvfp4_paged_attention(qs, c, table, at)
    one(plain)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one(cache)
    for t in (cache, plain):
        for x in t:
            if x is not None:
                x.zero_()
    for s in range(steps):
        for a, b in ((qs, q), (ks, k), (vs, v)):
            a.copy_(b[s * B: (s + 1) * B])
        at += 1
        graph.replay()
        assert torch.equal(out, one(plain)) and same(cache, plain), s


def test_autograd_in_a_graph():
    nq = [100, 30]
    rows = rnd(sum(nq), 6, 64, seed=1).requires_grad_()
    cu, u = offsets(nq), rnd(sum(nq), 2, 64, seed=2)

    def grad():
        return torch.autograd.grad(nv.attention(*rows.split(2, 1), causal=True, cu_q=cu, cu_k=cu), rows, u)[0]
    want = grad().clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        grad()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grad()
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("shape", SHAPES)
def test_two_calls_at_once_on_two_streams(shape):
    calls = [call(shape, seed=s) for s in (0, 50)]
    want = [step(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(step(*c))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_stream_arguments():
    q, k, v, u, cu = call(SHAPES[1])
    want = step(q, k, v, u, cu)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, stream=s, **cu)
    grads = nv.nvfp4_attention_backward(u, q, k, v, out, lse, stream=s, **cu)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))
    cache, table, lengths = filled([600, 33], 16, 2, 64, True)
    qd = rnd(2, 4, 64, seed=3)
    want = nv.nvfp4_paged_attention(qd, cache, table, lengths)
    torch.cuda.synchronize()
    got = nv.nvfp4_paged_attention(qd, cache, table, lengths, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("shape", SHAPES)
def test_given_workspaces_of_any_content(shape):
    q, k, v, u, cu = call(shape)
    nq, nk, Hq, Hkv, D = shape
    want = step(q, k, v, u, cu)
    sizes = (sum(nq), sum(nk), Hq, Hkv, D, len(nq))
    n = max(nv.nvfp4_attention_workspace_bytes(*sizes), 16)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, workspace=ws, **cu)
    ws = torch.full((nv.nvfp4_attention_backward_workspace_bytes(*sizes),), 0xFF, dtype=torch.uint8, device=DEV)
    grads = nv.nvfp4_attention_backward(u, q, k, v, out, lse, workspace=ws, **cu)
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_attention_backward(u, q, k, v, out, lse, workspace=ws[: ws.numel() // 2], **cu)
    with pytest.raises(ValueError):
        nv.nvfp4_attention(q, k, v, workspace=ws.cpu(), **cu)


@pytest.mark.parametrize("m,n,Hq,Hkv,D,causal", [(1, 3000, 2, 1, 64, True), (17, 4096, 8, 2, 128, True), (200, 1500, 3, 3, 96, False),
                                                 (500, 300, 2, 2, 72, True), (64, 20000, 1, 1, 40, False)])
def test_few_queries_over_many_keys(m, n, Hq, Hkv, D, causal):
    """Several workgroups share a block of queries, and join their sums."""
    assert nv.nvfp4_attention_workspace_bytes(m, n, Hq, Hkv, D, 1) > 0 or m == 500
    q, k, v = qkv([m], [n], Hq, Hkv, D, seed=n)
    out, lse = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True)
    check(out, lse, definition(q, k, v, [m], [n], causal, D ** -0.5))
    again, l2 = nv.nvfp4_attention(q, k, v, causal=causal, save_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, l2)


def test_long_prompt_prefix_of_shared_pages():
    """Two sequences whose tables name the same pages for a common prefix read the same rows."""
    page, D = 16, 64
    cache, table, lengths = filled([64, 80], page, 2, D, False)
    both = table.clone()
    both[1, :4] = table[0, :4]
    q = rnd(2, 4, D, seed=3)
    q[1] = q[0]
    n = torch.tensor([64, 64], dtype=torch.int32, device=DEV)
    out = nv.nvfp4_paged_attention(q, cache, both, n)
    assert torch.equal(out[0], out[1])


def test_heads_of_no_size_are_refused_by_the_calls():
    q, k, v, u, cu = call(SHAPES[0])
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True, **cu)
    none = lambda t: t[..., :0].contiguous()  # noqa: E731
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_attention(none(q), none(k), none(v), **cu)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_attention_backward(none(u), none(q), none(k), none(v), none(out), lse, **cu)
    cache = nv.paged_cache(4, 16, 2, 0)
    table, lengths = torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_paged_attention(none(q[:1]), cache, table, lengths)

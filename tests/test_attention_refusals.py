"""What the attention and cache calls refuse, on the host: no GPU is needed (fake device pointers are never dereferenced,
because validation fails first)."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv

S = nv.Status
P = [0x1000000 * (i + 1) for i in range(12)]
P8, PODD = 0x10008, 0x10001
STOPS = (S.ERR_HIP, S.ERR_DEVICE)  # past validation: without a GPU the device check ends the call
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers")
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def attention(L, q=P[0], qt=256, qh=64, k=P[1], kt=128, kh=64, v=P[2], vt=128, vh=64, Tq=100, Tk=90, Hq=4, Hkv=2, D=64,
              cq=P[3], ck=P[4], B=3, causal=1, scale=0.125, o=P[5], ot=256, oh=64, lse=P[6], ws=P[7], n=1 << 30):
    return L.nvfp4_attention(q, qt, qh, k, kt, kh, v, vt, vh, Tq, Tk, Hq, Hkv, D, cq, ck, B, causal, scale, o, ot, oh, lse, ws,
                             n, None)


def backward(L, do=P[8], dot=256, doh=64, q=P[0], qt=256, qh=64, k=P[1], kt=128, kh=64, v=P[2], vt=128, vh=64, o=P[5],
             ot=256, oh=64, lse=P[6], Tq=100, Tk=90, Hq=4, Hkv=2, D=64, cq=P[3], ck=P[4], B=3, scale=0.125, dq=P[9], dqt=256,
             dqh=64, dk=P[10], dkt=128, dkh=64, dv=P[11], dvt=128, dvh=64, ws=P[7], n=1 << 30):
    return L.nvfp4_attention_backward(do, dot, doh, q, qt, qh, k, kt, kh, v, vt, vh, o, ot, oh, lse, Tq, Tk, Hq, Hkv, D, cq, ck,
                                      B, 1, scale, dq, dqt, dqh, dk, dkt, dkh, dv, dvt, dvh, ws, n, None)


@pytest.mark.parametrize("call", [attention, backward])
def test_shapes_and_scale(L, call):
    for kw in (dict(Tq=-1), dict(Tk=-1), dict(Tq=1 << 31), dict(Tk=1 << 31), dict(Hq=-1), dict(Hkv=-1), dict(Hq=3), dict(Hkv=0),
               dict(Hkv=8), dict(D=0), dict(D=4), dict(D=60), dict(D=136), dict(B=-1), dict(B=(1 << 20) + 1), dict(Hq=1 << 17, Hkv=1),
               dict(Tq=1 << 30, Hq=32, Hkv=1), dict(Tk=1 << 30, Hq=32, Hkv=1)):
        assert call(L, **kw) == S.ERR_SHAPE, kw
    for kw in (dict(B=3, Tq=100, Tk=90), dict(B=3, Tq=99, Tk=91)):  # equal sequences
        assert call(L, cq=None, ck=None, **kw) == S.ERR_SHAPE, kw
    assert call(L, cq=None, ck=None, B=0) == S.ERR_SHAPE  # rows of no sequence
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(L, scale=scale) == S.ERR_MODE, scale
    assert call(L, cq=None) == S.ERR_NULL and call(L, ck=None) == S.ERR_NULL


@pytest.mark.parametrize("call,inputs,outputs", [(attention, "q k v", "o"), (backward, "do q k v o", "dq dk dv")])
def test_tensors(L, call, inputs, outputs):
    for name in (inputs + " " + outputs).split():
        assert call(L, **{name: None}) == S.ERR_NULL, name
        for bad in (P8, PODD):
            assert call(L, **{name: bad}) == S.ERR_ALIGN, name
        assert call(L, **{name + "t": 257}) == S.ERR_ALIGN and call(L, **{name + "t": 1024, name + "h": 68}) == S.ERR_ALIGN, name
        for kw in ({name + "t": 32}, {name + "t": 0}, {name + "t": -64}, {name + "h": -64}, {name + "t": 1 << 23}, {name + "t": BIG},
                   {name + "h": BIG}):
            assert call(L, **kw) == S.ERR_STRIDE, kw
    for name in outputs.split():  # rows that overlap
        for kw in ({name + "h": 0}, {name + "h": 32}, {name + "t": 64, name + "h": 64}):
            assert call(L, **kw) == S.ERR_STRIDE, kw
    assert call(L, lse=PODD) == S.ERR_ALIGN and call(L, cq=PODD) == S.ERR_ALIGN and call(L, ck=PODD) == S.ERR_ALIGN


def test_workspaces(L):
    n = L.nvfp4_attention_workspace_bytes(17, 8192, 4, 2, 64, 1)
    assert n > 0
    few = dict(Tq=17, Tk=8192, B=1)
    assert attention(L, ws=None, n=0, **few) == S.ERR_WORKSPACE and attention(L, n=n - 1, **few) == S.ERR_WORKSPACE
    assert attention(L, ws=P8, n=1 << 30, **few) == S.ERR_ALIGN
    assert L.nvfp4_attention_workspace_bytes(8192, 8192, 32, 8, 128, 1) == 0
    for args in ((-1, 8, 4, 2, 64, 1), (8, 8, 4, 3, 64, 1), (8, 8, 4, 2, 60, 1), (8, 8, 4, 2, 64, -1), (8, 8, 0, 0, 64, 1)):
        assert L.nvfp4_attention_workspace_bytes(*args) == 0 == L.nvfp4_attention_backward_workspace_bytes(*args), args
    n = L.nvfp4_attention_backward_workspace_bytes(100, 90, 4, 2, 64, 3)
    assert n >= 2 * 4 * 100 * 4
    assert backward(L, ws=None) == S.ERR_WORKSPACE and backward(L, n=n - 1) == S.ERR_WORKSPACE
    assert backward(L, ws=P8) == S.ERR_ALIGN and backward(L, lse=None) == S.ERR_NULL
    n = L.nvfp4_paged_attention_workspace_bytes(2, 32, 8, 128, 8192)
    assert n > 0 and L.nvfp4_paged_attention_workspace_bytes(2, 32, 8, 128, 128) == 0
    for args in ((0, 32, 8, 128, 8192), (1 << 16, 32, 8, 128, 8192), (2, 30, 8, 128, 8192), (2, 32, 0, 128, 8192), (2, 32, 8, 12, 8192),
                 (2, 32, 8, 128, -1), (2, 32, 8, 128, 1 << 30)):
        assert L.nvfp4_paged_attention_workspace_bytes(*args) == 0, args


def test_written_in_an_inputs_place(L):
    assert attention(L, o=P[0], ot=512) == S.ERR_STRIDE and attention(L, o=P[0], qt=512) == S.ERR_STRIDE
    for out in ("dq", "dk", "dv"):
        for other in (P[8], P[0], P[1], P[2], P[5]):
            assert backward(L, **{out: other}) == S.ERR_STRIDE, (out, other)


@NO_GPU
def test_what_is_taken(L):
    for kw in ({}, dict(o=P[0]), dict(lse=None), dict(cq=None, ck=None, B=10), dict(ck=P[3]), dict(Tk=0, k=None, v=None),
               dict(Tq=1, qt=0, ot=0), dict(Hq=1, Hkv=1, qh=0, kh=-8, vh=5 * 8, oh=0, qt=64, kt=64, vt=64, ot=64), dict(kh=0, vh=0),
               dict(qt=64, qh=6400, ot=64, oh=6400)):
        assert attention(L, **kw) in STOPS or kw.get("kh") == -8, kw
    for kw in ({}, dict(cq=None, ck=None, B=10), dict(Tk=0, k=None, v=None, dk=None, dv=None), dict(Tq=0, q=None, o=None, do=None, dq=None)):
        assert backward(L, **kw) in STOPS, kw
    for call in (attention, backward):
        for kw in (dict(Hq=0, Hkv=0), dict(B=0)):
            assert call(L, **kw) == S.OK, kw
    assert attention(L, Tq=0, q=None, o=None) == S.OK and backward(L, Tq=0, Tk=0) == S.OK


def append(L, k=P[0], kt=128, kh=64, v=P[1], vt=128, vh=64, T=20, H=2, D=64, cu=P[2], le=P[3], B=4, ck=P[4], ks=P[5], cv=P[6],
           vs=P[7], pages=9, size=16, table=P[8], ld=5, most=5):
    return L.nvfp4_cache_append(k, kt, kh, v, vt, vh, T, H, D, cu, le, B, ck, ks, cv, vs, pages, size, table, ld, most, None)


def paged(L, q=P[0], qt=256, qh=64, B=4, Hq=4, H=2, D=64, ck=P[4], ks=P[5], cv=P[6], vs=P[7], pages=9, size=16, table=P[8], ld=500,
          most=500, le=P[3], scale=0.125, o=P[9], ot=256, oh=64, ws=P[10], n=1 << 30):
    return L.nvfp4_paged_attention(q, qt, qh, B, Hq, H, D, ck, ks, cv, vs, pages, size, table, ld, most, le, scale, o, ot, oh, ws, n,
                                   None)


@pytest.mark.parametrize("call", [append, paged])
def test_caches(L, call):
    for kw in (dict(D=0), dict(D=12), dict(D=136), dict(H=-1), dict(B=-1), dict(B=1 << 16), dict(pages=-1), dict(pages=1 << 31),
               dict(size=0), dict(size=8), dict(size=24), dict(size=1 << 21), dict(most=-1), dict(most=1 << 28), dict(most=1 << 26, ld=1 << 26), dict(pages=1 << 30, size=1 << 14)):
        assert call(L, **kw) == S.ERR_SHAPE, kw
    for name in ("ck", "ks", "cv", "vs", "table", "le"):
        assert call(L, **{name: None}) == S.ERR_NULL, name
    for name in ("ck", "cv"):
        assert call(L, **{name: P8}) == S.ERR_ALIGN, name
    assert call(L, table=PODD) == S.ERR_ALIGN and call(L, le=PODD) == S.ERR_ALIGN
    assert call(L, ld=4, most=5) == S.ERR_STRIDE and call(L, ld=1 << 50) == S.ERR_STRIDE


def test_append(L):
    for kw in (dict(T=-1), dict(T=1 << 30), dict(cu=None, T=5)):
        assert append(L, **kw) == S.ERR_SHAPE, kw
    for name in "kv":
        assert append(L, **{name: None}) == S.ERR_NULL and append(L, **{name: P8}) == S.ERR_ALIGN
        assert append(L, **{name + "t": 32}) == S.ERR_STRIDE and append(L, **{name + "t": 132}) == S.ERR_ALIGN
    assert append(L, cu=PODD) == S.ERR_ALIGN
    assert append(L, T=0, k=None, v=None) == S.OK and append(L, B=0, T=3) == S.OK


def test_paged(L):
    for kw in (dict(Hq=-1), dict(Hq=3), dict(H=0), dict(Hq=1 << 17, H=1)):
        assert paged(L, **kw) == S.ERR_SHAPE, kw
    for scale in (0.0, -2.0, float("nan"), float("inf")):
        assert paged(L, scale=scale) == S.ERR_MODE
    for name in "qo":
        assert paged(L, **{name: None}) == S.ERR_NULL and paged(L, **{name: P8}) == S.ERR_ALIGN
        assert paged(L, **{name + "t": 32}) == S.ERR_STRIDE and paged(L, **{name + "h": 36}) in (S.ERR_ALIGN, S.ERR_STRIDE)
    assert paged(L, o=P[0], ot=512) == S.ERR_STRIDE and paged(L, oh=0) == S.ERR_STRIDE
    need = L.nvfp4_paged_attention_workspace_bytes(4, 4, 2, 64, 8000)
    assert need > 0 and paged(L, ws=None) == S.ERR_WORKSPACE and paged(L, n=need - 1) == S.ERR_WORKSPACE and paged(L, ws=P8) == S.ERR_ALIGN
    assert paged(L, B=0) == S.OK and paged(L, Hq=0, H=0) == S.OK


@NO_GPU
def test_caches_that_are_taken(L):
    for kw in ({}, dict(ks=None, vs=None), dict(most=0, table=None)):
        assert append(L, **kw) in STOPS and paged(L, **kw) in STOPS, kw
    assert append(L, pages=0, ck=None, cv=None) in STOPS and paged(L, pages=0, ck=None, cv=None) in STOPS
    assert append(L, cu=None, T=4) in STOPS and paged(L, o=P[0]) in STOPS and paged(L, most=8, ws=None, n=0) in STOPS


def test_python_refuses_host_tensors_and_wrong_forms():
    q, kv = torch.zeros(6, 4, 64).bfloat16(), torch.zeros(6, 2, 64).bfloat16()
    cache = nv.paged_cache(3, 16, 2, 64, device="cpu")
    table, lengths = torch.zeros(6, 1, dtype=torch.int32), torch.ones(6, dtype=torch.int32)
    for call in (lambda: nv.nvfp4_attention(q, kv, kv), lambda: nv.nvfp4_attention(q[0], kv, kv), lambda: nv.attention(q, kv, kv),
                 lambda: nv.nvfp4_attention_backward(q, q, kv, kv, q, torch.zeros(4, 6)),
                 lambda: nv.nvfp4_cache_append(kv, kv, cache, table, lengths), lambda: nv.nvfp4_cache_append(kv[0], kv, cache, table, lengths),
                 lambda: nv.nvfp4_paged_attention(q, cache, table, lengths), lambda: nv.nvfp4_paged_attention(q[0], cache, table, lengths)):
        with pytest.raises(ValueError):
            call()

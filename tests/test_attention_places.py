"""Outputs at the address of an array that the same call reads or writes: refused on the host (fake device pointers are never
dereferenced), but for a query's output in the query's place."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_attention_refusals import NO_GPU, P, STOPS, S, append, attention, backward, paged


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def test_outputs_in_the_place_of_keys_and_values(L):
    for i in (1, 2):
        assert attention(L, o=P[i]) == S.ERR_STRIDE
        assert attention(L, o=P[i], Tq=90, Tk=90, Hkv=4, ot=256, kt=256, vt=256) == S.ERR_STRIDE
    for i in (4, 6):
        assert paged(L, o=P[i]) == S.ERR_STRIDE
        assert paged(L, ks=None, vs=None, o=P[i]) == S.ERR_STRIDE


def test_two_gradients_in_one_place(L):
    for a, b in (("dq", "dk"), ("dq", "dv"), ("dk", "dv")):
        assert backward(L, **{a: P[9], b: P[9], "Tq": 90}) == S.ERR_STRIDE


def test_negative_pitches_of_a_single_head_are_refused(L):
    for kw in (dict(kh=-8), dict(vh=-8), dict(qh=-8), dict(oh=-8)):
        assert attention(L, Hq=1, Hkv=1, qt=64, kt=64, vt=64, ot=64, **kw) == S.ERR_STRIDE


@NO_GPU
def test_what_is_taken(L):
    for kw in (dict(o=P[0]), dict(k=P[2]), dict(Tk=0, k=P[5], v=P[5])):
        assert attention(L, **kw) in STOPS, kw
    for kw in (dict(Tq=0, q=None, o=None, do=None, dq=P[10]), dict(Tk=0, k=None, v=None, dk=P[9], dv=P[9])):
        assert backward(L, **kw) in STOPS, kw
    assert paged(L, o=P[0]) in STOPS and paged(L, cv=P[4]) in STOPS  # keys that are the values, too
    assert append(L) in STOPS


@pytest.mark.gpu
def test_refused_by_the_calls():
    q, k, v = (torch.zeros(20, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for out in (k, v):
        with pytest.raises(nv.NVFP4Error):
            nv.nvfp4_attention(q, k, v, out=out)
    out, lse = nv.nvfp4_attention(q, k, v, save_lse=True)
    one = torch.empty_like(q)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_attention_backward(q, q, k, v, out, lse, dk=one, dv=one)

"""Scores that share a large offset: softmax does not see it.  Two places of a head are not 0, so that scores are exact in fp32
(an offset and 0 .. 16 in steps of 1/4); tolerances as in test_gpu_attention_large_scores.py, 2^-8 |o| + 2^-8 A for the
roundings to bf16 and 2^-15 A for fp32's."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import BF, DEV, rnd
from test_gpu_attention_large_scores import close
from test_gpu_paged_attention import filled, values

pytestmark = pytest.mark.gpu

OFFSETS = [0, 2 ** 8, 2 ** 12, 2 ** 15, 2 ** 17, 2 ** 18, 2 ** 19, 2 ** 20, 2 ** 21]


def deltas(n, kind):
    g = torch.Generator().manual_seed(n)
    d = torch.randint(0, 64, (n,), generator=g).float() / 4
    if kind == "rising":  # many small ones before a few that rise past the step at which a maximum moves
        d = torch.arange(n).float() * 64 / n
        d = d.floor() / 4
        d[: n // 2] = d[: n // 2] / 4
        d = (d * 4).floor() / 4
    return d.to(DEV)


def rows(n, D, kind):
    k = torch.zeros(n, D, dtype=BF, device=DEV)
    k[:, 1], k[:, 2] = 1.0, deltas(n, kind).to(BF)
    return k


def query(H, D, offset, sign):
    q = torch.zeros(1, H, D, dtype=BF, device=DEV)
    q[..., 1], q[..., 2] = sign * float(offset), 1.0
    return q


def wanted(q, k, v):
    s = q.double() @ k.double().t()
    p = torch.softmax(s, 1)
    return p @ v.double(), p @ v.double().abs()


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kind", ["random", "rising"])
@pytest.mark.parametrize("nq,nk", [(1, 300), (150, 1000), (5, 4096)])
def test_attention(offset, sign, kind, nq, nk):
    D = 64
    q, k, v = query(2, D, offset, sign).expand(nq, 2, D).contiguous(), rows(nk, D, kind)[:, None], rnd(nk, 1, D, seed=2)
    out, lse = nv.nvfp4_attention(q, k, v, scale=1.0, save_lse=True)
    want, A = wanted(q[0, :1], k[:, 0], v[:, 0])
    close(out, want.expand(nq, 2, D), A.expand(nq, 2, D))
    exact = torch.logsumexp(q[0, :1].double() @ k[:, 0].double().t(), 1)
    assert bool(((lse.double() - exact).abs() <= 2.0 ** -21 * exact.abs() + 2.0 ** -20).all())


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kind", ["random", "rising"])
@pytest.mark.parametrize("n,Hq", [(100, 2), (500, 1), (4096, 2), (3000, 40)])
def test_single_tokens(offset, sign, kind, n, Hq):
    D, page = 64, 16
    cache, table, lengths = filled([n], page, 1, D, False)
    pages = table[0, : -(-n // page)].long()
    cache.k[pages, 0] = rows(len(pages) * page, D, kind).view(len(pages), page, D)
    q = query(Hq, D, offset, sign)
    out = nv.nvfp4_paged_attention(q, cache, table, lengths, scale=1.0)
    k, v = values(cache, table, [n], D)
    want, A = wanted(q[0, :1], k[:, 0], v[:, 0])
    close(out, want.expand(1, Hq, D), A.expand(1, Hq, D))

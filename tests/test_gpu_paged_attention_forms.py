"""More forms of the paged cache's calls: more than 16 query heads over one key head (two sets of columns) at every head size,
with and without a join, and appending with offsets of any content, against a model of the rule."""
import pytest
import torch

import nvfp4_quantized_gemm_amd as nv
from test_gpu_attention import DEV, rnd
from test_gpu_paged_attention import I32, new_cache, place, run, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [8, 32, 40, 64, 96, 104, 128])
@pytest.mark.parametrize("group", [16, 17, 32, 33, 35])
@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("lens,page", [([100, 0, 1, 333], 16), ([1500, 31, 0, 700], 128)])
def test_many_query_heads_over_a_key_head(D, group, mx8, lens, page):
    run(lens, 2 * group, 2, D, page, mx8, seed=D + group)


def test_those_are_joined():
    assert nv.nvfp4_paged_attention_workspace_bytes(4, 34, 2, 128, 13 * 128) > 0
    assert nv.nvfp4_paged_attention_workspace_bytes(4, 34, 2, 128, 22 * 16) == 0


def token_place(cu, lengths, t):
    """(sequence, position) of token t: the last sequence that the search takes to begin at or before it; None: nobody's."""
    lo, hi = 0, len(lengths)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if cu[mid] <= t:
            lo = mid
        else:
            hi = mid
    behind = cu[lo + 1] - t
    return None if behind <= 0 or cu[lo] > t else (lo, lengths[lo] - behind)


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("cu", [[0, 3, 3, 7, 12], [2, 5, 9, 9, 11], [5, 4, 3, 2, 1], [-9, 2, 2 ** 31 - 1, -2 ** 31, 7], [0, 0, 0, 0, 0],
                                [-3, 40, 50, 60, 70], [0, 6, 2, 12, 12], [2 ** 31 - 1, -2 ** 31, 4, 4, 9]])
def test_append_with_any_offsets(cu, mx8):
    """Each sequence has pages of its own, and every token at most one place."""
    T, H, D, page, most = 12, 2, 72, 16, 3
    lengths = [30, 5, 48, 16]
    table = torch.arange(4 * most, dtype=I32).flip(0).view(4, most)
    k, v = rnd(T, H, D, seed=1), rnd(T, H, D, seed=2)
    cache = new_cache(4 * most, page, H, D, mx8)
    tokens, where, at = [], [], []
    for t in range(T):
        p = token_place(cu, lengths, t)
        if p and 0 <= p[1] < most * page:
            tokens.append(t)
            where.append(int(table[p[0], p[1] // page]))
            at.append(p[1] % page)
    want = place(cache, k[tokens], v[tokens], torch.tensor(where, dtype=torch.long, device=DEV),
                 torch.tensor(at, dtype=torch.long, device=DEV)) if tokens else [None if x is None else x.clone() for x in cache]
    nv.nvfp4_cache_append(k, v, cache, table.to(DEV), torch.tensor(lengths, dtype=I32, device=DEV),
                          torch.tensor(cu, dtype=torch.int64).to(I32).to(DEV))
    assert same(cache, want)
    assert tokens or cu in ([5, 4, 3, 2, 1], [0, 0, 0, 0, 0], [2 ** 31 - 1, -2 ** 31, 4, 4, 9], [-9, 2, 2 ** 31 - 1, -2 ** 31, 7])

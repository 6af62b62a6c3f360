"""Edges of the calls around a paged cache. Bounds as in test_gpu_paged, whose references
these tests use."""
import math

import pytest
import torch

import sparse_attention_decode_step_gb300 as csa
from helpers import need_gpu
from test_gpu_paged import DEV, TYPES, Paged, _check, _ints, _kept, _np, _queries

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# ================================================================ chunk attention: what a token does not see
BORDERS = [
    # heads, first token, entry (of 16 to a page) from which on something is wrong
    (1, 3, 304),                    # token 304 is row 301 of the group, in the tile of rows 256 .. 383
    (16, 3, 304),                   # eight tokens to a tile: 299 .. 306 share one
    (20, 0, 304),                   # a tile's border inside a token
    (64, 3, 304),                   # two tokens to a tile: 303 and 304
    (64, 0, 16),
    (8, 1, 512),                    # on the border of a tile of entries
]


def _prompt(h, first, seed, types):
    s = next(x for x in (Paged([600], 16, seed + 100 * i, spare=60) for i in range(99)) if 0 not in x.table_host[0, :38].tolist())
    q = _queries(600 - first, h, TYPES[types[0]], seed + 1)
    out = torch.zeros(600 - first, h, 512, dtype=TYPES[types[1]], device=DEV)
    return s, q, out, torch.zeros(600 - first, h, device=DEV)


@pytest.mark.parametrize("types", [("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("h, first, bad", BORDERS)
def test_chunk_a_bad_page_stays_with_the_tokens_that_see_it(h, first, bad, types):
    # page 0, which no sequence has, holds NaN scales: nothing of it may reach any token
    s, q, out, lse = _prompt(h, first, 101, types)
    s.table_host[0, bad // 16] = 1 << 20
    cnt = csa.new_counters()
    csa.chunk_attn(s.cache, csa.Groups([0], [0, 600 - first]), q, out, lse, pos=_ints([first]), pages=csa.Pages(s.table_host.to(DEV), 16),
                   counters=cnt)
    torch.cuda.synchronize()
    c = _np(cnt).tolist()
    assert c[0] == c[1] == c[3] == 0 and c[2] >= 1
    k = bad - first
    _check(lambda _g: s.values(0, bad), [0, k], [bad], [first], 1, q[:k], out[:k], lse[:k])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("groups", [slice(0, 32), slice(7, 8), slice(31, 32)])
@pytest.mark.parametrize("types", [("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("h, first, bad", BORDERS)
def test_chunk_a_nan_entry_stays_with_the_tokens_that_see_it(h, first, bad, types, groups):
    # one entry whose scales, all or one, are NaN: the tokens that see it are NaN, the others as without it
    s, q, out, lse = _prompt(h, first, 103, types)
    row = s._rows(s.table_host, 16, 0, 600)[bad].item()
    s.cache.scales[row, groups] = 0x7F if h != 16 else 0xFF
    csa.chunk_attn(s.cache, csa.Groups([0], [0, 600 - first]), q, out, lse, pos=_ints([first]), pages=s.pages)
    torch.cuda.synchronize()
    k = bad - first
    _check(lambda _g: s.values(0, bad), [0, k], [bad], [first], 1, q[:k], out[:k], lse[:k])
    assert torch.isnan(out[k:]).all() and torch.isnan(lse[k:]).all()


# ================================================================ eviction: weights at the ends of fp32
@pytest.mark.parametrize("lens", [[300], [70000], [300000], [500] * 130])
def test_evict_prefers_infinity_to_the_largest_number(lens):
    s = Paged(lens, 16, 107, to=[40] * len(lens))
    w = torch.rand(len(lens), max(lens))
    big = torch.finfo(torch.float32).max
    w[:, 10:40] = big                                       # more of them than there is room for, in front of
    w[:, 200::7][:, :20] = math.inf                         # the infinite ones
    w[:, 5:8], w[:, -9:] = math.nan, -big
    kept = torch.zeros(len(lens), 40, dtype=torch.int32, device=DEV)
    csa.cache_evict(s.cache, s.cache, w.to(DEV), 40, kept, first=4, last=8, pages=s.pages, to_pages=csa.Pages(s.to_host.to(DEV), 16))
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        want = _kept(w[b].tolist(), n, 40, 4, 8)
        assert _np(kept[b]).tolist() == want

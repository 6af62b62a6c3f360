"""Edges of the calls around a paged cache. Bounds as in test_gpu_paged, whose references
these tests use."""
import math

import pytest
import torch

import sparse_attention_decode_step_gb300 as csa
from helpers import need_gpu
from test_gpu_paged import DEV, TYPES, Paged, _check, _check_mass, _ints, _kept, _mass_reference, _np, _queries, _rope_reference, _sees

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


# ================================================================ attention weights: plans
@pytest.mark.parametrize("tokens", [1019, 1020, 1090])
def test_mass_few_groups_of_many_blocks(tokens):
    # 128 heads: a block to a token, and one more for each of the five of another sequence: up to 1,024 blocks a
    # plan of few groups is made by a thread to a block, more the general way. A sequence once more, offsets that
    # fall and the group behind them are counted once each.
    h, nq = 128, tokens + 10
    s = Paged([40, 33, 20, 17], 16, 105)
    q = _queries(nq, h, torch.bfloat16, 106)
    lse = torch.full((nq, h), 5.0, device=DEV)
    prev = torch.rand(4, 64, device=DEV)
    mass = torch.full((4, 64), 7.0, device=DEV)
    cnt = csa.new_counters()
    off, pos = [0, tokens, tokens + 5, nq, nq - 2, nq], [45 - tokens, 0, 30, 0, 0]
    csa.attn_mass(s.cache, csa.Groups([0, 0, 1, 2, 3], off), q, lse, mass, pos=_ints(pos), pages=s.pages, prev=prev, decay=0.5, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 3, 0]
    _check_mass(s.values, [0, tokens], [40], [pos[0]], 1, q, lse, prev, 0.5, mass)
    _check_mass(lambda g: s.values(1), [tokens + 5, nq], [33], [30], 1, q, lse, prev, 0.5, mass, seqs=[1])
    assert (mass[2:] == 7).all() and (mass[0, 40:] == 7).all() and (mass[1, 33:] == 7).all()


@pytest.mark.parametrize("h, tokens", [(2, 1), (64, 1), (20, 7), (128, 3)])
@pytest.mark.parametrize("spread", [0.0, 20.0, 40.0, 43.0, 46.0, 90.0])
@pytest.mark.parametrize("at", [-30.0, 10.0, 60.0])
def test_mass_small_weights_of_rows_far_apart(at, spread, h, tokens):
    # log sums of a block's rows that lie up to `spread` apart (a merged partial result makes one large), and weights
    # down to nothing: an fp32 exponential loses what lies below 2^-126, and a row is at most 2^32 from what its
    # block is computed relative to, so a weight may lose 2^-94 besides its relative error
    s = Paged([700, 90], 16, 109)
    q = _queries(2 * tokens, h, torch.float16, 110, 0.5)
    g = torch.Generator().manual_seed(111)
    lse = at + spread * torch.rand(2 * tokens, h, generator=g)
    lse[::2, 0], lse[1::2, -1] = at, at + spread
    lse = lse.to(DEV)
    off = [0, tokens, 2 * tokens]
    groups, pos = csa.Groups([0, 1], off), _ints([650, 60])
    out, own = torch.zeros(2 * tokens, h, 512, device=DEV), torch.zeros(2 * tokens, h, device=DEV)
    csa.chunk_attn(s.cache, groups, q, out, own, pos=pos, pages=s.pages, sm_scale=2.0)
    lse = torch.maximum(lse, own)                           # (a weight is at most 1)
    mass = torch.zeros(2, 700, device=DEV)
    csa.attn_mass(s.cache, groups, q, lse, mass, pos=pos, pages=s.pages, sm_scale=2.0)
    torch.cuda.synchronize()
    for b, n in enumerate([700, 90]):
        rows = slice(off[b], off[b + 1])
        want, bound = _mass_reference(s.values(b), q[rows].reshape(-1, 512), lse[rows].reshape(-1),
                                      _sees(off, b, n, [650, 60], 1, h), 2.0)
        far = (mass[b, :n].double() - want).abs() - bound - 2.0 ** -23 * want - tokens * h * 2.0 ** -94
        assert torch.isfinite(mass[b]).all() and far.max() <= 0, (far.max().item(), want[far.argmax()].item())


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


# ================================================================ norm and rotation
SPLITS = [
    # tokens, heads, rotated, type, out: enough rows that a warp takes 2, 4, 8 or 16 heads of a token, of which the
    # last warp's are fewer where the heads do not divide
    (6001, 5, 64, "bf16", "bf16"),
    (12001, 5, 512, "bf16", "f16"),
    (6001, 20, 64, "f16", "bf16"),
    (900, 65, 96, "f32", "f32"),
    (1850, 65, 128, "bf16", "bf16"),
    (1900, 127, 16, "bf16", "f32"),
    (4096, 64, 64, "bf16", "bf16"),
]


def _rope_check(got, x, w, eps, pos, freq, halves):
    y, size = _rope_reference(x, w, eps, pos, freq, halves)
    e = torch.finfo(got.dtype).eps / 2
    got64 = got.double().cpu()
    far = (got64 - y).abs() - size * 2.0 ** -20 - e * y.abs() * (1 + 2.0 ** -10) - torch.finfo(got.dtype).tiny * 2 * e
    assert torch.isfinite(got64).all() and far.max() <= 0, far.max().item()


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("n, h, rot, t, to", SPLITS)
def test_norm_rope_splits_of_heads(n, h, rot, t, to, weighted, halves):
    g = torch.Generator().manual_seed(n + h)
    gd = torch.Generator(DEV).manual_seed(n + h)
    x = torch.randn(n, h, 512, generator=gd, device=DEV).to(TYPES[t])
    pos = torch.randint(-1000, 1 << 20, (n,), generator=g, dtype=torch.int32)
    freq = (10000.0 ** (-torch.arange(rot // 2).double() / (rot // 2))).float()
    w = torch.randn(512, generator=g) if weighted else None
    kw = dict(weight=None if w is None else w.to(DEV), eps=1e-5, inv_freq=freq.to(DEV), halves=halves)
    out = torch.full((n, h, 512), float("nan"), dtype=TYPES[to], device=DEV)
    csa.norm_rope(x, out, pos=pos.to(DEV), **kw)
    # some tokens against float64, all of them against calls of few tokens, whose warps take a head each
    some = torch.cat([torch.tensor([0, n - 1]), torch.randint(0, n, (60,), generator=g)])
    torch.cuda.synchronize()
    _rope_check(out[some.to(DEV)], x[some.to(DEV)].cpu(), w, 1e-5, pos[some], freq, halves)
    few = torch.full_like(out, float("nan"))
    step = max(1, 20000 // h)
    for i in range(0, n, step):
        csa.norm_rope(x[i:i + step], few[i:i + step], pos=pos[i:i + step].to(DEV), **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, few)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("to", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n, h", [(1, 1), (1, 20), (7, 0), (700, 5)])
def test_norm_without_rotation(n, h, t, to, weighted):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(*((n, h, 512) if h else (n, 512)), generator=g).to(TYPES[t])
    w = torch.randn(512, generator=g) if weighted else None
    out = torch.full(x.shape, float("nan"), dtype=TYPES[to], device=DEV)
    csa.norm_rope(x.to(DEV), out, weight=None if w is None else w.to(DEV), eps=1e-5)
    torch.cuda.synchronize()
    _rope_check(out, x, w, 1e-5, None, None, False)

"""Attention of chunks over a paged cache, attention weights by entry, eviction, and
the norm with the rotation, against float64.

Bounds of the attention are those of the dense attention (its kernel, its arithmetic):
  the logit: 32 fp32 additions of 16-term products, each off by at most 2^-23 of
  the sum of |q v|, q's f16 subnormals (2^-25 each) and 2^-21 around the hardware
  exponential; a weight: f16, half a step 2^-11, or 2^-25 of the row's largest; the
  sums: n / 16 fp32 additions of 2^-23 and the joining of at most 152 parts; the
  output type: half a step of what is stored.
A weight of attn_mass is off by the logit's error, by 2^-24 of |x| and of |lse| for
each of the constant's and the product's roundings, and by 2^-21 for the two
exponentials; the sum by 32 + 4 additions of 2^-24 and one for each block of rows.
A rotated value is off by 2^-20 of its pair's length: 21 additions of squares (half of
21 * 2^-24 in the root), the root 2^-22, two products, cos and sin within 2^-21."""
import math
import threading

import numpy as np
import pytest
import torch

import oracle as O
import sparse_attention_decode_step_gb300 as csa
from helpers import need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _np(t):
    return t.detach().cpu().numpy()


# ================================================================ caches in pages
class Paged:
    """Sequences of `lens` entries in pages of a random order; every row that is no
    sequence's entry holds NaN scales, every table entry behind a sequence's pages is no page."""

    def __init__(self, lens, page, seed, m=1, spare=3, keys=0, to=()):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in list(lens) + list(to)]
        total = sum(need) + spare
        cap = max(page, total * page)
        codes = torch.randint(0, 256, (cap, 256), generator=g, dtype=torch.uint8)
        scales = torch.randint(0x20, 0x3C, (cap, 32), generator=g, dtype=torch.uint8)
        order = torch.randperm(total, generator=g)
        table = torch.full((len(need), max([1] + need) + 1), -7, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k].int()
            at += k
        table[:, -1] = 1 << 30
        used = torch.zeros(cap, dtype=torch.bool)
        for b, n in enumerate(lens):
            used[self._rows(table, page, b, n)] = True
        scales[~used] = 0x7F
        self.lens, self.page, self.m = list(lens), page, m
        self.table_host = table[:len(lens)].contiguous()
        self.to_host = table[len(lens):].contiguous()
        kidx = torch.randint(0, 0x7E, (cap, keys), generator=g, dtype=torch.uint8).to(DEV) if keys else None
        ks = torch.rand(cap, generator=g).to(DEV) if keys else None
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.cache = csa.Cache.over(codes.to(DEV), scales.to(DEV), kidx, ks, None, self.seq_len, m)
        self.pages = csa.Pages(self.table_host.to(DEV), page)

    @staticmethod
    def _rows(table, page, b, n):
        j = torch.arange(n)
        return table[b, j // page].long() * page + j % page

    def values(self, b, n=None):
        n = self.lens[b] if n is None else n
        r = self._rows(self.table_host, self.page, b, n).to(DEV)
        return torch.from_numpy(O.fp4_decode_rows(_np(self.cache.codes[r]), _np(self.cache.scales[r]))).reshape(n, 512).to(DEV)


def _sees(off, g, n, pos, m, h):
    """Entries that each row (query, head) of group g sees."""
    i = torch.arange(off[g + 1] - off[g])
    s = torch.full_like(i, n) if pos is None else ((pos[g] + i + 1).div(m, rounding_mode="floor")).clamp(0, n)
    return s.repeat_interleave(h).to(DEV)


def _reference(v, q, sees, sm, prev):
    """out, lse and their bounds (out's but for its storage) of rows q [r][512] over v [n][512]."""
    n, q = v.shape[0], q.double()
    x = sm * (q @ v.T)
    seen = torch.arange(n, device=DEV) < sees[:, None]
    x = torch.where(seen, x, -np.inf)
    pl = prev[1].double()[:, None] if prev is not None else torch.full((q.shape[0], 1), -np.inf, dtype=torch.float64, device=DEV)
    lse = torch.logsumexp(torch.cat([x, pl], 1), 1)
    p = torch.where(seen, torch.exp(x - lse[:, None]), 0.0)
    w = torch.exp(pl - lse[:, None]).nan_to_num(0.0)
    po = torch.where(w > 0, prev[0].double(), 0.0) if prev is not None else torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    out = p @ v + w * po
    d = 32 * 2.0 ** -23 * abs(sm) * (q.abs() @ v.abs().T) + 2.0 ** -25 * abs(sm) * v.abs().sum(1) + 2.0 ** -21
    dmax = torch.where(seen, d, 0.0).amax(1, keepdim=True) if n else torch.zeros(q.shape[0], 1, dtype=torch.float64, device=DEV)
    sums = n / 16 * 2.0 ** -23 + 2 * 152 * 2.0 ** -24 + 2.0 ** -20
    top = p.amax(1, keepdim=True) if n else 0.0
    bound = (2 * dmax + 2.0 ** -11 + 2 * sums) * (p @ v.abs() + w * po.abs()) + 2.0 ** -25 * top * (v.abs().sum(0) if n else 0.0)
    lbound = dmax[:, 0] + sums + 2.0 ** -22 * lse.abs().nan_to_num(0.0, 0.0, 0.0) + 2.0 ** -22
    return out, lse, bound, lbound


def _check(values, off, lens, pos, m, q, out, lse, prev=None, sm=1.0):
    """values(g): the entries of group g's sequence."""
    h = q.shape[1]
    for g, n in enumerate(lens):
        a, e = off[g], off[g + 1]
        if a == e:
            continue
        v, sees = values(g), _sees(off, g, n, pos, m, h)
        for i in range(a, e, 64):                     # (64-bit scores of 64 queries at a time)
            k = min(e, i + 64)
            pr = None if prev is None else (prev[0][i:k].reshape(-1, 512), prev[1][i:k].reshape(-1))
            o, l, bo, bl = _reference(v, q[i:k].reshape(-1, 512), sees[(i - a) * h:(k - a) * h], sm, pr)
            got, gl = out[i:k].reshape(-1, 512).double(), lse[i:k].reshape(-1).double()
            eps = torch.finfo(out.dtype).eps / 2
            off_by = (got - o).abs() - bo - eps * o.abs() - torch.finfo(out.dtype).tiny
            assert torch.isfinite(got).all() and off_by.max() <= 0, (g, n, off_by.max().item())
            inf = torch.isinf(l)
            assert torch.equal(torch.isinf(gl), inf)
            if (~inf).any():
                assert ((gl - l).abs() - bl)[~inf].max() <= 0, (g, n)


def _queries(nq, h, t, seed, scale=0.11):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(nq, h, 512, generator=g) * scale).to(t).to(DEV)


def _prev(nq, h, seed):
    g = torch.Generator().manual_seed(seed)
    po, pl = torch.randn(nq, h, 512, generator=g), torch.randn(nq, h, generator=g) + 6
    po[::2], pl[::2] = float("nan"), float("-inf")       # rows without a partial result: whatever it holds is not read
    return po.to(DEV), pl.to(DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ================================================================ chunk attention
CHUNKS = [
    # heads, page, m, (queries, entries, first position) of each group; position None: the last query sees all
    (16, 16, 1, [(1, 1, None)]),
    (64, 16, 1, [(1, 0, 0)]),
    (64, 32, 2, [(1, 1, 0), (1, 1, 1), (3, 2, 0)]),                     # the first token sees nothing at m = 2
    (1, 16, 1, [(1, 7, None), (3, 128, None), (200, 300, 100)]),
    (5, 64, 1, [(13, 127, None), (1, 0, 0), (26, 1000, None)]),
    (20, 16, 2, [(7, 300, None), (33, 17, None), (2, 4097, None)]),
    (64, 256, 1, [(1, 5003, None), (1, 20000, None)]),
    (64, 64, 1, [(300, 300, 0)]),                                       # a whole prompt
    (64, 16, 4, [(300, 75, 0), (41, 513, None)]),
    (128, 128, 1, [(3, 1025, None), (260, 260, 0)]),
    (16, 512, 3, [(100, 640, None), (1, 640, None)]),
    (8, 16, 1, [(1, 100, None)] * 45),
    (4, 16, 1, [(1, 30 + i % 7, None) for i in range(700)]),
    (2, 32, 2, [(i % 3, (i * 37) % 300, None) for i in range(1100)]),
    (32, 64, 1, [(700, 700, 0), (1, 3000, None), (513, 2000, None)]),
    (8, 16, 1, [(600, 400, -150)]),                                     # a run that begins before the cache does
    (8, 16, 1, [(5, 100, 1 << 30), (70, 90, 40)]),                      # beyond it
    (1, 16, 1, [(2000, 2000, 0)]),
]


def _chunk(case):
    h, page, m, each = CHUNKS[case]
    lens = [n for _c, n, _p in each]
    off = np.concatenate([[0], np.cumsum([c for c, _n, _p in each])]).tolist()
    pos = [max(0, n * m + (m - 1) - c) if p is None else p for c, n, p in each]
    return h, page, m, lens, off, pos


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("with_prev", [False, True])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunk_against_float64(case, with_prev, types):
    h, page, m, lens, off, pos = _chunk(case)
    s = Paged(lens, page, case, m)
    q = _queries(off[-1], h, TYPES[types[0]], case + 100)
    out = torch.full((off[-1] + 2, h, 512), 7.0, dtype=TYPES[types[1]], device=DEV)
    lse = torch.full((off[-1] + 2, h), 7.0, device=DEV)
    prev = _prev(off[-1], h, case + 200) if with_prev else None
    cnt = csa.new_counters()
    csa.chunk_attn(s.cache, csa.Groups(list(range(len(lens))), off), q, out[:-2], lse[:-2], pos=_ints(pos), pages=s.pages,
                   prev=prev, counters=cnt, max_n=max(lens))
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 0, 0]
    assert (out[-2:] == 7).all() and (lse[-2:] == 7).all()
    _check(s.values, off, lens, pos, m, q, out, lse, prev)


@pytest.mark.parametrize("pos", [None, [100, 0, 7]])
def test_chunk_of_contiguous_sequences(pos):
    # no pages: rows from seq_base on; without positions it is the dense attention, bit for bit
    lens, off = [400, 37, 2100], [0, 5, 42, 50]
    cache = csa.Cache(lens, 64, 2, DEV)
    g = torch.Generator().manual_seed(5)
    cache.codes.copy_(torch.randint(0, 256, (cache.cap, 256), generator=g, dtype=torch.uint8))
    cache.scales.copy_(torch.randint(0x20, 0x3C, (cache.cap, 32), generator=g, dtype=torch.uint8))
    cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    q = _queries(50, 20, torch.bfloat16, 6)
    out, lse = torch.zeros(50, 20, 512, device=DEV), torch.zeros(50, 20, device=DEV)
    groups = csa.Groups([0, 1, 2], off)
    csa.chunk_attn(cache, groups, q, out, lse, pos=None if pos is None else _ints(pos))
    torch.cuda.synchronize()

    def values(b):
        r = cache.base_host[b]
        return torch.from_numpy(O.fp4_decode_rows(_np(cache.codes[r:r + lens[b]]), _np(cache.scales[r:r + lens[b]]))).reshape(-1, 512).to(DEV)

    _check(values, off, lens, pos, 2, q, out, lse)
    if pos is None:
        o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
        csa.dense_attn(cache, groups, q, o2, l2)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_chunk_shares_pages_and_respects_lengths():
    # two sequences share their first pages; one is attended only in part
    s = Paged([200, 200], 16, 7)
    s.table_host[1, :8] = s.table_host[0, :8]
    s.pages = csa.Pages(s.table_host.to(DEV), 16)
    q = _queries(9, 64, torch.float16, 8)
    out, lse = torch.zeros(9, 64, 512, device=DEV), torch.zeros(9, 64, device=DEV)
    csa.chunk_attn(s.cache, csa.Groups([0, 1], [0, 4, 9], [133, 200]), q, out, lse, pos=_ints([130, 195]), pages=s.pages)
    torch.cuda.synchronize()
    _check(lambda b: s.values(b)[:[133, 200][b]], [0, 4, 9], [133, 200], [130, 195], 1, q, out, lse)


def test_chunk_out_of_contract():
    s = Paged([200, 100, 300], 32, 9)
    s.table_host[2, 3] = 1000                                     # no page of the cache
    s.pages = csa.Pages(s.table_host.to(DEV), 32)
    seqs, off, length = [0, 3, 1, 2, -1, 1], [0, 3, 5, 6, 8, 9, 11], [201, 5, 100, 300, 4, 99]
    q = _queries(12, 16, torch.bfloat16, 10)
    out = torch.full((12, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((12, 16), 7.0, device=DEV)
    cnt = csa.new_counters()
    pos = [190, 0, 99, 250, 0, 97]
    csa.chunk_attn(s.cache, csa.Groups(seqs, off, length), q, out, lse, pos=_ints(pos), pages=s.pages, counters=cnt)
    torch.cuda.synchronize()
    c = _np(cnt).tolist()
    assert c[0] == c[1] == c[3] == 0 and c[2] >= 4                # groups 0, 1 and 4; the page once or more
    for g in (2, 5):
        _check(lambda _g: s.values(seqs[g], length[g]), [off[g], off[g + 1]], [length[g]], [pos[g]], 1, q, out, lse)
    for a, e in ((0, 5), (8, 9), (11, 12)):
        assert (out[a:e] == 7).all() and (lse[a:e] == 7).all()
    # a sequence longer than its pages reach, and offsets that fall
    long = csa.Cache.over(s.cache.codes, s.cache.scales, None, None, None, _ints([5000]), 1)
    out.fill_(7)
    cnt.zero_()
    few = csa.Pages(s.table_host[:1].contiguous().to(DEV), 32)
    csa.chunk_attn(long, csa.Groups([0], [0, 12]), q, out, lse, pos=_ints([4988]), pages=few, max_n=5000, counters=cnt)
    csa.chunk_attn(s.cache, csa.Groups([1, 0, 1], [0, 5, 3, 12]), q, out, lse, pos=_ints([90, 0, 0]), pages=s.pages, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 3, 0]
    _check(lambda _g: s.values(1), [0, 5], [100], [90], 1, q, out, lse)
    assert (out[5:] == 7).all()


def test_chunk_keeps_later_tokens_out():
    # entries behind what a row tile sees hold NaN: only the rows that see them may
    s = Paged([600], 16, 11)
    rows = s._rows(s.table_host, 16, 0, 600)[300:]
    s.cache.scales[rows.to(DEV)] = 0x7F
    q = _queries(600, 64, torch.bfloat16, 12)
    out, lse = torch.zeros(600, 64, 512, device=DEV), torch.zeros(600, 64, device=DEV)
    csa.chunk_attn(s.cache, csa.Groups([0], [0, 600]), q, out, lse, pos=_ints([0]), pages=s.pages)
    torch.cuda.synchronize()
    _check(lambda _g: s.values(0)[:300], [0, 300], [300], [0], 1, q[:300], out[:300], lse[:300])
    assert torch.isnan(out[300:]).any()


def test_chunk_merges_a_window_like_the_sparse_step():
    # an earlier partial result in place (out is prev_out, lse is prev_lse), twice on one workspace
    s = Paged([3000, 40], 64, 13)
    q = _queries(8, 64, torch.bfloat16, 14)
    po, pl = (t.nan_to_num(0.0, neginf=1.0) for t in _prev(8, 64, 15))
    out, lse = po.clone(), pl.clone()
    ws = csa.workspace(csa.dense_workspace_size(2, 8, 64, 3000))
    csa.chunk_attn(s.cache, csa.Groups([0, 1], [0, 3, 8]), q, out, lse, pos=_ints([2997, 35]), pages=s.pages, prev=(out, lse), ws=ws, max_n=3000)
    torch.cuda.synchronize()
    _check(s.values, [0, 3, 8], [3000, 40], [2997, 35], 1, q, out, lse, (po, pl))
    again, l2 = po.clone(), pl.clone()
    csa.chunk_attn(s.cache, csa.Groups([0, 1], [0, 3, 8]), q, again, l2, pos=_ints([2997, 35]), pages=s.pages, prev=(again, l2), ws=ws, max_n=3000)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("sm", [-0.5, 0.0, 3.0])
def test_chunk_other_scales(sm):
    s = Paged([300, 2000], 16, 17)
    q = _queries(40, 32, torch.bfloat16, 18, 0.3)
    out, lse = torch.zeros(40, 32, 512, device=DEV), torch.zeros(40, 32, device=DEV)
    csa.chunk_attn(s.cache, csa.Groups([0, 1], [0, 10, 40]), q, out, lse, pos=_ints([290, 1970]), pages=s.pages, sm_scale=sm)
    torch.cuda.synchronize()
    _check(s.values, [0, 10, 40], [300, 2000], [290, 1970], 1, q, out, lse, sm=sm)


# ================================================================ attention weights
def _mass_reference(v, q, lse, sees, sm):
    q, l = q.double(), lse.double()[:, None]
    x = sm * (q @ v.T)
    seen = (torch.arange(v.shape[0], device=DEV) < sees[:, None]) & torch.isfinite(l)
    p = torch.where(seen, torch.exp(x - l), 0.0)
    d = 32 * 2.0 ** -23 * abs(sm) * (q.abs() @ v.abs().T) + 2.0 ** -25 * abs(sm) * v.abs().sum(1) + 2.0 ** -21
    d = d + 2.0 ** -23 * (x.abs() + l.abs()) + (36 + q.shape[0] / 128) * 2.0 ** -24
    return p.sum(0), torch.where(seen, p * d, 0.0).sum(0) + 2.0 ** -120


def _check_mass(values, off, lens, pos, m, q, lse, prev, decay, mass, sm=1.0, seqs=None):
    h = q.shape[1]
    for g, n in enumerate(lens):
        b = g if seqs is None else seqs[g]
        a, e = off[g], off[g + 1]
        want = torch.zeros(n, dtype=torch.float64, device=DEV)
        bound = torch.full((n,), 2.0 ** -120, dtype=torch.float64, device=DEV)
        v, sees = values(g), _sees(off, g, n, pos, m, h)
        for i in range(a, e, 64):
            k = min(e, i + 64)
            w, d = _mass_reference(v, q[i:k].reshape(-1, 512), lse[i:k].reshape(-1), sees[(i - a) * h:(k - a) * h], sm)
            want += w
            bound += d + (e - a) * h / 128 * 2.0 ** -24 * w
        if prev is not None:
            want += decay * prev[b, :n].double()
            bound += 2.0 ** -23 * abs(decay) * prev[b, :n].double().abs()
        got = mass[b, :n].double()
        bound += 2.0 ** -23 * want.abs()
        far = (got - want).abs() - bound
        assert n == 0 or (torch.isfinite(got).all() and far.max() <= 0), (g, n, far.max().item())


@pytest.mark.parametrize("types", ["bf16", "f16"])
@pytest.mark.parametrize("how", ["alone", "prev", "in place"])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_mass_against_float64(case, how, types):
    h, page, m, lens, off, pos = _chunk(case)
    s = Paged(lens, page, case + 40, m)
    q = _queries(off[-1], h, TYPES[types], case + 100)
    g = torch.Generator().manual_seed(case)
    lse = (torch.randn(off[-1], h, generator=g) + 6).to(DEV)
    if off[-1] > 1:
        lse[1, 0], lse[0, -1] = -math.inf, math.inf       # rows that add nothing, whatever their queries hold
        q[1, 0] = float("nan")
    ld = max(lens) + 5
    mass = torch.full((len(lens), ld), 7.0, device=DEV)
    prev = torch.rand(len(lens), ld, generator=g).to(DEV) * 3 if how != "alone" else None
    if how == "in place":
        mass = prev.clone()
    cnt = csa.new_counters()
    csa.attn_mass(s.cache, csa.Groups(list(range(len(lens))), off), q, lse, mass, pos=_ints(pos), pages=s.pages,
                  prev=mass if how == "in place" else prev, decay=0.75, counters=cnt, max_n=max(lens))
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 0, 0]
    q = torch.where(torch.isfinite(lse)[..., None], q, 0.0)
    _check_mass(s.values, off, lens, pos, m, q, lse, prev, 0.75, mass)
    for b, n in enumerate(lens):
        assert torch.equal(mass[b, n:], prev[b, n:] if how == "in place" else torch.full_like(mass[b, n:], 7.0))


def test_mass_of_the_attention_adds_up():
    # with the attention's own lse, without a partial result, each row gives 1 in all
    s = Paged([5000, 77], 64, 21)
    q = _queries(40, 64, torch.bfloat16, 22)
    groups, pos = csa.Groups([0, 1], [0, 30, 40]), _ints([4970, 67])
    out, lse = torch.zeros(40, 64, 512, device=DEV), torch.zeros(40, 64, device=DEV)
    csa.chunk_attn(s.cache, groups, q, out, lse, pos=pos, pages=s.pages)
    mass = torch.zeros(2, 5000, device=DEV)
    csa.attn_mass(s.cache, groups, q, lse, mass, pos=pos, pages=s.pages)
    torch.cuda.synchronize()
    assert (mass.double().sum(1).cpu() / 64 - torch.tensor([30.0, 10.0])).abs().max() < 1e-3
    _check_mass(s.values, [0, 30, 40], [5000, 77], [4970, 67], 1, q, lse, None, 0.0, mass)


def test_mass_more_blocks_than_parts():
    # 256 MB of parts hold 32 blocks at a million entries: 70 blocks of one group go in turns
    n, nq, h = 700, 70, 128
    s = Paged([n, 50], 64, 23)
    q = _queries(nq + 1, h, torch.bfloat16, 24)
    lse = torch.full((nq + 1, h), 7.0, device=DEV)
    prev = torch.rand(2, 1 << 20, device=DEV)
    mass = torch.zeros(2, 1 << 20, device=DEV)
    csa.attn_mass(s.cache, csa.Groups([1, 0], [0, 1, nq + 1]), q, lse, mass, pos=_ints([49, n - nq]), pages=s.pages, prev=prev, decay=0.5)
    torch.cuda.synchronize()
    _check_mass(lambda g: s.values(1 - g), [0, 1, nq + 1], [50, n], [49, n - nq], 1, q, lse, prev, 0.5, mass, seqs=[1, 0])
    assert not mass[0, n:].any() and not mass[1, 50:].any()


@pytest.mark.parametrize("lens", [[1], [5, 3, 130], [1000, 7]])
def test_mass_of_contiguous_sequences(lens):
    # rows from seq_base on, of any alignment; a cache smaller than a tile
    base = [0]
    for n in lens:
        base.append(base[-1] + n)
    cap = -(-base[-1] // 8) * 8
    g = torch.Generator().manual_seed(27)
    codes = torch.randint(0, 256, (cap, 256), generator=g, dtype=torch.uint8)
    scales = torch.randint(0x20, 0x3C, (cap, 32), generator=g, dtype=torch.uint8)
    cache = csa.Cache.over(codes.to(DEV), scales.to(DEV), None, None, torch.tensor(base, device=DEV), _ints(lens), 1)
    off = [0] + [3 * (b + 1) for b in range(len(lens))]
    q = _queries(off[-1], 20, torch.bfloat16, 28)
    lse = torch.full((off[-1], 20), 5.0, device=DEV)
    mass = torch.zeros(len(lens), max(lens), device=DEV)
    csa.attn_mass(cache, csa.Groups(list(range(len(lens))), off), q, lse, mass)
    torch.cuda.synchronize()

    def values(b):
        r = slice(base[b], base[b + 1])
        return torch.from_numpy(O.fp4_decode_rows(codes[r].numpy(), scales[r].numpy())).reshape(-1, 512).to(DEV)

    _check_mass(values, off, lens, None, 1, q, lse, None, 0.0, mass)


@pytest.mark.parametrize("far", [-150.0, 150.0])
@pytest.mark.parametrize("spread", [0.0, 90.0])
def test_mass_of_logits_far_from_zero(far, spread):
    # every value of the cache near 3, every query near far / (3 * 512): logits, and so lse, far from zero;
    # rows that lie far from each other; columns without a row (5 and 65 of 16 and 80)
    s = Paged([700, 100], 16, 29)
    g = torch.Generator().manual_seed(30)
    nib = torch.randint(4, 7, s.cache.codes.shape + (2,), generator=g, dtype=torch.uint8)
    s.cache.codes.copy_(nib[..., 0] | (nib[..., 1] << 4))
    s.cache.scales.fill_(0x38)                                    # 1.0
    at = torch.full((14,), far)
    at[1::3] -= math.copysign(spread, far)
    q = ((at / 1536)[:, None, None] + 0.002 * torch.randn(14, 5, 512, generator=g)).to(torch.float16).to(DEV)
    groups, pos = csa.Groups([1, 0], [0, 1, 14]), _ints([99, 687])
    out, lse = torch.zeros(14, 5, 512, device=DEV), torch.zeros(14, 5, device=DEV)
    csa.chunk_attn(s.cache, groups, q, out, lse, pos=pos, pages=s.pages)
    mass = torch.zeros(2, 700, device=DEV)
    csa.attn_mass(s.cache, groups, q, lse, mass, pos=pos, pages=s.pages)
    torch.cuda.synchronize()
    assert lse[0, 0].abs() > 100
    _check_mass(lambda i: s.values(1 - i), [0, 1, 14], [100, 700], [99, 687], 1, q, lse, None, 0.0, mass, seqs=[1, 0])


def test_mass_out_of_contract():
    s = Paged([200, 100, 300], 32, 25)
    seqs, off = [0, 0, 3, 2, 2], [0, 3, 5, 6, 8, 9]               # groups 1 and 4: again; 2: no sequence
    q = _queries(9, 16, torch.bfloat16, 26)
    lse = torch.full((9, 16), 6.0, device=DEV)
    mass = torch.full((3, 300), 7.0, device=DEV)
    cnt = csa.new_counters()
    csa.attn_mass(s.cache, csa.Groups(seqs, off), q, lse, mass, pages=s.pages, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 3, 0]
    _check_mass(lambda g: s.values(0), [0, 3], [200], None, 1, q, lse, None, 0.0, mass)
    _check_mass(lambda g: s.values(2), [6, 8], [300], None, 1, q, lse, None, 0.0, mass, seqs=[2])
    assert (mass[1] == 7).all() and (mass[0, 200:] == 7).all()
    # offsets that fall, no queries at all (what was there decays), a page outside the cache
    cnt.zero_()
    csa.attn_mass(s.cache, csa.Groups([1, 0, 2], [0, 5, 3, 9]), q, lse, mass.fill_(7), pages=s.pages, counters=cnt)
    csa.attn_mass(s.cache, csa.Groups([2], [0, 0]), q[:0], lse[:0], mass, pages=s.pages, prev=mass, decay=0.5, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 2, 0]
    _check_mass(lambda g: s.values(1), [0, 5], [100], None, 1, q, lse, None, 0.0, mass, seqs=[1])
    assert (mass[0] == 7).all() and (mass[2] == 3.5).all()
    s.table_host[1, 1] = -1
    csa.attn_mass(s.cache, csa.Groups([1], [0, 9]), q, lse, mass, pages=csa.Pages(s.table_host.to(DEV), 32), counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist()[2] > 2


# ================================================================ eviction
def _kept(mass, n, keep, first, last):
    if n <= keep:
        return list(range(n))
    inner = sorted(range(first, n - last), key=lambda j: (-(mass[j] if mass[j] == mass[j] else -math.inf), j))
    return sorted(list(range(first)) + list(range(n - last, n)) + inner[:keep - first - last])


EVICTS = [
    # page, keys, lens, keep, first, last
    (16, 64, [1, 40, 17, 0], 16, 0, 0),
    (16, 0, [100, 33], 33, 1, 32),
    (32, 128, [4099, 1024, 1000, 2048, 1025], 1024, 4, 128),
    (64, 64, [70000, 300, 12345], 9000, 64, 1000),
    (16, 128, [300000], 5000, 10, 10),
    (16, 0, [20 + 3 * i for i in range(130)], 37, 2, 5),
    (128, 128, [513], 1, 0, 1),
    (128, 64, [100], 1 << 20, 5, 7),
    (32, 0, [12000 - 50 * i for i in range(100)], 5000, 100, 200),
]


def _weights(b, n, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(2 * torch.randn(b, n, generator=g))
    w[:, ::3] = torch.randint(0, 4, (b, len(range(0, n, 3))), generator=g).float()        # ties, zeros
    w[:, 1::17] = -0.0
    w[:, 5::31], w[:, 7::41], w[:, 9::53] = float("nan"), math.inf, -math.inf
    return w


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict_keeps_the_heaviest(case, paged):
    page, keys, lens, keep, first, last = EVICTS[case]
    k = [min(n, keep) for n in lens]
    s = Paged(lens, page, case + 60, keys=keys, to=k)
    w = _weights(len(lens), max(lens), case)
    mass = w.to(DEV)
    wide = keep if keep < 1 << 19 else max(lens) + 3
    kept = torch.full((len(lens), max(keep, wide)), -5, dtype=torch.int32, device=DEV)
    out = torch.full((len(lens), max(keep, wide)), -5.0, device=DEV)
    cnt = csa.new_counters()
    c = s.cache
    if paged:
        to = csa.Cache.over(c.codes, c.scales, c.kidx, c.kscale, None, torch.zeros_like(s.seq_len), 1)
        to_pages = csa.Pages(s.to_host.to(DEV), page)
        rows = [s._rows(s.to_host, page, b, n) for b, n in enumerate(k)]
    else:
        to = csa.Cache(k, keys or 64, 1, DEV)
        if not keys:
            to = csa.Cache.over(to.codes, to.scales, None, None, to.seq_base, to.seq_len, 1)
        to_pages = None
        base = np.cumsum([0] + [-(-n // 8) * 8 for n in k])
        rows = [torch.arange(n) + int(base[b]) for b, n in enumerate(k)]
    before = c.codes.clone()
    csa.cache_evict(c, to, mass, keep, kept, out, first=first, last=last, pages=s.pages, to_pages=to_pages, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 0, 0]
    assert _np(to.seq_len).tolist() == k and _np(s.seq_len).tolist() == lens
    changed = torch.zeros(c.codes.shape[0], dtype=torch.bool)
    for b, n in enumerate(lens):
        want = torch.tensor(_kept(w[b].tolist(), n, keep, first, last), dtype=torch.long)
        assert torch.equal(kept[b, :k[b]].cpu().long(), want)
        assert (kept[b, k[b]:] == -5).all() and (out[b, k[b]:] == -5).all()
        assert torch.equal(out[b, :k[b]].cpu().view(torch.int32), w[b][want].view(torch.int32))
        src, dst = s._rows(s.table_host, page, b, n)[want].to(DEV), rows[b].to(DEV)
        for name in ("codes", "scales") + (("kidx", "kscale") if keys else ()):
            assert torch.equal(getattr(to, name)[dst], getattr(c, name)[src]), name
        if paged:
            changed[rows[b]] = True
    assert torch.equal(c.codes[~changed.to(DEV)], before[~changed.to(DEV)])


def test_evict_some_sequences_in_place_of_their_lengths():
    # the new length goes where the old one was; a sequence listed twice; the others stay
    lens = [500, 300, 400]
    s = Paged(lens, 16, 71, to=[64, 64, 64])
    w = _weights(3, 500, 72)
    kept = torch.zeros(3, 64, dtype=torch.int32, device=DEV)
    csa.cache_evict(s.cache, s.cache, w.to(DEV), 64, kept, seq=_ints([2, 0, 2]), first=3, last=9, pages=s.pages,
                    to_pages=csa.Pages(s.to_host.to(DEV), 16))
    torch.cuda.synchronize()
    assert _np(s.seq_len).tolist() == [64, 300, 64]
    for i, b in enumerate((2, 0, 2)):
        want = _kept(w[b].tolist(), lens[b], 64, 3, 9)
        assert _np(kept[i]).tolist() == want
        src = s._rows(s.table_host, 16, b, lens[b])[torch.tensor(want)].to(DEV)
        assert torch.equal(s.cache.codes[s._rows(s.to_host, 16, b, 64).to(DEV)], s.cache.codes[src])


def test_rows_past_two_gigabytes_of_codes():
    # pages at the far end of a cache of 17 million rows give what a small cache gives
    s = Paged([900, 130], 64, 75, to=[50, 50])
    cap, shift = 17 << 20, (17 << 20) // 64 - 40
    codes = torch.empty(cap, 256, dtype=torch.uint8, device=DEV)
    scales = torch.empty(cap, 32, dtype=torch.uint8, device=DEV)
    n = s.cache.codes.shape[0]
    assert n <= 40 * 64
    codes[shift * 64:shift * 64 + n], scales[shift * 64:shift * 64 + n] = s.cache.codes, s.cache.scales
    big = csa.Cache.over(codes, scales, None, None, None, s.seq_len, 1)
    q = _queries(40, 64, torch.bfloat16, 76)
    groups, pos = csa.Groups([0, 1], [0, 30, 40]), _ints([870, 120])
    got = []
    for cache, add in ((s.cache, 0), (big, shift)):
        pages, to = csa.Pages((s.table_host + add).to(DEV), 64), csa.Pages((s.to_host + add).to(DEV), 64)
        out, lse, mass = torch.zeros(40, 64, 512, device=DEV), torch.zeros(40, 64, device=DEV), torch.zeros(2, 900, device=DEV)
        csa.chunk_attn(cache, groups, q, out, lse, pos=pos, pages=pages)
        csa.attn_mass(cache, groups, q, lse, mass, pos=pos, pages=pages)
        kept = torch.zeros(2, 50, dtype=torch.int32, device=DEV)
        short = csa.Cache.over(cache.codes, cache.scales, None, None, None, torch.zeros_like(s.seq_len), 1)
        csa.cache_evict(cache, short, mass, 50, kept, pages=pages, to_pages=to)
        x = torch.zeros(100, 512, device=DEV)
        csa.cache_read(short, to.rows(torch.arange(2, device=DEV).repeat_interleave(50), torch.arange(50, device=DEV).repeat(2)), x)
        got.append((out, lse, mass, kept, x))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_evict_out_of_contract():
    lens = [500, 300, 400, -1, 600]
    s = Paged([max(n, 0) for n in lens], 16, 73)
    s.seq_len.copy_(_ints(lens))
    to = csa.Cache([64, 64, 40, 64, 64], 64, 1, DEV)
    to = csa.Cache.over(to.codes, to.scales, None, None, to.seq_base, to.seq_len, 1)
    s.table_host[1, 2] = 1 << 20                                      # no page: its 16 entries are not copied
    w = torch.rand(5, 600)
    kept = torch.full((7, 64), -5, dtype=torch.int32, device=DEV)
    cnt = csa.new_counters()
    csa.cache_evict(s.cache, to, w.to(DEV), 64, kept, seq=_ints([0, 1, 2, 3, 4, 5, -1]), first=64, max_n=500,
                    pages=csa.Pages(s.table_host.to(DEV), 16), counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 1, 4 + 16, 0]                     # room of 2; 3, 4 (past max_n), 5 and -1; the page
    assert _np(to.seq_len).tolist() == [64, 64, 0, 0, 0]
    assert (kept[2:] == -5).all()
    assert _np(kept[0]).tolist() == list(range(64))
    assert not to.codes[64 + 32:64 + 48].any()


# ================================================================ norm and rotation
def _rope_reference(x, weight, eps, pos, freq, halves):
    x = x.double().cpu()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double().cpu()
    size = y.abs()
    half = 0 if freq is None else freq.shape[0]
    if half:
        # the angle's fraction of a turn from whole numbers: freq is a 24-bit number times a power of two
        inv = int("28be60db9391054a7f09d5f47d4d377036d8a5664f10e4107f9458eaf7aef158", 16)     # 2^256 / (2 pi) 
        f = [math.frexp(v) for v in freq.double().tolist()]
        turn = torch.empty(len(pos), half, dtype=torch.float64)
        for p, (mant, e) in enumerate(f):
            k = (int(mant * 2 ** 24) * inv >> (24 - e)) if e <= 24 else int(mant * 2 ** 24) * inv << (e - 24)
            turn[:, p] = torch.tensor([(t * k % (1 << 256) >> 203) / 2 ** 53 for t in pos.tolist()], dtype=torch.float64)
        c, s = torch.cos(2 * math.pi * turn), torch.sin(2 * math.pi * turn)
        if x.dim() == 3:
            c, s = c[:, None], s[:, None]
        z = y[..., 512 - 2 * half:]
        u, v = (z[..., :half], z[..., half:]) if halves else (z[..., 0::2], z[..., 1::2])
        r = torch.hypot(u, v)
        u, v = u * c - v * s, u * s + v * c
        join = (lambda a, b: torch.cat([a, b], -1)) if halves else (lambda a, b: torch.stack([a, b], -1).flatten(-2))
        y = torch.cat([y[..., :512 - 2 * half], join(u, v)], -1)
        size = torch.cat([size[..., :512 - 2 * half], join(r, r)], -1)
    return y, size


ROPES = [
    # tokens, heads (0: [n][512]), rotated, type, out, extra
    (1, 1, 64, "bf16", "bf16", 0),
    (1, 0, 0, "f32", "f32", 0),
    (3, 16, 64, "bf16", "bf16", 8),
    (37, 5, 512, "f16", "f32", 0),
    (130, 64, 64, "bf16", "bf16", 0),
    (2000, 0, 64, "f32", "bf16", 64),
    (1001, 3, 48, "bf16", "f16", 16),
    (257, 128, 16, "f16", "f16", 0),
    (5, 20, 336, "f32", "f32", 4),
    (20000, 1, 128, "bf16", "f32", 0),
]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("case", range(len(ROPES)))
def test_norm_rope_against_float64(case, weighted, halves):
    n, h, rot, t, to, extra = ROPES[case]
    g = torch.Generator().manual_seed(case)
    wide = torch.randn(n, max(1, h) * 512 + extra, generator=g).mul(torch.exp2(torch.randint(-6, 7, (n, 1), generator=g).float())).to(TYPES[t])
    wide[n // 2] = 0                                                     # a row of zeros
    wd = wide.to(DEV)
    shape = (lambda v: v[:, :max(1, h) * 512].unflatten(1, (h, 512)) if h else v[:, :512])
    x = shape(wd)
    pos = torch.randint(-1000, 1 << 20, (n,), generator=g, dtype=torch.int32)
    freq = (10000.0 ** (-torch.arange(rot // 2).double() / max(1, rot // 2))).float() if rot else None
    w = torch.randn(512, generator=g) if weighted else None
    out = torch.full((n, max(1, h) * 512 + 8), 7.0, dtype=TYPES[to], device=DEV)
    csa.norm_rope(x, shape(out), weight=None if w is None else w.to(DEV), eps=1e-5, pos=pos.to(DEV) if rot else None,
                  inv_freq=None if freq is None else freq.to(DEV), halves=halves)
    torch.cuda.synchronize()
    y, size = _rope_reference(shape(wide), w, 1e-5, pos, freq, halves)
    got = shape(out).double().cpu()
    eps = torch.finfo(TYPES[to]).eps / 2
    far = (got - y).abs() - size * 2.0 ** -20 - eps * y.abs() * (1 + 2.0 ** -10) - torch.finfo(TYPES[to]).tiny * 2 * eps
    assert torch.isfinite(got).all() and far.max() <= 0, far.max().item()
    assert (out[:, max(1, h) * 512:] == 7).all()


def test_norm_rope_in_place_far_positions_and_back():
    n, h = 64, 20
    g = torch.Generator().manual_seed(3)
    x = torch.randn(n, h, 512, generator=g)
    pos = torch.cat([torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), 1 << 30, 1 << 24]),
                     torch.randint(-(1 << 31), (1 << 31) - 1, (n - 7,), generator=g)]).to(torch.int32)
    freq = (500000.0 ** (-torch.arange(64).double() / 64)).float()
    xd = x.to(DEV)
    csa.norm_rope(xd, xd, pos=pos.to(DEV), inv_freq=freq.to(DEV), halves=True, eps=0.0)
    torch.cuda.synchronize()
    y, size = _rope_reference(x, None, 0.0, pos, freq, True)
    assert ((xd.double().cpu() - y).abs() - size * 2.0 ** -20).max() <= 0
    # the opposite position turns it back (a normed row has norm sqrt(512) already: 2^-22 of the squares' mean)
    back = torch.empty_like(xd)
    safe = pos.clone()
    safe[safe == -(1 << 31)] = 0
    csa.norm_rope(x.to(DEV), xd, pos=safe.to(DEV), inv_freq=freq.to(DEV), halves=True, eps=0.0)
    csa.norm_rope(xd, back, pos=(-safe).to(DEV), inv_freq=freq.to(DEV), halves=True, eps=0.0)
    torch.cuda.synchronize()
    flat, _ = _rope_reference(x, None, 0.0, pos, None, True)
    pair = torch.hypot(flat[..., 384:448], flat[..., 448:])
    near = (back.double().cpu() - flat).abs()
    assert (near[..., 384:] - torch.cat([pair, pair], -1) * 2.0 ** -18).max() <= 0 and (near[..., :384] - flat[..., :384].abs() * 2.0 ** -19).max() <= 0


# ================================================================ together
def _serve(s, x, w, freq, q_raw, pos_q, groups, pos, rows, state):
    """A chunk's step: its latents normed, turned, written; its queries normed, turned; attended; weighed."""
    csa.norm_rope(x, state["x"], weight=w, pos=pos_q, inv_freq=freq)
    csa.cache_write(s.cache, rows, state["x"])
    csa.norm_rope(q_raw, state["q"], pos=pos_q, inv_freq=freq)
    csa.chunk_attn(s.cache, groups, state["q"], state["out"], state["lse"], pos=pos, pages=s.pages, sm_scale=512 ** -0.5, ws=state["ws"], max_n=1200)
    csa.attn_mass(s.cache, groups, state["q"], state["lse"], state["mass"], pos=pos, pages=s.pages, prev=state["mass"], decay=0.5,
                  sm_scale=512 ** -0.5, ws=state["mws"], max_n=1200)


@pytest.mark.parametrize("how", ["eager", "graph", "other stream"])
def test_serving_a_chunk_then_evicting(how):
    lens, new = [1000, 130, 37], [40, 1, 37]
    s = Paged(lens, 16, 81, to=[100] * 3)
    h, nq = 64, sum(new)
    off = [0, 40, 41, 78]
    g = torch.Generator().manual_seed(82)
    x = torch.randn(nq, 512, generator=g).to(torch.bfloat16).to(DEV)
    q_raw = torch.randn(nq, h, 512, generator=g).to(torch.bfloat16).to(DEV)
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(DEV)
    freq = (10000.0 ** (-torch.arange(32).double() / 32)).float().to(DEV)
    at = torch.cat([torch.arange(n - c, n) for n, c in zip(lens, new)]).to(DEV)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(new)).to(DEV)
    rows = s.pages.rows(seq, at)
    assert torch.equal(rows.cpu(), torch.cat([s._rows(s.table_host, 16, b, n)[n - c:] for b, (n, c) in enumerate(zip(lens, new))]))
    groups, pos = csa.Groups([0, 1, 2], off), _ints([n - c for n, c in zip(lens, new)])
    state = {"x": torch.zeros_like(x), "q": torch.zeros_like(q_raw), "out": torch.zeros(nq, h, 512, device=DEV),
             "lse": torch.zeros(nq, h, device=DEV), "mass": torch.zeros(3, 1200, device=DEV),
             "ws": csa.workspace(csa.dense_workspace_size(3, nq, h, 1200)), "mws": csa.workspace(csa.mass_workspace_size(3, 3, nq, h, 1200))}
    args = (s, x, w, freq, q_raw, at.int(), groups, pos, rows, state)
    kept = torch.zeros(3, 100, dtype=torch.int32, device=DEV)
    short = csa.Cache.over(s.cache.codes, s.cache.scales, None, None, None, torch.zeros_like(s.seq_len), 1)
    to_pages = csa.Pages(s.to_host.to(DEV), 16)
    m2 = torch.zeros(3, 100, device=DEV)
    ews = csa.workspace(csa.evict_workspace_size(3, 1200))
    prev = torch.rand(3, 1200, generator=g).to(DEV)

    def all_of_it():
        state["mass"].copy_(prev)
        _serve(*args)
        csa.cache_evict(s.cache, short, state["mass"], 100, kept, m2, first=4, last=20, pages=s.pages, to_pages=to_pages, ws=ews)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    if how == "eager":
        all_of_it()
    elif how == "other stream":
        with torch.cuda.stream(stream):
            all_of_it()
    else:
        with torch.cuda.stream(stream):
            all_of_it()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            all_of_it()
        for t in (state["out"], state["mass"], kept, m2, short.seq_len):
            t.zero_()
        for _ in range(2):
            graph.replay()
    torch.cuda.synchronize()
    v = {b: s.values(b) for b in range(3)}
    y, _ = _rope_reference(x, w, 1e-6, at.cpu(), freq.cpu(), False)
    assert (state["x"].double().cpu() - y).abs().max() <= 2.0 ** -8 * y.abs().max()
    stored = torch.zeros(nq, 512, device=DEV)
    csa.cache_read(s.cache, rows, stored)
    assert torch.equal(stored.double(), torch.cat([v[b][n - c:] for b, (n, c) in enumerate(zip(lens, new))]))
    pos_host = [n - c for n, c in zip(lens, new)]
    _check(lambda b: v[b], off, lens, pos_host, 1, state["q"], state["out"], state["lse"], sm=512 ** -0.5)
    _check_mass(lambda b: v[b], off, lens, pos_host, 1, state["q"], state["lse"], prev, 0.5, state["mass"], sm=512 ** -0.5)
    for b, n in enumerate(lens):
        want = _kept(state["mass"][b].tolist(), n, 100, 4, 20)
        assert _np(kept[b, :len(want)]).tolist() == want
    # the cut sequences are attended like any other: one more token, every entry visible
    q1 = state["q"][[39, 40, 77]].contiguous()
    out, lse = torch.zeros(3, h, 512, device=DEV), torch.zeros(3, h, device=DEV)
    k = [min(n, 100) for n in lens]
    csa.chunk_attn(short, csa.Groups([0, 1, 2], [0, 1, 2, 3]), q1, out, lse, pos=_ints([n - 1 for n in k]), pages=to_pages)
    torch.cuda.synchronize()
    _check(lambda b: v[b][torch.tensor(_kept(state["mass"][b].tolist(), lens[b], 100, 4, 20), device=DEV)], [0, 1, 2, 3], k,
           [n - 1 for n in k], 1, q1, out, lse)


def test_calls_from_two_threads_agree():
    s = Paged([700, 900], 32, 91)
    q = _queries(6, 64, torch.bfloat16, 92)
    groups, pos = csa.Groups([0, 1], [0, 2, 6]), _ints([698, 896])
    got = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out, lse = torch.zeros(6, 64, 512, device=DEV), torch.zeros(6, 64, device=DEV)
                mass = torch.zeros(2, 900, device=DEV)
                csa.chunk_attn(s.cache, groups, q, out, lse, pos=pos, pages=s.pages)
                csa.attn_mass(s.cache, groups, q, lse, mass, pos=pos, pages=s.pages)
            torch.cuda.current_stream().synchronize()
            got.append((out, lse, mass))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 2 and all(torch.equal(a, b) for a, b in zip(*got))

"""Cache rows by number and dense attention of query groups against float64.

Rows: bytes equal the oracle's, values read back are exact in every type.
Dense attention: the bound of each output is summed from its roundings --
  the logit: 32 fp32 additions of 16-term products, each off by at most 2^-23 of
  the sum of |q v| (an accumulator that truncates), q's f16 subnormals (2^-25
  each), and 2^-22 of the hardware exponential;
  a weight: f16, half a step 2^-11, or 2^-25 absolute below f16's normals (the
  largest weight of a row is at least 1 before normalisation);
  the sum over n entries: n / 16 fp32 additions, 2^-23 each, and the joining of
  at most 152 parts (2^-24 each, twice);
  the output type: half a step of what is stored."""
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


# ================================================================ rows
def _oracle_rows(x, key):
    n = x.shape[0]
    d = key.shape[1] if key is not None else 64
    k = key if key is not None else torch.zeros(n, d)
    codes, scales, kidx, ksc, _x, _ = O.append(x.float().numpy()[None], None, k.float().numpy()[None], 1)
    return codes, scales, kidx, ksc


def _latents(n, t, seed):
    """Rows of several magnitudes, ties of the FP4 grid, a zero row, saturating groups."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 512, generator=g) * torch.exp2(torch.randint(-12, 9, (n, 32), generator=g).float()).repeat_interleave(16, 1)
    if n > 2:
        x[1] = 0
        x[2] = torch.randint(-24, 25, (512,), generator=g).float() / 4     # k / 4: midpoints among them
        x[2, ::16] = 6
    if n > 4:
        x[4, :16] = 3000.0
        x[4, 16] = 2688.0
    return x.to(t)


@pytest.mark.parametrize("n,t,d_idx,extra", [(1, "bf16", 128, 0), (3, "f16", 64, 8), (37, "bf16", 128, 136),
                                              (8, "f32", 64, 4), (1001, "bf16", 0, 64), (4099, "f32", 128, 0),
                                              (4099, "f16", 0, 0), (20011, "bf16", 64, 64)])
def test_write_bytes_and_read_values(n, t, d_idx, extra):
    dt, d = TYPES[t], d_idx or 64
    cap = -(-(2 * n + 5) // 8) * 8
    g = torch.Generator().manual_seed(n)
    cache = csa.Cache([cap], d, 1, DEV)
    cache.kidx.fill_(0x11)
    wide = torch.zeros(n, 512 + extra + d, dtype=dt)
    wide[:, :512] = _latents(n, dt, n)
    wide[:, 512 + extra:] = (torch.randn(n, d, generator=g) * 3).to(dt)
    rows = torch.randperm(cap, generator=g)[:n]
    wd = wide.to(DEV)
    off = 512 + extra
    # (a key slice must begin on 16 bytes)
    key = wd[:, off:] if d_idx else None
    cnt = csa.new_counters()
    csa.cache_write(cache, rows.to(DEV), wd[:, :512], key, counters=cnt)
    xb = torch.full((n, 512 + extra), 7.0, dtype=dt, device=DEV)
    kb = torch.zeros(n, d, device=DEV)
    csa.cache_read(cache, rows.to(DEV), xb[:, :512], kb if d_idx else None, counters=cnt)
    torch.cuda.synchronize()
    codes, scales, kidx, ksc = _oracle_rows(wide[:, :512], wide[:, off:] if d_idx else None)
    at = rows.numpy()
    gc, gs = _np(cache.codes)[at], _np(cache.scales)[at]
    assert np.array_equal(gc, codes) and np.array_equal(gs, scales)
    saturated = int((wide[:, :512].float().abs().reshape(n, 32, 16).amax(-1) > 2688).sum())
    assert _np(cnt).tolist() == [saturated, 0, 0, 0]
    other = np.ones(cap, bool)
    other[at] = False
    assert not _np(cache.codes)[other].any() and not _np(cache.scales)[other].any()
    if d_idx:
        assert np.array_equal(_np(cache.kidx)[at], kidx) and np.array_equal(_np(cache.kscale)[at], ksc)
        want = torch.from_numpy(kidx).view(torch.float8_e4m3fn).double().numpy() * ksc[:, None].astype(np.float64)
        assert np.array_equal(_np(kb).astype(np.float64), want)
        assert (_np(cache.kidx)[other] == 0x11).all()
    else:
        assert (_np(cache.kidx) == 0x11).all()
    want = O.fp4_decode_rows(codes, scales)
    assert np.array_equal(_np(xb[:, :512].double()), want)
    assert (_np(xb[:, 512:].float()) == 7).all()


def test_rows_padding_and_bad_numbers():
    cache = csa.Cache([16], 64, 1, DEV)
    x = _latents(6, torch.float32, 5)
    rows = torch.tensor([3, -1, 16, 1 << 40, -(1 << 40), 15])
    cnt = csa.new_counters()
    csa.cache_write(cache, rows.to(DEV), x.to(DEV), counters=cnt)
    out = torch.full((6, 512), 9.0, device=DEV)
    csa.cache_read(cache, rows.to(DEV), out, counters=cnt)
    torch.cuda.synchronize()
    codes, scales, _k, _s = _oracle_rows(x[[0, 5]], None)
    assert np.array_equal(_np(cache.codes)[[3, 15]], codes)
    untouched = [i for i in range(16) if i not in (3, 15)]
    assert not _np(cache.codes)[untouched].any()
    assert _np(cnt).tolist() == [0, 0, 4, 0]            # two rows past the cache, written and read
    got = _np(out)
    assert (got[1:5] == 9).all()
    assert np.array_equal(got[[0, 5]].astype(np.float64), O.fp4_decode_rows(codes, scales))


def test_read_repeats_rows_and_infinities_saturate():
    cache = csa.Cache([8], 64, 1, DEV)
    x = torch.zeros(1, 512)
    x[0, 0], x[0, 16], x[0, 17] = float("inf"), float("-inf"), 1.0
    cnt = csa.new_counters()
    csa.cache_write(cache, torch.tensor([5], device=DEV), x.to(DEV), counters=cnt)
    out = torch.zeros(300, 512, dtype=torch.float16, device=DEV)
    csa.cache_read(cache, torch.full((300,), 5, device=DEV), out)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [2, 0, 0, 0]
    got = _np(out.float())
    assert (got == got[0]).all() and got[0, 0] == 2688 and got[0, 16] == -2688 and got[0, 17] == 0


def _midpoints(t):
    """Every scale's midpoints, and their neighbours some of the type's steps away."""
    s = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()       # 126 scales
    m = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
    whole = torch.int32 if t == torch.float32 else torch.int16
    far = [-40, -17, -9, -8, -7, -4, -2, -1, 0, 1, 2, 4, 7, 8, 9, 17, 40] if t == torch.float32 else range(-8, 9)
    bits = (s[:, None] * m).to(t).view(whole)[:, :, None]                                # exact in t
    v = (bits + torch.tensor(list(far), dtype=whole)).view(t).float().reshape(126, -1)   # 119 a scale
    v = torch.cat([v, -v, torch.zeros(126, 2)], 1).reshape(126, 16, 15)                  # 16 groups of 15 ..
    x = torch.cat([(6 * s)[:, None, None].expand(126, 16, 1), v], 2)                     # .. and the scale's 6 s
    return x.reshape(63, 512).to(t)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_write_next_to_the_midpoints(t):
    x = _midpoints(TYPES[t])
    n = x.shape[0]
    cache = csa.Cache([64], 64, 1, DEV)
    csa.cache_write(cache, torch.arange(n, device=DEV), x.to(DEV))
    torch.cuda.synchronize()
    codes, scales, _k, _s = _oracle_rows(x, None)
    assert np.array_equal(_np(cache.scales)[:n], scales) and np.array_equal(_np(cache.codes)[:n], codes)
    assert np.array_equal(scales.reshape(126, 16), np.repeat(np.arange(1, 127)[:, None], 16, 1))


# ================================================================ dense attention
def _random_cache(lens, seed, m=1, gap=0):
    """A cache of random entries (scales 2^-3 .. 2, values near unit size); every row
    past a sequence's entries holds NaN scales."""
    g = torch.Generator().manual_seed(seed)
    cache = csa.Cache([n + gap for n in lens], 64, m, DEV)
    cache.codes.copy_(torch.randint(0, 256, (cache.cap, 256), generator=g, dtype=torch.uint8))
    s = torch.randint(0x20, 0x3C, (cache.cap, 32), generator=g, dtype=torch.uint8)
    for b, n in enumerate(lens):
        s[cache.base_host[b] + n:cache.base_host[b + 1]] = 0x7F
    cache.scales.copy_(s)
    cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    return cache


def _values(cache, b, n):
    r = cache.base_host[b]
    return torch.from_numpy(O.fp4_decode_rows(_np(cache.codes[r:r + n]), _np(cache.scales[r:r + n]))).reshape(n, 512)


def _reference(v, q, sm, prev):
    """out, lse and out's bound (but for its storage) of rows q [r][512] over the entries v [n][512]."""
    n = v.shape[0]
    v, q = v.to(DEV), q.double()
    x = sm * (q @ v.T)
    pl = prev[1].double()[:, None] if prev is not None else torch.full((q.shape[0], 1), -np.inf, dtype=torch.float64, device=DEV)
    both = torch.cat([x, pl], 1)
    lse = torch.logsumexp(both, 1)
    p = torch.exp(x - lse[:, None]).nan_to_num(0.0)
    w = torch.exp(pl - lse[:, None]).nan_to_num(0.0)
    po = torch.where(w > 0, prev[0].double(), 0.0) if prev is not None else torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    out = p @ v + w * po
    d = 32 * 2.0 ** -23 * abs(sm) * (q.abs() @ v.abs().T) + 2.0 ** -25 * abs(sm) * v.abs().sum(1) + 2.0 ** -21
    dmax = d.amax(1, keepdim=True) if n else torch.zeros(q.shape[0], 1, dtype=torch.float64, device=DEV)
    sums = n / 16 * 2.0 ** -23 + 2 * 152 * 2.0 ** -24 + 2.0 ** -20
    a = p @ v.abs() + (w * po.abs())
    # weights off by 2 d (numerator and denominator), f16, and the sums; below f16's normals 2^-25 of the largest
    top = p.amax(1, keepdim=True) if n else 0.0
    bound = (2 * dmax + 2.0 ** -11 + 2 * sums) * a + 2.0 ** -25 * top * (v.abs().sum(0) if n else 0.0)
    # a logsumexp moves by at most the largest move of its terms; log2 and the products in fp32
    lbound = dmax[:, 0] + sums + 2.0 ** -22 * lse.abs().nan_to_num(0.0, 0.0, 0.0) + 2.0 ** -22
    return out, lse, bound, lbound


def _storage(out, t):
    eps = torch.finfo(t).eps / 2
    return eps * out.abs() + torch.finfo(t).tiny * eps * 2


def _check(cache, seqs, off, lens, q, out, lse, prev=None, sm=1.0):
    for g, b in enumerate(seqs):
        a, e, n = off[g], off[g + 1], lens[g]
        if a == e:
            continue
        pr = None if prev is None else (prev[0][a:e].reshape(-1, 512), prev[1][a:e].reshape(-1))
        o, l, bo, bl = _reference(_values(cache, b, n), q[a:e].reshape(-1, 512), sm, pr)
        got = out[a:e].reshape(-1, 512).double()
        off_by = (got - o).abs() - bo - _storage(o, out.dtype)
        assert torch.isfinite(got).all() and off_by.max() <= 0, (g, n, off_by.max().item())
        if lse is not None:
            gl = lse[a:e].reshape(-1).double()
            inf = torch.isinf(l)
            assert torch.equal(torch.isinf(gl), inf)
            if (~inf).any():
                far = ((gl - l).abs() - bl)[~inf].max()
                assert far <= 0, (g, n, far.item())


def _queries(nq, h, t, seed, scale=0.11):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(nq, h, 512, generator=g) * scale).to(t).to(DEV)


def _prev(nq, h, seed, empty=False):
    g = torch.Generator().manual_seed(seed)
    po, pl = torch.randn(nq, h, 512, generator=g), torch.randn(nq, h, generator=g) + 6
    if empty:                                    # rows without a partial result: whatever it holds is not read
        po[::2], pl[::2] = float("nan"), float("-inf")
    return po.to(DEV), pl.to(DEV)


CASES = [
    # heads, (queries, entries) of each group
    (16, [(1, 1)]),
    (64, [(1, 0)]),
    (1, [(1, 7), (3, 128), (1, 129)]),
    (5, [(13, 127), (1, 0), (26, 1000)]),
    (20, [(7, 300), (0, 50), (33, 1), (2, 4097)]),
    (64, [(1, 5003)]),
    (64, [(2, 333), (1, 20000)]),
    (64, [(9, 2048), (5, 129)]),
    (128, [(3, 1025)]),
    (64, [(40, 1500)]),
    (16, [(100, 640), (1, 640)]),
    (8, [(1, 100)] * 45),
    (4, [(1, 30 + i % 7) for i in range(700)]),
    (2, [(i % 3, (i * 37) % 300) for i in range(1100)]),
]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("with_prev", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_dense_against_float64(case, with_prev, types):
    h, each = CASES[case]
    lens = [n for _c, n in each]
    off = np.concatenate([[0], np.cumsum([c for c, _n in each])]).tolist()
    cache = _random_cache(lens, case)
    q = _queries(off[-1], h, TYPES[types[0]], case + 100)
    out = torch.full((off[-1], h, 512), 7.0, dtype=TYPES[types[1]], device=DEV)
    lse = torch.full((off[-1], h), 7.0, device=DEV)
    prev = _prev(off[-1], h, case + 200, empty=True) if with_prev else None
    cnt = csa.new_counters()
    seqs = list(range(len(lens)))
    csa.dense_attn(cache, csa.Groups(seqs, off), q, out, lse, prev=prev, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 0, 0]
    _check(cache, seqs, off, lens, q, out, lse, prev)


@pytest.mark.parametrize("nq", [1, 3])
def test_dense_rescales_when_the_maximum_moves_late(nq):
    # logits of several hundred: the winner sits near the end, one row's at the start
    n = 3001
    cache = _random_cache([n], 31)
    v = _values(cache, 0, n).to(DEV)
    q = _queries(nq, 64, torch.float32, 32, 0.02)
    q += (v[n - 2] * 0.2).float()
    q[0, 5] = (v[3] * 0.4).float()
    q = q.to(torch.bfloat16)
    out, lse = torch.zeros(nq, 64, 512, device=DEV), torch.zeros(nq, 64, device=DEV)
    csa.dense_attn(cache, csa.Groups([0], [0, nq]), q, out, lse, sm_scale=0.7)
    torch.cuda.synchronize()
    _check(cache, [0], [0, nq], [n], q, out, lse, sm=0.7)


@pytest.mark.parametrize("sm", [-0.5, 0.0])
def test_dense_scale_may_be_negative_or_zero(sm):
    lens = [300, 2000]
    cache = _random_cache(lens, 35)
    q = _queries(4, 32, torch.bfloat16, 36, 0.3)
    out, lse = torch.zeros(4, 32, 512, device=DEV), torch.zeros(4, 32, device=DEV)
    csa.dense_attn(cache, csa.Groups([0, 1], [0, 1, 4]), q, out, lse, sm_scale=sm)
    torch.cuda.synchronize()
    _check(cache, [0, 1], [0, 1, 4], lens, q, out, lse, sm=sm)


def test_dense_lengths_padding_and_groups_out_of_contract():
    cache = _random_cache([200, 300, 64], 41, gap=24)
    seqs = [1, 0, 3, 2, 1, -1, 0]
    off = [0, 3, 5, 6, 8, 9, 11, 12]
    length = [77, 201, 5, -1, 300, 4, 0]         # group 1: past its entries, 2 and 5: no sequence, 3: negative
    q = _queries(15, 16, torch.bfloat16, 42)
    out = torch.full((15, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((15, 16), 7.0, device=DEV)
    cnt = csa.new_counters()
    csa.dense_attn(cache, csa.Groups(seqs, off, length), q, out, lse, max_n=300, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 4, 0]
    for g in (0, 4, 6):
        _check(cache, [seqs[g]], [off[g], off[g + 1]], [length[g]],
               q, out, lse)
    for a, e in ((3, 8), (9, 11), (12, 15)):     # skipped groups, and queries of no group
        assert (out[a:e] == 7).all() and (lse[a:e] == 7).all()


def test_dense_offsets_out_of_contract_and_max_n():
    cache = _random_cache([200, 100], 43)
    q = _queries(6, 16, torch.bfloat16, 44)
    out = torch.full((6, 16, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    cnt = csa.new_counters()
    csa.dense_attn(cache, csa.Groups([1, 1, 0], [0, 4, 2, 9]), q, out, max_n=150, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 2, 0]     # offsets that fall, and past the queries
    _check(cache, [1], [0, 4], [100], q, out, None)
    assert (out[4:] == 7).all()
    csa.dense_attn(cache, csa.Groups([0], [0, 6]), q, out.fill_(7.0), max_n=150, counters=cnt.zero_())
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, 1, 0] and (out == 7).all()    # 200 entries, at most 150 declared


@pytest.mark.parametrize("ng,at", [(3, 1), (3, 0), (2, 1), (32, 17), (45, 20), (45, 44), (1100, 700), (1100, 1)])
def test_dense_offsets_that_fall_end_the_groups(ng, at):
    """Groups behind one whose offsets fall may own the same queries as those before:
    they are skipped and counted, whatever they ask for, and what is before is computed."""
    h, lens = 4, [(i * 37) % 300 for i in range(7)]
    cache = _random_cache(lens, 45)
    seqs = [g % 7 for g in range(ng)]
    off = [2 * g for g in range(ng + 1)]
    for g in range(at + 1, ng + 1):              # falls by one at group `at`, ascends again from there
        off[g] = off[at] - 1 + 2 * (g - at - 1)
    assert off[at + 1] < off[at] and all(a <= b for g, (a, b) in enumerate(zip(off, off[1:])) if g != at)
    nq = max(off) + 5
    q = _queries(nq, h, torch.bfloat16, 46)
    out, lse = torch.full((nq, h, 512), 7.0, device=DEV), torch.full((nq, h), 7.0, device=DEV)
    prev = _prev(nq, h, 47)
    cnt = csa.new_counters()
    csa.dense_attn(cache, csa.Groups(seqs, off), q, out, lse, prev=prev, counters=cnt)
    torch.cuda.synchronize()
    assert _np(cnt).tolist() == [0, 0, ng - at, 0]
    _check(cache, seqs[:at], off[:at + 1], [lens[b] for b in seqs[:at]], q, out, lse, prev)
    assert (out[off[at]:] == 7).all() and (lse[off[at]:] == 7).all()


def test_dense_takes_and_leaves_its_own_partial_result():
    # three levels of shared prompts, each call in place over the last one's result
    lens = [700, 260, 1]
    cache = _random_cache(lens, 51)
    q = _queries(9, 64, torch.bfloat16, 52)
    out, lse = torch.zeros(9, 64, 512, device=DEV), torch.full((9, 64), -np.inf, device=DEV)
    for b in range(3):
        csa.dense_attn(cache, csa.Groups([b], [0, 9]), q, out, lse, prev=(out, lse))
    torch.cuda.synchronize()
    v = torch.cat([_values(cache, b, n) for b, n in enumerate(lens)])
    o, l, bo, bl = _reference(v, q.reshape(-1, 512), 1.0, None)
    # (each level rounds out and lse once more: 2^-23 of each, far below three times one level's bound)
    assert ((out.reshape(-1, 512).double() - o).abs() - 3 * bo).max() <= 0
    assert ((lse.reshape(-1).double() - l).abs() - 3 * bl).max() <= 0


def test_dense_nan_query_stays_in_its_row():
    for n, nq in ((400, 4), (6000, 1)):
        cache = _random_cache([n], 61)
        q = _queries(nq, 64, torch.bfloat16, 62)
        clean = q.clone()
        q[0, 3, 17] = float("nan")
        out = torch.zeros(nq, 64, 512, device=DEV)
        lse = torch.zeros(nq, 64, device=DEV)
        csa.dense_attn(cache, csa.Groups([0], [0, nq]), q, out, lse)
        want = torch.zeros_like(out)
        csa.dense_attn(cache, csa.Groups([0], [0, nq]), clean, want)
        torch.cuda.synchronize()
        assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
        out[0, 3], want[0, 3] = 0, 0
        assert torch.equal(out, want)


def test_dense_keeps_a_long_tail_below_one_large_entry():
    """One entry holds nearly all of a row's weight, 65,535 others 2^-24.3 to 2^-27.3 of it
    each, and every pair of CTAs runs through the whole sequence, so that the reference
    maximum is that entry's all along: the tail's weights must not vanish or be rounded
    one way.  The bound is the module's, but with 2^-32 of the row's largest weight for
    weights below f16's normals (half a step of 2^-24, and the largest is at least 2^7)."""
    n, h = 65536, 64
    nq = max(1, torch.cuda.get_device_properties(0).multi_processor_count // 2) * 128 // h
    cache = _random_cache([n], 101)
    g = torch.Generator().manual_seed(102)
    # tail: channels 0 .. 15 zero, the others positive (codes 1 .. 7, scale 1); entry 0: 24 in channel 0 alone
    codes = torch.randint(1, 8, (n, 512), generator=g, dtype=torch.uint8)
    codes[:, :16] = 0
    codes[0] = 0
    codes[0, 0] = 7
    cache.codes[:n].copy_(codes[:, 0::2] | (codes[:, 1::2] << 4))
    scales = torch.full((n, 32), 0x38, dtype=torch.uint8)
    scales[0] = 0x48                                          # 4
    cache.scales[:n].copy_(scales)
    deep = torch.tensor([24.3, 25.6, 26.6, 27.3]).repeat(h // 4)
    q = torch.zeros(nq, h, 512)
    q[:, :, 0] = deep * float(np.log(2)) / 24
    q = q.to(torch.bfloat16).to(DEV)
    out, lse = torch.zeros(nq, h, 512, device=DEV), torch.zeros(nq, h, device=DEV)
    csa.dense_attn(cache, csa.Groups([0], [0, nq]), q, out, lse)
    torch.cuda.synchronize()
    v = _values(cache, 0, n).to(DEV)
    assert v[0, 0] == 24 and not v[0, 1:].any() and not v[1:, :16].any() and (v[1:, 16:] > 0).all()
    x = q[0].double() @ v.T                                   # (every query is the same)
    lref = torch.logsumexp(x, 1)
    p = torch.exp(x - lref[:, None])
    want = p @ v
    dmax = (32 * 2.0 ** -23 * (q[0].double().abs() @ v.abs().T) + 2.0 ** -21).amax(1, keepdim=True)
    sums = n / 16 * 2.0 ** -23 + 2 * 152 * 2.0 ** -24 + 2.0 ** -20
    bound = (2 * dmax + 2.0 ** -11 + 2 * sums) * want + 2.0 ** -32 * p.amax(1, keepdim=True) * v.sum(0)
    far = (out.double() - want).abs() - bound - _storage(want, torch.float32)
    assert far.max() <= 0, (far.amax((0, 2)).tolist()[:4], (out[0, :4, 16:].double().sum(1) / want[:4, 16:].sum(1)).tolist())
    assert ((lse.double() - lref).abs() - dmax[:, 0] - sums - 2.0 ** -22 * (lref.abs() + 1)).max() <= 0


@pytest.mark.parametrize("queries,n,later", [(152, 600, 300), (1, 256 * 152, 300), (1, 256 * 152, 30000)])
def test_dense_logits_where_fp32_is_coarse(queries, n, later):
    """Two entries with logits near 6e7 (fp32 in steps of 4) that differ by one step, the
    others far below, sums exact: the weights are 1 and e^-4, in one run of tiles and over several pieces."""
    h = 64
    cache = _random_cache([n], 105)
    codes = torch.zeros(n, 512, dtype=torch.uint8)
    scales = torch.full((n, 32), 0x38, dtype=torch.uint8)
    for j in (0, later):                                      # 496 channels of 6 x 16, and one channel of 1 in the later entry
        codes[j, :496], scales[j, :31] = 7, 0x58
    codes[later, 511] = 2
    cache.codes[:n].copy_(codes[:, 0::2] | (codes[:, 1::2] << 4))
    cache.scales[:n].copy_(scales)
    v = _values(cache, 0, n).to(DEV)
    assert (v[[0, later], :496] == 96).all() and v[later, 511] == 1 and v.sum() == 2 * 496 * 96 + 1
    q = torch.zeros(queries, h, 512)
    q[:, :, :496] = (1032 + 8 * (torch.arange(h) % 46)).float()[None, :, None]
    q[:, :, 511] = 4
    q = q.to(torch.bfloat16).to(DEV)
    out, lse = torch.zeros(queries, h, 512, device=DEV), torch.zeros(queries, h, device=DEV)
    csa.dense_attn(cache, csa.Groups([0], [0, queries]), q, out, lse)
    torch.cuda.synchronize()
    x = q[0].double() @ v.T
    assert ((x[:, later] - x[:, 0]) == 4).all() and (x.amax(1) < 2.0 ** 26).all()
    w = 1 / (1 + float(np.exp(-4.0)))
    want = torch.zeros(512, dtype=torch.float64, device=DEV)
    want[:496], want[511] = 96, w
    # each weight: half a step of f16 and 2^-20 for the exponential and sums, in numerator and denominator
    far = (out.double() - want).abs() - 2 * (2.0 ** -11 + 2.0 ** -20) * want
    assert far.max() <= 0, far.max().item()
    # lse: the reference, log2 and their sum and product in fp32, four roundings
    lref = torch.logsumexp(x, 1)
    assert ((lse.double() - lref).abs() / lref).max() <= 4 * 2.0 ** -24


def test_dense_is_reproducible_on_streams_and_in_graphs():
    cache = _random_cache([5000, 900], 71)
    groups = csa.Groups([0, 1], [0, 2, 5])
    q = _queries(5, 64, torch.bfloat16, 72)
    want, wl = torch.zeros(5, 64, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(5, 64, device=DEV)
    csa.dense_attn(cache, groups, q, want, wl)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(want) for _ in range(2)]
    lses = [torch.zeros_like(wl) for _ in range(2)]
    need = csa.dense_workspace_size(2, 5, 64, cache.cap)
    graphs = []
    for i in range(2):                           # two graphs, each with its own workspace, replayed together
        ws = csa.workspace(need)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            csa.dense_attn(cache, groups, q, outs[i], lses[i], ws=ws)
        graphs.append((g, ws))
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want) and torch.equal(l, wl)
    with torch.cuda.stream(side):
        outs[0].zero_()
        csa.dense_attn(cache, groups, q, outs[0], lses[0])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)


def test_calls_from_two_threads():
    # each thread with its stream and the call's own workspace, many calls in flight
    cache = _random_cache([3000, 70], 81)
    groups = csa.Groups([0, 1], [0, 3, 4])
    q = _queries(4, 33, torch.float16, 82)
    want = torch.zeros(4, 33, 512, device=DEV)
    csa.dense_attn(cache, groups, q, want)
    rows = torch.arange(3000, device=DEV)
    values = torch.zeros(3000, 512, dtype=torch.bfloat16, device=DEV)
    csa.cache_read(cache, rows, values)
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                o, v = torch.zeros_like(want), torch.zeros_like(values)
                for _ in range(40):
                    o.zero_()
                    csa.dense_attn(cache, groups, q, o)
                    csa.cache_read(cache, rows, v)
                torch.cuda.current_stream().synchronize()
                got[k] = (o, v)
        except Exception as e:                   # (an assertion in a thread would go unseen)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for k in range(2):
        assert torch.equal(got[k][0], want) and torch.equal(got[k][1], values)


def test_refusals_with_tensors_on_the_device():
    cache = _random_cache([64], 91)
    g = csa.Groups([0], [0, 2])
    q = _queries(2, 4, torch.bfloat16, 92)
    out, lse = torch.full((2, 4, 512), 5.0, device=DEV), torch.full((2, 4), 5.0, device=DEV)
    prev = (torch.zeros(2, 4, 512, device=DEV), torch.zeros(2, 4, device=DEV))
    cnt = csa.new_counters()

    def refused(f, *args, **kw):
        with pytest.raises(csa.CsaError):
            f(*args, **kw)

    dense = lambda **kw: (lambda a: csa.dense_attn(cache, a.pop("groups"), a.pop("q"), a.pop("out"), a.pop("lse"), **a))(
        dict(dict(groups=g, q=q, out=out, lse=lse, counters=cnt), **kw))
    for bad in (dict(q=None), dict(q=q.cpu()), dict(q=q.float()), dict(q=q[..., :256]), dict(q=q.transpose(0, 1)),
                dict(q=q[0]), dict(out=None), dict(out=out.cpu()), dict(out=out.double()), dict(out=out[:1]),
                dict(out=out.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(lse=lse.cpu()), dict(lse=lse.half()), dict(lse=lse[:1]), dict(prev=(prev[0], None)),
                dict(prev=(prev[0].half(), prev[1])), dict(prev=(prev[0], prev[1][:1])), dict(prev=(prev[0].cpu(), prev[1])),
                dict(groups=csa.Groups([0], [0, 2], device="cpu")), dict(max_n=-1), dict(max_n=1 << 31),
                dict(ws=csa.workspace(256)), dict(ws=csa.workspace(1 << 22)[1:]), dict(counters=cnt.cpu()),
                dict(counters=cnt.float()), dict(counters=cnt[:3])):
        refused(dense, **bad)
    rows = torch.tensor([3, 1], device=DEV)
    x, key = torch.full((2, 512), 5.0, device=DEV), torch.full((2, 64), 5.0, device=DEV)
    bare = csa.Cache.over(cache.codes, cache.scales, None, None, cache.seq_base, cache.seq_len, 1)
    for f in (csa.cache_write, csa.cache_read):
        for bad in ((None, x), ([3, 1], x), (rows.cpu(), x), (rows.int(), x), (rows[:1], x), (rows[:, None], x), (rows, None),
                    (rows, x.cpu()), (rows, x.double()), (rows, x[:, :256]), (rows, x.t().contiguous().t()),
                    (rows, torch.zeros(2, 514, device=DEV)[:, 1:513]), (rows, x, key.cpu()), (rows, x, key[:, :32]),
                    (rows, x, key.double()), (rows, x, None, cnt.float()), (rows, x, None, cnt.cpu())):
            refused(f, cache, *bad)
        refused(f, bare, rows, x, torch.zeros(2, 128, device=DEV))
        refused(f, csa.Cache([8], 128, 1, "cpu"), rows, x)
    torch.cuda.synchronize()
    assert (out == 5).all() and (lse == 5).all() and (x == 5).all() and not cnt.any()
    dense()                                      # and the call itself still works
    csa.cache_read(bare, rows, x, counters=cnt)
    torch.cuda.synchronize()
    assert (out != 5).all() and not cnt.any()
    assert np.array_equal(_np(x.double()), _values(cache, 0, 64)[[3, 1]].numpy())


def test_every_refusal_is_the_packages_error():
    cache = _random_cache([64], 93)
    g = csa.Groups([0], [0, 2])
    q = _queries(2, 4, torch.bfloat16, 94)
    out, lse = torch.full((2, 4, 512), 5.0, device=DEV), torch.full((2, 4), 5.0, device=DEV)
    rows, x = torch.tensor([3, 1], device=DEV), torch.full((2, 512), 5.0, device=DEV)
    sparse = torch.zeros(2, 512, device=DEV).to_sparse()
    calls = [lambda a=a, k=k: csa.dense_attn(*a, **k) for a, k in (
        ((None, g, q, out, lse), {}), ((object(), g, q, out, lse), {}), ((cache, None, q, out, lse), {}),
        ((cache, (0, 1), q, out, lse), {}), ((cache, g, q, out, lse), dict(max_n=1.5)),
        ((cache, g, q, out, lse), dict(max_n=1 << 70)), ((cache, g, q, out, lse), dict(max_n="64")),
        ((cache, g, q, out, lse), dict(sm_scale="x")), ((cache, g, q, out, lse), dict(sm_scale=None)),
        ((cache, g, q, out, lse), dict(prev=5)), ((cache, g, q, out, lse), dict(prev=(out,))),
        ((cache, g, q, out, lse), dict(prev=(out, lse, lse))))]
    for f in (csa.cache_write, csa.cache_read):
        calls += [lambda a=a, f=f: f(*a) for a in ((None, rows, x), ("cache", rows, x), (cache, rows, sparse),
                                                   (cache, sparse, x), (cache, rows, x, sparse))]
    for call in calls:
        with pytest.raises(csa.CsaError):
            call()
    # what Python raised on the way is kept as the cause
    with pytest.raises(csa.CsaError) as e:
        csa.dense_attn(cache, g, q, out, lse, max_n=1.5)
    assert isinstance(e.value.__cause__, TypeError)
    torch.cuda.synchronize()
    assert (out == 5).all() and (lse == 5).all() and (x == 5).all()


def test_no_memory_for_a_workspace_is_pytorchs_error():
    cache = _random_cache([3000], 95)
    q = _queries(40, 64, torch.bfloat16, 96)
    out = torch.zeros(40, 64, 512, dtype=torch.bfloat16, device=DEV)
    groups = csa.Groups([0], [0, 40])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-4)          # 28 MB: the workspace needs 40
    try:
        assert csa.dense_workspace_size(1, 40, 64, cache.cap) > 30 << 20
        with pytest.raises(torch.OutOfMemoryError):
            csa.dense_attn(cache, groups, q, out)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    csa.dense_attn(cache, groups, q, out)
    torch.cuda.synchronize()
    _check(cache, [0], [0, 40], [3000], q, out, None)


def test_rows_and_dense_past_32_bit_offsets():
    # 18 M rows: 4.6 GB of codes; the second sequence lies past 2^32 bytes
    cap0, n = 17_500_000, 700
    cache = csa.Cache([cap0, 1024], 64, 1, DEV)
    rows = cache.base_host[1] + torch.arange(n)
    x = torch.randn(n, 512, generator=torch.Generator().manual_seed(81)).to(torch.bfloat16)
    csa.cache_write(cache, rows.to(DEV), x.to(DEV))
    cache.seq_len.copy_(torch.tensor([0, n], dtype=torch.int32))
    back = torch.zeros(n, 512, dtype=torch.bfloat16, device=DEV)
    csa.cache_read(cache, rows.to(DEV), back)
    q = _queries(3, 64, torch.bfloat16, 82)
    out, lse = torch.zeros(3, 64, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 64, device=DEV)
    csa.dense_attn(cache, csa.Groups([1], [0, 3]), q, out, lse, max_n=n)
    torch.cuda.synchronize()
    codes, scales, _k, _s = _oracle_rows(x, None)
    assert np.array_equal(_np(back.double()), O.fp4_decode_rows(codes, scales))
    assert not bool(cache.codes[:1 << 20].any())
    _check(cache, [1], [0, 3], [n], q, out, lse)


# ================================================================ together
def test_shared_prompt_with_each_sequences_own_entries():
    """A prompt written once by row number, read back, and attended by every
    sequence's query together with that sequence's own selected entries and
    window (csa2_sparse_attn): one softmax over all of them."""
    batch, n0, own, h, n_win = 6, 3000, 200, 64, 32
    cache = csa.Cache([n0] + [own] * batch, 64, 1, DEV)
    g = torch.Generator().manual_seed(91)
    prompt = torch.randn(n0, 512, generator=g).to(torch.bfloat16).to(DEV)
    rows = torch.arange(n0, device=DEV)
    csa.cache_write(cache, rows, prompt)
    cache.seq_len[0] = n0
    for b in range(batch):
        C = torch.randn(1, own, 512, generator=g).to(DEV)
        csa.quantize_append(cache, C, None, torch.randn(1, own, 64, generator=g).to(DEV), seq=1 + b)
    back = torch.zeros(n0, 512, dtype=torch.float32, device=DEV)
    csa.cache_read(cache, rows, back)
    q = _queries(batch, h, torch.bfloat16, 92)
    k = 50
    idx = torch.stack([torch.randperm(own, generator=g)[:k].sort().values for _ in range(batch)]).int().to(DEV)
    cnt = torch.full((batch,), k, dtype=torch.int32, device=DEV)
    win = torch.randn(1 + batch, n_win, 512, generator=g).to(torch.bfloat16).to(DEV)
    qs = csa.Queries(list(range(1, 1 + batch)), [own - 1] * batch, 1, DEV)
    part, plse = torch.zeros(batch, h, 512, device=DEV), torch.zeros(batch, h, device=DEV)
    counters = csa.new_counters()
    csa.sparse_attn(cache, qs, idx, cnt, q, win, n_win, part, plse, counters=counters)
    out, lse = torch.zeros(batch, h, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(batch, h, device=DEV)
    csa.dense_attn(cache, csa.Groups([0], [0, batch]), q, out, lse, prev=(part, plse), counters=counters)
    torch.cuda.synchronize()
    assert _np(counters).tolist() == [0, 0, 0, 0]
    assert torch.equal(back.double().cpu(), _values(cache, 0, n0))
    for b in range(batch):
        mine = _values(cache, 1 + b, own)[idx[b].long().cpu()]
        pos = torch.arange(own - n_win, own) % n_win
        v = torch.cat([back.double().cpu(), mine, win[1 + b].double().cpu()[pos]])
        o, l, bo, bl = _reference(v, q[b], 1.0, None)
        # (the sparse part rounds its own weights and sums: twice one part's bound)
        assert ((out[b].double() - o).abs() - 2 * bo - _storage(o, torch.bfloat16)).max() <= 0
        assert ((lse[b].double() - l).abs() - 2 * bl).max() <= 0


def test_cross_attention_over_appended_encoder_entries():
    """Decoder queries over the whole of their sequence's encoder cache (m = 2),
    whose length seq_len holds on the device, before and after an append."""
    cache = csa.Cache([300, 80], 64, 2, DEV)
    g = torch.Generator().manual_seed(95)
    q = _queries(5, 20, torch.float16, 96)
    off, lens = [0, 2, 5], [0, 0]
    groups = csa.Groups([0, 1], off)
    for n_tok in (4, 130):
        C, Z = (torch.randn(2, n_tok, 512, generator=g).to(DEV) for _ in range(2))
        csa.quantize_append(cache, C, Z, torch.randn(2, n_tok // 2, 64, generator=g).to(DEV))
        lens = [n + n_tok // 2 for n in lens]
        out, lse = torch.zeros(5, 20, 512, dtype=torch.float16, device=DEV), torch.zeros(5, 20, device=DEV)
        csa.dense_attn(cache, groups, q, out, lse)
        torch.cuda.synchronize()
        assert _np(cache.seq_len).tolist() == lens
        _check(cache, [0, 1], off, lens, q, out, lse)

"""Host-side argument checks of the norm with rotation, chunk attention, attention
weights and eviction: each call returns before it touches a device."""
import ctypes

import pytest
import torch

import sparse_attention_decode_step_gb300 as csa

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
OUT_OF_4 = ctypes.c_void_p(4097)
INVALID, ALIGN, CAPACITY, UNSUPPORTED = -1, -2, -3, -4


def _cache(**over):
    c = csa._Cache(4096, 4096, 4096, 4096, 4096, 4096, 64, 2, 128, 1)
    for k, v in over.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _pages(table=4096, ld=4, page=16):
    return ctypes.byref(csa._Pages(table, ld, page))


# ---------------------------------------------------------------- norm and rotation
def _rope(x=P, type=1, ld_x=2048, n=3, H=4, weight=None, eps=1e-6, pos=P, freq=P, rot=64, halves=0, out=P, out_type=1, ld_out=2048):
    return csa.lib().csa2_norm_rope(x, type, ld_x, n, H, weight, eps, pos, freq, rot, halves, out, out_type, ld_out, None)


def test_norm_rope_rejects_bad_arguments_on_host():
    assert _rope(n=0) == 0
    assert _rope(n=0, x=None, out=None, pos=None) == 0
    for bad in (dict(n=-1), dict(x=None), dict(out=None), dict(pos=None), dict(freq=None), dict(ld_x=2047), dict(ld_out=2040),
                dict(ld_x=1 << 31), dict(ld_out=1 << 31), dict(eps=-1.0), dict(eps=float("nan")), dict(n=1 << 31), dict(n=1 << 30, H=2)):
        assert _rope(**bad) == INVALID, bad
    for bad in (dict(type=3), dict(out_type=-1), dict(H=0), dict(H=129), dict(rot=-16), dict(rot=528), dict(rot=24)):
        assert _rope(**bad) == UNSUPPORTED, bad
    for bad in (dict(x=ODD), dict(out=ODD), dict(ld_x=2052), dict(out_type=0, ld_out=2050), dict(weight=ODD), dict(pos=OUT_OF_4),
                dict(freq=OUT_OF_4)):
        assert _rope(**bad) == ALIGN, bad


def test_norm_rope_in_place_needs_one_type_and_one_stride():
    for bad in (dict(out_type=0), dict(out_type=2), dict(ld_out=4096), dict(ld_x=4096)):
        assert _rope(**bad) == INVALID, bad


# ---------------------------------------------------------------- pages and groups
def _chunk(cache=None, pages=None, ng=2, nq=5, seq=4096, off=4096, length=None, groups=True, pos=None, max_n=64, q=P, q_type=1, H=16,
           prev=(None, None), out=P, out_type=1, lse=None, ws=P, ws_bytes=1 << 40, counters=None):
    g = csa._Groups(seq, off, length, ng, nq)
    return csa.lib().csa2_chunk_attn(cache or _cache(), pages, ctypes.byref(g) if groups else None, pos, max_n, q, q_type, H, 1.0,
                                     prev[0], prev[1], out, out_type, lse, ws, ws_bytes, counters, None)


def _mass(cache=None, pages=None, ng=2, nq=5, seq=4096, off=4096, length=None, groups=True, pos=None, max_n=64, q=P, q_type=1, H=16,
          lse=P, prev=None, mass=P, ld=64, ws=P, ws_bytes=1 << 40, counters=None):
    g = csa._Groups(seq, off, length, ng, nq)
    return csa.lib().csa2_attn_mass(cache or _cache(), pages, ctypes.byref(g) if groups else None, pos, max_n, q, q_type, H, 1.0, lse,
                                    prev, 1.0, mass, ld, ws, ws_bytes, counters, None)


@pytest.mark.parametrize("call", [_chunk, _mass])
def test_chunk_and_mass_reject_bad_arguments_on_host(call):
    assert call(ng=0) == 0
    for bad in (dict(groups=False), dict(ng=-1), dict(nq=-1), dict(seq=None), dict(off=None), dict(q=None), dict(max_n=-1),
                dict(max_n=1 << 31), dict(cache=_cache(scales=None)), dict(cache=_cache(seq_base=None)),
                dict(pages=_pages(table=None)), dict(pages=_pages(ld=0)), dict(pages=_pages(ld=1 << 31)),
                dict(pages=_pages(page=128)), dict(ws=None)):          # (128: more than the cache's 64 rows)
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=0), dict(H=129), dict(q_type=0), dict(q_type=3), dict(nq=1 << 30, H=128), dict(ng=1 << 24),
                dict(pages=_pages(page=8)), dict(pages=_pages(page=48)), dict(pages=_pages(page=0)), dict(pages=_pages(page=-16))):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(q=ODD), dict(seq=4098), dict(length=4097), dict(lse=OUT_OF_4), dict(pos=OUT_OF_4), dict(counters=OUT_OF_4),
                dict(pages=_pages(table=4098)), dict(cache=_cache(codes=4100)), dict(ws=ctypes.c_void_p(4104))):
        assert call(**bad) == ALIGN, bad


def test_chunk_and_mass_reject_what_is_their_own():
    assert _chunk(nq=0) == 0
    for bad in (dict(out=None), dict(prev=(P, None)), dict(prev=(None, P))):
        assert _chunk(**bad) == INVALID, bad
    assert _chunk(out=ODD) == ALIGN and _chunk(prev=(ODD, P)) == ALIGN and _chunk(out_type=3) == UNSUPPORTED
    need = csa.dense_workspace_size(2, 5, 16, 64)
    assert need > 0 and _chunk(ws_bytes=need - 1) == CAPACITY
    for bad in (dict(lse=None), dict(mass=None), dict(ld=63), dict(ld=1 << 31)):
        assert _mass(**bad) == INVALID, bad
    assert _mass(mass=OUT_OF_4) == ALIGN and _mass(prev=OUT_OF_4) == ALIGN
    need = csa.mass_workspace_size(2, 2, 5, 16, 64)
    assert need > 0 and _mass(ws_bytes=need - 1) == CAPACITY


def test_mass_workspace_sizes():
    size = csa.mass_workspace_size
    for bad in ((0, 1, 1, 16, 64), (1, 0, 1, 16, 64), (1, 1, -1, 16, 64), (1, 1, 1, 0, 64), (1, 1, 1, 129, 64), (1, 1, 1, 16, -1),
                (1, 1, 1, 16, 1 << 31), (1, 1 << 24, 1, 16, 64), (1, 1, 1 << 30, 1, 64)):
        assert size(*bad) == 0, bad
    # 64 rows and fewer write their weights themselves; more leave parts, 256 MB of them at most
    assert size(8, 1, 1, 64, 1 << 20) < 1 << 16 < size(8, 1, 2, 64, 1 << 20)
    assert size(8, 1, 1 << 20, 128, 1 << 20) < (256 << 20) + (1 << 20) * 80 + (1 << 16)


@pytest.mark.parametrize("n", [1 << 20, (1 << 20) + 1, 1 << 22, 1 << 24, (1 << 31) - 1])
def test_mass_workspace_of_long_sequences(n):
    # beyond a million entries the parts of 32 blocks of rows, 8 bytes an entry each, or of as many as there are
    size = csa.mass_workspace_size
    most, plan = 32 * 8 * n, (1 << 20) * 80 + (1 << 16)
    assert most <= size(8, 1, 1 << 20, 128, n) < most + plan
    assert 2 * 8 * n <= size(8, 1, 2, 64, n) < 2 * 8 * n + (1 << 16)
    assert size(8, 1, 1, 64, n) < 1 << 16


# ---------------------------------------------------------------- eviction
def _evict(cache=None, pages=None, to=None, to_pages=None, seq=None, ns=2, mass=P, ld=64, max_n=64, keep=16, first=2, last=3, kept=P,
           ld_kept=16, out=None, ld_out=0, ws=P, ws_bytes=1 << 40, counters=None):
    return csa.lib().csa2_cache_evict(cache or _cache(), pages, to or _cache(codes=8192), to_pages, seq, ns, mass, ld, max_n, keep, first, last,
                                      kept, ld_kept, out, ld_out, ws, ws_bytes, counters, None)


def test_evict_rejects_bad_arguments_on_host():
    assert _evict(ns=0, seq=P) == 0
    far = ctypes.c_void_p(1 << 20)
    for bad in (dict(ns=3), dict(ns=-1, seq=P), dict(mass=None), dict(kept=None), dict(max_n=-1), dict(max_n=1 << 31), dict(keep=0),
                dict(first=-1), dict(last=-1), dict(first=8, last=9), dict(ld=63), dict(ld_kept=15), dict(out=far, ld_out=15),
                dict(ld=1 << 31), dict(ld_kept=1 << 31), dict(out=far, ld_out=1 << 31),
                dict(out=P, ld_out=16), dict(out=ctypes.c_void_p(4096 + 64 * 2 * 4 - 4), ld_out=16),      # overlaps mass
                dict(mass=ctypes.c_void_p(8192), out=ctypes.c_void_p(8192 - 16 * 2 * 4 + 4), ld_out=16),
                dict(to=_cache(batch=3)), dict(to=_cache(kidx=None)), dict(cache=_cache(kidx=None)), dict(to=_cache(d_idx=64)),
                dict(cache=_cache(seq_base=None)), dict(to=_cache(seq_base=None)), dict(to_pages=_pages(ld=0)),
                dict(to=_cache(cap=8), to_pages=_pages(page=16)), dict(ws=None), dict(first=(1 << 31) - 1, last=(1 << 31) - 1),
                dict(to=_cache()), dict(to=_cache(), pages=_pages(), to_pages=_pages())):          # onto itself
        assert _evict(**bad) == INVALID, bad
    for bad in (dict(ns=65536, seq=P), dict(cache=_cache(d_idx=96), to=_cache(d_idx=96)), dict(to_pages=_pages(page=17))):
        assert _evict(**bad) == UNSUPPORTED, bad
    for bad in (dict(mass=OUT_OF_4), dict(kept=OUT_OF_4), dict(seq=OUT_OF_4), dict(out=ctypes.c_void_p((1 << 20) + 1), ld_out=16),
                dict(counters=OUT_OF_4), dict(ws=ctypes.c_void_p(4104)), dict(cache=_cache(kidx=4100))):
        assert _evict(**bad) == ALIGN, bad
    need = csa.evict_workspace_size(2, 64)
    assert need > 0 and _evict(ws_bytes=need - 1) == CAPACITY
    assert csa.evict_workspace_size(0, 64) == csa.evict_workspace_size(2, -1) == csa.evict_workspace_size(2, 1 << 31) == 0


# ---------------------------------------------------------------- the binding
def test_python_refusals_before_any_launch():
    table = torch.zeros(2, 4, dtype=torch.int32)
    cache = csa.Cache([8, 8], 64, 1, "cpu")
    g = csa.Groups([0], [0, 4], device="cpu")
    pages = csa.Pages(table, 16, device="cpu")
    q, lse = torch.zeros(4, 2, 512, dtype=torch.bfloat16), torch.zeros(4, 2)
    mass, kept = torch.zeros(2, 8), torch.zeros(2, 4, dtype=torch.int32)
    for bad in (lambda: csa.Pages(table, 8, device="cpu"), lambda: csa.Pages(table, 24, device="cpu"), lambda: csa.Pages(table[0], 16, device="cpu")):
        with pytest.raises(csa.CsaError):
            bad()
    refused = (
        lambda: csa.chunk_attn(cache, g, q, q.clone()),                                       # not on a CUDA device
        lambda: csa.chunk_attn(cache, g, q.float(), q),
        lambda: csa.chunk_attn(cache, g, q, q.double()),
        lambda: csa.chunk_attn(cache, g, q, q[:3]),
        lambda: csa.chunk_attn(cache, g, q, q.clone(), lse[:3]),
        lambda: csa.chunk_attn(cache, g, q, q.clone(), prev=(q.float(), None)),
        lambda: csa.chunk_attn(cache, g, q, q.clone(), prev=3),
        lambda: csa.chunk_attn(cache, None, q, q.clone()),
        lambda: csa.chunk_attn(cache, g, q, q.clone(), pages=3),
        lambda: csa.attn_mass(cache, g, q, lse, mass),
        lambda: csa.attn_mass(cache, g, q, lse.half(), mass),
        lambda: csa.attn_mass(cache, g, q, lse, mass[:, ::2]),
        lambda: csa.attn_mass(cache, g, q, None, mass),
        lambda: csa.cache_evict(cache, cache, mass, 4, kept),
        lambda: csa.cache_evict(cache, cache, mass, 4, kept, pages=3),
        lambda: csa.cache_evict(cache, cache, mass, 1 << 40, kept),
        lambda: csa.norm_rope(q, q),
        lambda: csa.norm_rope(q, q.double()),
        lambda: csa.norm_rope(q[..., :256], q[..., :256]),
        lambda: csa.norm_rope(q.transpose(0, 1), q.transpose(0, 1)),
        lambda: csa.norm_rope(q, q[:2]),
        lambda: csa.norm_rope("x", q),
        lambda: csa.Cache.over(cache.codes, cache.scales, cache.kidx, cache.kscale, None, cache.seq_len, 1).struct(),
    )
    for bad in refused:
        with pytest.raises(csa.CsaError):
            bad()


def test_pages_find_rows():
    pages = csa.Pages(torch.tensor([[3, 1, -1], [0, 2, 5]], dtype=torch.int32), 32, device="cpu")
    seq, entry = torch.tensor([0, 0, 1, 1, 1]), torch.tensor([0, 33, 31, 32, 95])
    assert pages.rows(seq, entry).tolist() == [96, 33, 31, 64, 191]
    assert csa.Pages([[1, 2]], 16, device="cpu").table.tolist() == [[1, 2]]


def test_a_cache_in_pages_needs_no_seq_base():
    c = csa.Cache([8, 16], 64, 2, "cpu")
    d = csa.Cache.over(c.codes, c.scales, c.kidx, c.kscale, None, c.seq_len, 2)
    assert (d.cap, d.batch, d.seq_base) == (24, 2, None)
    # the calls that go by seq_base say so
    with pytest.raises(csa.CsaError):
        csa.quantize_append(d, torch.zeros(2, 2, 512), None, None)

"""Host-side argument checks of the cache row calls and the dense attention:
each call returns before it touches a device."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

import sparse_attention_decode_step_gb300 as csa

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
INVALID, ALIGN, CAPACITY, UNSUPPORTED = -1, -2, -3, -4


def _cache(**over):
    c = csa._Cache(4096, 4096, 4096, 4096, 4096, 4096, 64, 1, 128, 1)
    for k, v in over.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _write(cache=None, rows=P, n=3, x=P, type=1, ld_x=512, key=None, ld_key=0, counters=None):
    return csa.lib().csa2_cache_write(cache or _cache(), rows, n, x, type, ld_x, key, ld_key, counters, None)


def _read(cache=None, rows=P, n=3, x=P, type=1, ld_x=512, key=None, ld_key=0, counters=None):
    return csa.lib().csa2_cache_read(cache or _cache(), rows, n, x, type, ld_x, key, ld_key, counters, None)


@pytest.mark.parametrize("call", [_write, _read])
def test_rows_reject_bad_arguments_on_host(call):
    assert call(n=0) == 0
    assert call(n=0, rows=None, x=None) == 0
    assert call(n=-1) == INVALID
    assert call(rows=None) == INVALID
    assert call(x=None) == INVALID
    assert call(type=3) == UNSUPPORTED
    assert call(type=-1) == UNSUPPORTED
    assert call(ld_x=511) == INVALID
    assert call(ld_x=0) == INVALID
    assert call(ld_x=516) == ALIGN                       # bf16: 1032 bytes
    assert call(type=0, ld_x=514) == ALIGN               # fp32: 2056 bytes
    assert call(x=ODD) == ALIGN
    assert call(rows=ctypes.c_void_p(4100)) == ALIGN
    assert call(key=P, ld_key=64) == INVALID             # d_idx 128
    assert call(key=ODD, ld_key=128) == ALIGN
    assert call(key=P, ld_key=130) == ALIGN
    assert call(cache=_cache(d_idx=96), key=P, ld_key=128) == UNSUPPORTED
    assert call(cache=_cache(kidx=None), key=P, ld_key=128) == INVALID
    assert call(cache=_cache(cap=60)) == INVALID
    assert call(cache=_cache(codes=4100)) == ALIGN
    assert call(counters=ctypes.c_void_p(4097)) == ALIGN
    f = csa.lib().csa2_cache_write if call is _write else csa.lib().csa2_cache_read
    assert f(None, P, 1, P, 1, 512, None, 0, None, None) == INVALID


def _dense(cache=None, ng=2, nq=5, seq=4096, off=4096, length=None, groups=True, max_n=64, q=P, q_type=1, H=16,
           prev=(None, None), out=P, out_type=1, lse=None, ws=P, ws_bytes=1 << 40, counters=None):
    g = csa._Groups(seq, off, length, ng, nq)
    return csa.lib().csa2_dense_attn(cache or _cache(), ctypes.byref(g) if groups else None, max_n, q, q_type, H, 1.0,
                                     prev[0], prev[1], out, out_type, lse, ws, ws_bytes, counters, None)


def test_dense_rejects_bad_arguments_on_host():
    assert _dense(ng=0) == 0
    assert _dense(nq=0) == 0
    assert _dense(groups=False) == INVALID
    assert _dense(ng=-1) == INVALID
    assert _dense(nq=-1) == INVALID
    assert _dense(seq=None) == INVALID
    assert _dense(off=None) == INVALID
    assert _dense(seq=4098) == ALIGN
    assert _dense(length=4097) == ALIGN
    assert _dense(q=None) == INVALID
    assert _dense(out=None) == INVALID
    assert _dense(q=ODD) == ALIGN
    assert _dense(out=ODD) == ALIGN
    assert _dense(lse=ctypes.c_void_p(4097)) == ALIGN
    assert _dense(H=0) == UNSUPPORTED
    assert _dense(H=129) == UNSUPPORTED
    assert _dense(q_type=0) == UNSUPPORTED
    assert _dense(q_type=3) == UNSUPPORTED
    assert _dense(out_type=3) == UNSUPPORTED
    assert _dense(nq=1 << 30, H=128) == UNSUPPORTED
    assert _dense(max_n=-1) == INVALID
    assert _dense(max_n=1 << 31) == INVALID
    assert _dense(prev=(P, None)) == INVALID
    assert _dense(prev=(None, P)) == INVALID
    assert _dense(prev=(ODD, P)) == ALIGN
    assert _dense(cache=_cache(scales=None)) == INVALID


def test_dense_workspace_is_checked():
    # many entries over few rows: the entries are divided over CTAs, whose partial results need space
    need = csa.dense_workspace_size(1, 1, 16, 1 << 20)
    if need == 0:
        pytest.skip("this host reports one SM: no division")
    big = _cache(cap=1 << 20)
    assert _dense(cache=big, ng=1, nq=1, max_n=1 << 20, ws_bytes=need - 1) == CAPACITY
    assert _dense(cache=big, ng=1, nq=1, max_n=1 << 20, ws=None, ws_bytes=0) == INVALID
    assert _dense(cache=big, ng=1, nq=1, max_n=1 << 20, ws=ctypes.c_void_p(4104), ws_bytes=need) == ALIGN


def test_dense_workspace_sizes_of_nothing():
    assert csa.dense_workspace_size(0, 1, 16, 64) == 0
    assert csa.dense_workspace_size(1, 0, 16, 64) == 0
    assert csa.dense_workspace_size(1, 1, 16, -1) == 0


def test_python_refusals_before_any_launch():
    cpu = torch.zeros(4, 512)
    rows = torch.zeros(4, dtype=torch.int64)
    cache = csa.Cache([8], 128, 1, "cpu")
    for call in (csa.cache_write, csa.cache_read):
        with pytest.raises(csa.CsaError):
            call(cache, rows, cpu)                                    # not on a CUDA device
        with pytest.raises(csa.CsaError):
            call(cache, rows.int(), cpu)
        with pytest.raises(csa.CsaError):
            call(cache, rows, cpu.double())
        with pytest.raises(csa.CsaError):
            call(cache, rows[:3], cpu)
    with pytest.raises(csa.CsaError):
        csa.cache_write(cache, rows, cpu.bfloat16(), torch.zeros(4, 128))     # key of another type
    with pytest.raises(csa.CsaError):
        csa.cache_read(cache, rows, cpu.bfloat16(), torch.zeros(4, 128).half())
    g = csa.Groups([0], [0, 4], device="cpu")
    q = torch.zeros(4, 2, 512, dtype=torch.bfloat16)
    with pytest.raises(csa.CsaError):
        csa.dense_attn(cache, g, q.float(), q.float())
    with pytest.raises(csa.CsaError):
        csa.dense_attn(cache, g, q, torch.zeros(4, 3, 512))
    with pytest.raises(csa.CsaError):
        csa.dense_attn(cache, g, q, q.clone(), torch.zeros(4, 3))
    with pytest.raises(csa.CsaError):
        csa.dense_attn(cache, g, q, q.clone())                        # not on a CUDA device
    with pytest.raises(csa.CsaError):
        csa.Groups([0, 1], [0, 4], device="cpu")
    with pytest.raises(csa.CsaError):
        csa.Groups([0], [0, 4], [1, 2], device="cpu")


def test_cache_over_checks_its_tensors():
    c = csa.Cache([8, 16], 64, 2, "cpu")
    d = csa.Cache.over(c.codes, c.scales, c.kidx, c.kscale, c.seq_base, c.seq_len, 2)
    assert (d.cap, d.batch, d.d_idx, d.m) == (24, 2, 64, 2)
    assert bytes(d.struct()) == bytes(c.struct())
    bare = csa.Cache.over(c.codes, c.scales, None, None, c.seq_base, c.seq_len, 2)
    assert bare.struct().kidx is None
    with pytest.raises(csa.CsaError):
        csa.Cache.over(c.codes, c.scales, c.kidx, None, c.seq_base, c.seq_len, 2)
    with pytest.raises(csa.CsaError):
        csa.Cache.over(c.codes[:16], c.scales, c.kidx, c.kscale, c.seq_base, c.seq_len, 2)
    with pytest.raises(csa.CsaError):
        csa.Cache.over(c.codes.int(), c.scales, c.kidx, c.kscale, c.seq_base, c.seq_len, 2)
    with pytest.raises(csa.CsaError):
        csa.Cache.over(c.codes, c.scales, c.kidx, c.kscale, c.seq_base[:2], c.seq_len, 2)


def test_refusals_of_what_is_no_tensor_or_has_no_storage():
    c = csa.Cache([8, 16], 64, 2, "cpu")
    rows, x = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 512)
    sparse = torch.zeros(24, 256, dtype=torch.uint8).to_sparse()
    for call in (lambda: csa.Cache.over(sparse, c.scales, c.kidx, c.kscale, c.seq_base, c.seq_len, 2),
                 lambda: csa.Cache.over("codes", c.scales, c.kidx, c.kscale, c.seq_base, c.seq_len, 2),
                 lambda: csa.cache_write(c, torch.zeros(4, dtype=torch.int64).to_sparse(), x),
                 lambda: csa.cache_read(c, rows, torch.zeros(4, 512).to_sparse()),
                 lambda: csa.dense_attn(c, None, x, x), lambda: csa.dense_attn(c, csa.Groups([0], [0, 4], device="cpu"), x, x, prev=3)):
        with pytest.raises(csa.CsaError):
            call()


def test_the_library_does_not_need_the_compiled_module(tmp_path):
    # a copy of the package whose module cannot be built: the C ABI and the ctypes calls work, the short calls say why not
    csa.lib()
    pkg = os.path.dirname(csa.__file__)
    to = tmp_path / os.path.basename(pkg)
    shutil.copytree(pkg, to, ignore=shutil.ignore_patterns("csa2_torch.*", "*.o", "__pycache__"))
    shutil.copytree(os.path.join(os.path.dirname(pkg), "include"), tmp_path / "include")
    (to / "csrc" / "csa2_torch.cpp").write_text("#error no PyTorch here\n")
    code = f"""
import {to.name} as csa, torch
assert csa.library_path().startswith({str(tmp_path)!r})
assert csa.topk_workspace_size(1, 1 << 20) > 0 and csa.dense_workspace_size(1, 1, 16, 64) > 0
cache = csa.Cache([8], 64, 1, "cpu")
try:
    csa.cache_write(cache, torch.zeros(1, dtype=torch.int64), torch.zeros(1, 512))
except RuntimeError as e:
    assert "csa2_torch.cpp" in str(e) and "no PyTorch here" in str(e), e
else:
    raise AssertionError("no error")
"""
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]


def test_the_compiled_module_is_rebuilt_for_another_pytorch(tmp_path, monkeypatch):
    from sparse_attention_decode_step_gb300 import build as b
    b.build_ext()
    assert b.ext_up_to_date()
    stamp = tmp_path / "for"
    monkeypatch.setattr(b, "EXT_STAMP", str(stamp))
    assert not b.ext_up_to_date()                                  # it is not known what it was built for
    stamp.write_text(b._ext_stamp())
    assert b.ext_up_to_date()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    assert not b.ext_up_to_date() and b.up_to_date()


def test_dense_workspace_sizes_of_calls_that_are_refused():
    for ng, nq, h, n in ((1, 1, 16, 1 << 31), (1, 1, 16, (1 << 63) - 1), (1, 1, 16, 1 << 62), (1, 1, 129, 64), (1, 1, 0, 64),
                         (1, 1 << 30, 1, 64), (1, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1), (1 << 24, 1 << 20, 1, 64)):
        assert csa.dense_workspace_size(ng, nq, h, n) == 0, (ng, nq, h, n)
        assert _dense(ng=ng, nq=nq, H=h, max_n=n) in (INVALID, UNSUPPORTED)
    # and of the largest that are not: no more than that of a full GPU
    most = csa.dense_workspace_size(1, 1 << 20, 128, 64)
    assert csa.dense_workspace_size((1 << 24) - 1, (1 << 30) - 1, 1, (1 << 31) - 1) == most > 0
    assert csa.dense_workspace_size(1, 1, 16, 1 << 20) > 0


def test_cache_over_refuses_tensors_of_two_devices():
    # (a call takes the addresses of all of them: one of host memory would fault on the GPU)
    c = csa.Cache([8, 16], 64, 2, "cpu")
    six = [c.codes, c.scales, c.kidx, c.kscale, c.seq_base, c.seq_len]
    for i in range(6):
        with pytest.raises(csa.CsaError):
            csa.Cache.over(*six[:i], six[i].to("meta"), *six[i + 1:], 2)
    assert csa.Cache.over(*six, 2).cap == 24

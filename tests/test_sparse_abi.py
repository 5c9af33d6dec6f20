"""Refusals of the block-sparse decode's calls: on the host, before anything
is enqueued (CPU only)."""
import ctypes
import os
import re

import pytest
import torch

from paged_kv_cache_246_gb300 import binding as B

NUL = ctypes.c_void_p(0)
PTR = ctypes.c_void_p(1 << 20)   # never followed: every call here is refused


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from paged_kv_cache_246_gb300 import build_lib
        build_lib.build()
    return B.lib()


def _p(**kw):
    base = dict(num_heads=32, num_kv_heads=8, head_size=128, block_size=16, dtype=B.PKV_BF16,
                scale=0.088, alibi_slopes=None, sliding_window=0, non_causal=0,
                kv_cache_dtype=B.PKV_CACHE_AUTO, k_scale=1.0, v_scale=1.0)
    base.update(kw)
    return B.AttnParams(**base)


def _rope(lib, p=None, **kw):
    a = dict(qo=PTR, so=4096, q=PTR, sq=4096, k=PTR, sk=1024, v=PTR, sv=1024, n=3, pos=PTR, cs=PTR,
             maxp=64, rot=128, inter=0, cache=NUL, nb=4, slots=PTR)
    a.update(kw)
    return lib.kv_cache_write_rope(*a.values(), ctypes.byref(p or _p()), NUL)


def test_rope_refusals(lib):
    assert _rope(lib, n=0) == B.PKV_OK
    assert _rope(lib) == B.PKV_ERR_INVALID                       # null cache
    ok = dict(cache=PTR)
    for bad in (dict(qo=NUL), dict(q=NUL), dict(k=NUL), dict(v=NUL), dict(pos=NUL), dict(cs=NUL),
                dict(slots=NUL), dict(n=-1), dict(maxp=0), dict(inter=2), dict(rot=0),
                dict(rot=144), dict(sq=4095), dict(sq=4088), dict(sq=4100), dict(sk=1023),
                dict(sv=0), dict(so=-4096), dict(nb=0), dict(q=ctypes.c_void_p((1 << 20) + 8)),
                dict(cs=ctypes.c_void_p((1 << 20) + 4)), dict(so=8192)):
        assert _rope(lib, **{**ok, **bad}) == B.PKV_ERR_INVALID, bad
    assert _rope(lib, rot=24, **ok) == B.PKV_ERR_UNSUPPORTED
    assert _rope(lib, n=1 << 31, **ok) == B.PKV_ERR_UNSUPPORTED
    assert _rope(lib, _p(head_size=96), **ok) == B.PKV_ERR_UNSUPPORTED
    fp8 = dict(kv_cache_dtype=B.PKV_CACHE_FP8_E4M3)
    assert _rope(lib, _p(k_scale=0.0, **fp8), **ok) == B.PKV_ERR_INVALID


def _bounds(lib, p=None, **kw):
    a = dict(bounds=PTR, cache=PTR, nb=4, tables=PTR, mb=2, ctx=NUL, lens=PTR, n=3, new=1)
    a.update(kw)
    return lib.kv_block_bounds(*a.values(), ctypes.byref(p or _p()), NUL)


def test_bounds_refusals(lib):
    assert _bounds(lib, n=0) == B.PKV_OK and _bounds(lib, new=0) == B.PKV_OK
    for bad in (dict(bounds=NUL), dict(cache=NUL), dict(tables=NUL), dict(lens=NUL), dict(nb=0),
                dict(mb=0), dict(n=-1), dict(n=65536), dict(new=-1),
                dict(ctx=ctypes.c_void_p((1 << 20) + 2))):
        assert _bounds(lib, **bad) == B.PKV_ERR_INVALID, bad
    assert _bounds(lib, _p(block_size=8)) == B.PKV_ERR_UNSUPPORTED
    assert _bounds(lib, mb=1 << 27, new=0x7fffffff) == B.PKV_ERR_UNSUPPORTED


def _select(lib, p=None, **kw):
    a = dict(sel=PTR, k=8, q=PTR, n=3, bounds=PTR, nb=4, tables=PTR, mb=2, lens=PTR, maxl=32, sink=1,
             recent=1)
    a.update(kw)
    return lib.paged_attn_select_blocks(*a.values(), ctypes.byref(p or _p()), NUL)


def test_select_refusals(lib):
    assert _select(lib, n=0) == B.PKV_OK
    for bad in (dict(sel=NUL), dict(q=NUL), dict(bounds=NUL), dict(tables=NUL), dict(lens=NUL),
                dict(nb=0), dict(mb=0), dict(n=-1), dict(n=65536), dict(maxl=-1), dict(sink=-1),
                dict(recent=0), dict(k=1), dict(k=0, sink=0), dict(sink=0x7fffffff, recent=0x7fffffff)):
        assert _select(lib, **bad) == B.PKV_ERR_INVALID, bad
    assert _select(lib, _p(alibi_slopes=1 << 20)) == B.PKV_ERR_UNSUPPORTED
    assert _select(lib, maxl=16 * B.PKV_SELECT_MAX_BLOCKS + 1) == B.PKV_ERR_UNSUPPORTED
    assert _select(lib, _p(num_heads=129, num_kv_heads=1)) == B.PKV_ERR_UNSUPPORTED
    assert _select(lib, _p(num_heads=65536, num_kv_heads=65536)) == B.PKV_ERR_UNSUPPORTED


def _sparse(lib, p=None, **kw):
    a = dict(out=PTR, q=PTR, n=3, cache=PTR, nb=4, tables=PTR, mb=2, lens=PTR, sel=PTR, k=8)
    a.update(kw)
    return lib.paged_attn_decode_sparse(*a.values(), ctypes.byref(p or _p()), NUL)


def test_sparse_refusals(lib):
    assert _sparse(lib, n=0) == B.PKV_OK
    for bad in (dict(out=NUL), dict(q=NUL), dict(cache=NUL), dict(tables=NUL), dict(lens=NUL),
                dict(sel=NUL), dict(nb=0), dict(mb=0), dict(n=-1), dict(n=65536), dict(k=0),
                dict(cache=ctypes.c_void_p((1 << 20) + 8))):
        assert _sparse(lib, **bad) == B.PKV_ERR_INVALID, bad
    assert _sparse(lib, _p(dtype=5)) == B.PKV_ERR_UNSUPPORTED
    assert _sparse(lib, k=(1 << 28) + 1) == B.PKV_ERR_UNSUPPORTED
    assert _sparse(lib, _p(num_heads=65536, num_kv_heads=65536)) == B.PKV_ERR_UNSUPPORTED


def test_select_limit_matches_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    m = re.search(r"#define PKV_SELECT_MAX_BLOCKS (\d+)", open(os.path.join(root, "include", "pkv.h")).read())
    assert m and int(m.group(1)) == B.PKV_SELECT_MAX_BLOCKS


def test_binding_wants_cuda_tensors():
    p = _p()
    cache = torch.zeros(2, 4, 16 * 1024, dtype=torch.bfloat16)
    i64, i32 = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    q, kv = torch.zeros(3, 4096, dtype=torch.bfloat16), torch.zeros(3, 1024, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.kv_cache_write_rope(q, q, kv, kv, cache, i64, i64, torch.zeros(8, 128), p)
    with pytest.raises(ValueError):
        B.kv_block_bounds(torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16), cache, i32.view(3, 1), i32, 1, p)
    with pytest.raises(ValueError):
        B.paged_attn_select_blocks(torch.zeros(3, 8, 4, dtype=torch.int32), q,
                                   torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16), i32.view(3, 1), i32, 16, p)
    with pytest.raises(ValueError):
        B.paged_attn_decode_sparse(q, q, cache, i32.view(3, 1), i32, torch.zeros(3, 8, 4, dtype=torch.int32), p)

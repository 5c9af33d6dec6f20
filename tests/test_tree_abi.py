"""Refusals of the calls over trees of drafted tokens: on the host, before
anything is enqueued (CPU only)."""
import ctypes
import os
import re

import pytest
import torch

from paged_kv_cache_246_gb300 import binding as B

NUL = ctypes.c_void_p(0)
PTR = ctypes.c_void_p(1 << 20)   # never followed: every call here is refused
ODD = ctypes.c_void_p((1 << 20) + 2)


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


def _axes(*values):
    return (ctypes.c_uint8 * 64)(*values)


def _rope(lib, p=None, **kw):
    a = dict(qo=PTR, so=4096, q=PTR, sq=4096, k=PTR, sk=1024, v=PTR, sv=1024, n=3, pos=PTR, ps=3,
             na=3, axes=_axes(0, 1, 2), cs=PTR, maxp=64, rot=128, inter=0, cache=PTR, nb=4, slots=PTR)
    a.update(kw)
    return lib.kv_cache_write_rope_axes(*a.values(), ctypes.byref(p or _p()), NUL)


def test_rope_axes_refusals(lib):
    assert _rope(lib, n=0) == B.PKV_OK
    for bad in (dict(qo=NUL), dict(q=NUL), dict(k=NUL), dict(v=NUL), dict(pos=NUL), dict(cs=NUL),
                dict(slots=NUL), dict(cache=NUL), dict(n=-1), dict(maxp=0), dict(inter=2), dict(rot=0),
                dict(rot=144), dict(sq=4095), dict(sk=1023), dict(nb=0), dict(axes=NUL), dict(na=0),
                dict(na=2), dict(ps=2), dict(axes=_axes(3)), dict(so=8192),
                dict(pos=ctypes.c_void_p((1 << 20) + 4))):
        assert _rope(lib, **bad) == B.PKV_ERR_INVALID, bad
    assert _rope(lib, na=5) == B.PKV_ERR_UNSUPPORTED
    assert _rope(lib, rot=24) == B.PKV_ERR_UNSUPPORTED
    assert _rope(lib, _p(head_size=96)) == B.PKV_ERR_UNSUPPORTED


def _tree(lib, p=None, **kw):
    a = dict(out=PTR, q=PTR, t=9, n=3, cu=PTR, up=PTR, most=64, cache=PTR, nb=4, tables=PTR, mb=2,
             lens=PTR, maxl=32)
    a.update(kw)
    ws, wb = a.pop("ws", PTR), a.pop("wb", 1 << 40)
    return lib.paged_attn_decode_tree(*a.values(), ctypes.byref(p or _p()), ws, wb, NUL)


def test_tree_refusals(lib):
    assert _tree(lib, n=0) == B.PKV_OK and _tree(lib, t=0) == B.PKV_OK
    for bad in (dict(out=NUL), dict(q=NUL), dict(cu=NUL), dict(up=NUL), dict(cache=NUL),
                dict(tables=NUL), dict(lens=NUL), dict(nb=0), dict(mb=0), dict(n=-1), dict(n=65536),
                dict(t=-1), dict(most=0), dict(maxl=-1), dict(cu=ODD), dict(up=ODD), dict(lens=ODD),
                dict(q=ctypes.c_void_p((1 << 20) + 8))):
        assert _tree(lib, **bad) == B.PKV_ERR_INVALID, bad
    assert _tree(lib, most=B.PKV_TREE_MAX_NODES + 1) == B.PKV_ERR_UNSUPPORTED
    assert _tree(lib, _p(non_causal=1)) == B.PKV_ERR_UNSUPPORTED
    assert _tree(lib, _p(num_heads=129, num_kv_heads=1)) == B.PKV_ERR_UNSUPPORTED
    assert _tree(lib, _p(head_size=96)) == B.PKV_ERR_UNSUPPORTED
    assert _tree(lib, t=1 << 31) == B.PKV_ERR_UNSUPPORTED


def _accept(lib, **kw):
    a = dict(acc=PTR, k=4, num=PTR, tok=PTR, draft=PTR, target=PTR, up=PTR, cu=PTR, n=3, t=9, most=64)
    a.update(kw)
    return lib.paged_attn_tree_accept(*a.values(), NUL)


def test_accept_refusals(lib):
    assert _accept(lib, n=0) == B.PKV_OK
    for bad in (dict(acc=NUL), dict(num=NUL), dict(tok=NUL), dict(draft=NUL), dict(target=NUL),
                dict(up=NUL), dict(cu=NUL), dict(k=0), dict(n=-1), dict(n=65536), dict(t=-1),
                dict(most=0), dict(acc=ODD), dict(tok=ctypes.c_void_p((1 << 20) + 4))):
        assert _accept(lib, **bad) == B.PKV_ERR_INVALID, bad
    assert _accept(lib, most=257) == B.PKV_ERR_UNSUPPORTED
    assert _accept(lib, t=1 << 31) == B.PKV_ERR_UNSUPPORTED


def _commit(lib, p=None, **kw):
    a = dict(caches=(ctypes.c_void_p * 2)(1 << 20, 1 << 21), layers=2, nb=4, acc=PTR, k=4, tables=PTR,
             mb=2, lens=PTR, cu=PTR, n=3)
    a.update(kw)
    return lib.kv_commit_tree(*a.values(), ctypes.byref(p or _p()), NUL)


def test_commit_refusals(lib):
    assert _commit(lib, n=0) == B.PKV_OK and _commit(lib, layers=0) == B.PKV_OK
    for bad in (dict(caches=NUL), dict(caches=(ctypes.c_void_p * 2)(1 << 20, 0)),
                dict(caches=(ctypes.c_void_p * 2)(1 << 20, 8)), dict(layers=257), dict(layers=-1),
                dict(acc=NUL), dict(tables=NUL), dict(lens=NUL), dict(cu=NUL), dict(nb=0), dict(mb=0),
                dict(n=-1), dict(n=65536), dict(k=0), dict(acc=ODD)):
        assert _commit(lib, **bad) == B.PKV_ERR_INVALID, bad
    twice = (ctypes.c_void_p * 3)(1 << 20, 1 << 21, 1 << 20)    # a cache named twice
    assert _commit(lib, caches=twice, layers=3) == B.PKV_ERR_INVALID
    assert _commit(lib, k=257) == B.PKV_ERR_UNSUPPORTED
    assert _commit(lib, _p(block_size=8)) == B.PKV_ERR_UNSUPPORTED


def test_node_limit_matches_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    m = re.search(r"#define PKV_TREE_MAX_NODES (\d+)", open(os.path.join(root, "include", "pkv.h")).read())
    assert m and int(m.group(1)) == B.PKV_TREE_MAX_NODES


def test_workspace_sizes(lib):
    p = _p()
    assert B.paged_attn_decode_tree_workspace_size(0, 64, 1024, p) == 0
    assert B.paged_attn_decode_tree_workspace_size(4, 257, 1024, p) == 0
    assert B.paged_attn_decode_tree_workspace_size(4, 64, 1024, _p(head_size=96)) == 0


def test_binding_wants_what_it_says():
    p = _p()
    cache = torch.zeros(2, 4, 16 * 1024, dtype=torch.bfloat16)
    i64, i32 = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int32)
    q, kv = torch.zeros(3, 4096, dtype=torch.bfloat16), torch.zeros(3, 1024, dtype=torch.bfloat16)
    axes = B.rope_pair_axes([16, 24, 24])

    def rope(positions=i64.expand(3, 3).contiguous(), pair_axes=axes):
        B.kv_cache_write_rope_axes(q, q, kv, kv, cache, i64, positions, torch.zeros(8, 128), pair_axes, p)

    for bad in (dict(), dict(positions=i64), dict(pair_axes=axes[1:]), dict(pair_axes=()),
                dict(pair_axes=(4,) * 64), dict(positions=i64.expand(2, 3).contiguous()),
                dict(positions=i64.expand(3, 3)), dict(positions=i64.expand(3, 3).contiguous().t()),
                dict(positions=i64.expand(3, 3).int())):
        with pytest.raises(ValueError):     # the first: not on a GPU
            rope(**bad)

    def tree(lens=i32, cu=cu, q=q, up=i32):
        B.paged_attn_decode_tree(q, q, cache, i32.view(3, 1), lens, cu, up, 4, 16, p)

    for bad in (dict(), dict(cu=i32), dict(lens=cu), dict(q=q[:, :128]), dict(up=i64)):
        with pytest.raises(ValueError):
            tree(**bad)
    acc = torch.zeros(3, 4, dtype=torch.int32)
    for bad in ((acc, i32, i64, i64, i64, i32, cu), (acc, i32, i64, i64, i64, i32, i32),
                (acc, i32, i64, i64, i64[:2], i32, cu), (acc, i32, i32, i64, i64, i32, cu)):
        with pytest.raises(ValueError):
            B.paged_attn_tree_accept(*bad, 4)
    for bad in ((acc, i32.view(3, 1), i32, cu), (acc[:2], i32.view(3, 1), i32, cu),
                (acc, i32.view(3, 1), i32, i32)):
        with pytest.raises(ValueError):
            B.kv_commit_tree([cache], *bad, p)
    with pytest.raises(ValueError):
        B.kv_commit_tree([cache, cache[:, :2].contiguous()], acc, i32.view(3, 1), i32, cu, p)

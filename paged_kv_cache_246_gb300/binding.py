"""Thin ctypes binding of libpkv.so (declared in include/pkv.h).

Argument marshalling only: each function checks the torch tensors it is given
(device, dtype, shape, contiguity), passes their data pointers, sizes and the
current CUDA stream to the C entry point of the same name, and raises
``PkvError`` on a non-OK status.  Every step of the computation runs in the
library's CUDA kernels; there is no fallback.  Loading fails loudly if the
library has not been built (``python -m paged_kv_cache_246_gb300.build_lib``).
"""
from __future__ import annotations

import array
import ctypes
import functools
import operator
import os
from typing import Optional, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpkv.so")

PKV_OK, PKV_ERR_INVALID, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA, PKV_ERR_BOUNDS, PKV_ERR_TIMEOUT = range(6)
PKV_FP16, PKV_BF16 = 0, 1
PKV_CACHE_AUTO, PKV_CACHE_FP8_E4M3 = 0, 1
PKV_DECODE_STATIC_SCRATCH_BYTES = 64 << 20   # include/pkv.h: paged_attn_decode_noalloc's limit
PKV_TREE_MAX_NODES = 256        # include/pkv.h: nodes of a sequence's tree of drafted tokens
PKV_SELECT_MAX_BLOCKS = 32768   # include/pkv.h: blocks per sequence of paged_attn_select_blocks
_DTYPES = {torch.float16: PKV_FP16, torch.bfloat16: PKV_BF16}

# Every function include/pkv.h declares.
EXPORTS = ("kv_cache_write", "paged_attn_decode", "paged_attn_decode_workspace_size",
           "paged_attn_decode_noalloc", "paged_attn_decode_multi",
           "paged_attn_decode_multi_workspace_size", "paged_attn_decode_dcp_partial",
           "paged_attn_decode_dcp_workspace_size", "paged_attn_dcp_combine",
           "paged_attn_prefill_varlen", "kv_copy_blocks", "kv_swap_blocks",
           "kv_cache_write_rope", "kv_block_bounds", "paged_attn_select_blocks",
           "paged_attn_decode_sparse", "kv_cache_write_rope_axes", "paged_attn_decode_tree",
           "paged_attn_decode_tree_workspace_size", "paged_attn_tree_accept", "kv_commit_tree",
           "pkv_status_string", "pkv_device_error", "pkv_abi_version",
           "pkv_check_wait_timeout")


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class AttnParams(ctypes.Structure):
    """Mirror of pkv_attn_params."""
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_size", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("alibi_slopes", ctypes.c_void_p), ("sliding_window", ctypes.c_int32),
                ("non_causal", ctypes.c_int32), ("kv_cache_dtype", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once; raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "python -m paged_kv_cache_246_gb300.build_lib")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(AttnParams)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "kv_cache_write": (i32, [vp, vp, i64, vp, i64, vp, P, vp]),
            "paged_attn_decode": (i32, [vp, vp, i32, vp, i64, vp, i32, vp, i32, P, vp, sz, vp]),
            "paged_attn_decode_workspace_size": (sz, [i32, i32, P]),
            "paged_attn_decode_noalloc": (i32, [vp, vp, i32, vp, i64, vp, i32, vp, i32, P, vp]),
            "paged_attn_decode_multi": (i32, [vp, vp, i32, i32, vp, i64, vp, i32, vp, i32, P, vp,
                                              sz, vp]),
            "paged_attn_decode_multi_workspace_size": (sz, [i32, i32, i32, P]),
            "paged_attn_decode_dcp_partial": (i32, [vp, vp, vp, i32, i32, vp, i64, vp, i32, vp,
                                                    i32, i32, i32, P, vp, sz, vp]),
            "paged_attn_decode_dcp_workspace_size": (sz, [i32, i32, i32, i32, P]),
            "paged_attn_dcp_combine": (i32, [vp, vp, vp, i32, i64, P, vp]),
            "paged_attn_prefill_varlen": (i32, [vp, vp, i64, i32, vp, vp, i32, i32, vp, i64, vp,
                                                i32, P, vp]),
            "kv_copy_blocks": (i32, [vp, i32, i64, vp, i64, P, vp]),
            "kv_swap_blocks": (i32, [vp, i64, vp, i64, vp, i64, P, vp]),
            "kv_cache_write_rope": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, vp, i64, i32,
                                          i32, vp, i64, vp, P, vp]),
            "kv_block_bounds": (i32, [vp, vp, i64, vp, i32, vp, vp, i32, i32, P, vp]),
            "paged_attn_select_blocks": (i32, [vp, i32, vp, i32, vp, i64, vp, i32, vp, i32, i32,
                                               i32, P, vp]),
            "paged_attn_decode_sparse": (i32, [vp, vp, i32, vp, i64, vp, i32, vp, vp, i32, P, vp]),
            "kv_cache_write_rope_axes": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, i64, i32,
                                               vp, vp, i64, i32, i32, vp, i64, vp, P, vp]),
            "paged_attn_decode_tree": (i32, [vp, vp, i64, i32, vp, vp, i32, vp, i64, vp, i32, vp,
                                             i32, P, vp, sz, vp]),
            "paged_attn_decode_tree_workspace_size": (sz, [i32, i32, i32, P]),
            "paged_attn_tree_accept": (i32, [vp, i32, vp, vp, vp, vp, vp, vp, i32, i64, i32, vp]),
            "kv_commit_tree": (i32, [vp, i32, i64, vp, i32, vp, i32, vp, vp, i32, P, vp]),
            "pkv_status_string": (ctypes.c_char_p, [i32]),
            "pkv_device_error": (i32, [ctypes.POINTER(ctypes.c_int64)]),
            "pkv_abi_version": (i32, []),
            "pkv_check_wait_timeout": (i32, [i64, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pkv_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != PKV_OK:
        raise PkvError(status, where)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None, cuda=True) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def make_params(num_heads: int, num_kv_heads: int, head_size: int, block_size: int,
                dtype: torch.dtype, scale: float, alibi_slopes: Optional[torch.Tensor] = None,
                sliding_window: int = 0, non_causal: bool = False,
                kv_cache_dtype: str = "auto", k_scale: float = 1.0,
                v_scale: float = 1.0) -> AttnParams:
    """pkv_attn_params; alibi_slopes is a CUDA fp32 tensor [num_heads] or None.
    kv_cache_dtype "auto" (the model dtype) or "fp8_e4m3" (uint8 cache of
    E4M3 codes with k_scale / v_scale).

    The caller keeps alibi_slopes alive while the params are in use."""
    if kv_cache_dtype not in ("auto", "fp8_e4m3"):
        raise ValueError(f"unsupported kv_cache_dtype {kv_cache_dtype}")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    ptr = None
    if alibi_slopes is not None:
        _need(alibi_slopes, "alibi_slopes", torch.float32, 1)
        if alibi_slopes.numel() != num_heads:
            raise ValueError("alibi_slopes must have num_heads entries")
        ptr = alibi_slopes.data_ptr()
    return AttnParams(num_heads, num_kv_heads, head_size, block_size, _DTYPES[dtype],
                      float(scale), ptr, int(sliding_window or 0), int(bool(non_causal)),
                      PKV_CACHE_FP8_E4M3 if kv_cache_dtype == "fp8_e4m3" else PKV_CACHE_AUTO,
                      float(k_scale), float(v_scale))


def _cache_blocks(kv_cache: torch.Tensor, p: AttnParams) -> int:
    if kv_cache.dim() != 3 or kv_cache.shape[0] != 2:
        raise ValueError("kv_cache must be [2, num_blocks, block_size*num_kv_heads*head_size]")
    if kv_cache.shape[2] != p.block_size * p.num_kv_heads * p.head_size:
        raise ValueError("kv_cache block size does not match params")
    if kv_cache.element_size() != (1 if p.kv_cache_dtype == PKV_CACHE_FP8_E4M3 else 2):
        raise ValueError("kv_cache element size does not match kv_cache_dtype")
    return int(kv_cache.shape[1])


def kv_cache_write(key: torch.Tensor, value: torch.Tensor, kv_cache: torch.Tensor,
                   slot_mapping: torch.Tensor, params: AttnParams, stream=None) -> None:
    for t, n in ((key, "key"), (value, "value"), (kv_cache, "kv_cache")):
        _need(t, n)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    nb = _cache_blocks(kv_cache, params)
    T = key.shape[0]
    row = params.num_kv_heads * params.head_size
    if key.numel() != T * row or value.numel() != T * row or slot_mapping.numel() != T:
        raise ValueError("key/value/slot_mapping sizes disagree")
    cache_dtype = torch.uint8 if params.kv_cache_dtype == PKV_CACHE_FP8_E4M3 else key.dtype
    if value.dtype != key.dtype or kv_cache.dtype != cache_dtype:
        raise ValueError("key/value dtype must match each other and the cache")
    _check(lib().kv_cache_write(key.data_ptr(), value.data_ptr(), T, kv_cache.data_ptr(), nb,
                                slot_mapping.data_ptr(), ctypes.byref(params), _stream(stream)),
           "kv_cache_write")


def paged_attn_decode_workspace_size(num_seqs: int, max_seq_len: int, params: AttnParams) -> int:
    return int(lib().paged_attn_decode_workspace_size(num_seqs, max_seq_len,
                                                      ctypes.byref(params)))


def paged_attn_decode(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                      params: AttnParams, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    for t, n in ((out, "out"), (query, "query"), (kv_cache, "kv_cache")):
        _need(t, n)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    nb = _cache_blocks(kv_cache, params)
    B = seq_lens.numel()
    hd = params.num_heads * params.head_size
    if query.numel() != B * hd or out.numel() != B * hd or block_tables.shape[0] != B:
        raise ValueError("query/out/block_tables sizes disagree with seq_lens")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib().paged_attn_decode(out.data_ptr(), query.data_ptr(), B, kv_cache.data_ptr(), nb,
                                   block_tables.data_ptr(), int(block_tables.shape[1]),
                                   seq_lens.data_ptr(), int(max_seq_len), ctypes.byref(params),
                                   ws_ptr, ws_bytes, _stream(stream)),
           "paged_attn_decode")


def paged_attn_decode_noalloc(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                              block_tables: torch.Tensor, seq_lens: torch.Tensor,
                              max_seq_len: int, params: AttnParams, stream=None) -> None:
    """paged_attn_decode without a workspace, for callers that may not
    allocate device memory: the split partials go to the library's static
    device scratch (PKV_DECODE_STATIC_SCRATCH_BYTES per GPU, shared by all
    calls; calls that overlap on the GPU race on it).  Sizes that need more
    scratch raise PkvError with PKV_ERR_UNSUPPORTED."""
    for t, n in ((out, "out"), (query, "query"), (kv_cache, "kv_cache")):
        _need(t, n)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    nb = _cache_blocks(kv_cache, params)
    B = seq_lens.numel()
    hd = params.num_heads * params.head_size
    if query.numel() != B * hd or out.numel() != B * hd or block_tables.shape[0] != B:
        raise ValueError("query/out/block_tables sizes disagree with seq_lens")
    _check(lib().paged_attn_decode_noalloc(out.data_ptr(), query.data_ptr(), B,
                                           kv_cache.data_ptr(), nb, block_tables.data_ptr(),
                                           int(block_tables.shape[1]), seq_lens.data_ptr(),
                                           int(max_seq_len), ctypes.byref(params),
                                           _stream(stream)),
           "paged_attn_decode_noalloc")


def paged_attn_decode_multi_workspace_size(num_seqs: int, query_len: int, max_seq_len: int,
                                           params: AttnParams) -> int:
    return int(lib().paged_attn_decode_multi_workspace_size(num_seqs, query_len, max_seq_len,
                                                            ctypes.byref(params)))


def paged_attn_decode_multi(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor, query_len: int,
                            max_seq_len: int, params: AttnParams,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Uniform batch of decodes of query_len tokens per sequence; query/out
    rows b * query_len + t."""
    for t, n in ((out, "out"), (query, "query"), (kv_cache, "kv_cache")):
        _need(t, n)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    nb = _cache_blocks(kv_cache, params)
    B = seq_lens.numel()
    hd = params.num_heads * params.head_size
    rows = B * int(query_len)
    if query.numel() != rows * hd or out.numel() != rows * hd or block_tables.shape[0] != B:
        raise ValueError("query/out/block_tables sizes disagree with seq_lens and query_len")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib().paged_attn_decode_multi(out.data_ptr(), query.data_ptr(), B, int(query_len),
                                         kv_cache.data_ptr(), nb, block_tables.data_ptr(),
                                         int(block_tables.shape[1]), seq_lens.data_ptr(),
                                         int(max_seq_len), ctypes.byref(params), ws_ptr, ws_bytes,
                                         _stream(stream)),
           "paged_attn_decode_multi")


def paged_attn_decode_dcp_workspace_size(num_seqs: int, query_len: int, max_seq_len: int,
                                         dcp_world_size: int, params: AttnParams) -> int:
    return int(lib().paged_attn_decode_dcp_workspace_size(num_seqs, query_len, max_seq_len,
                                                          dcp_world_size, ctypes.byref(params)))


def paged_attn_decode_dcp_partial(part_o: torch.Tensor, part_ml: torch.Tensor,
                                  query: torch.Tensor, kv_cache: torch.Tensor,
                                  block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                  query_len: int, max_seq_len: int, dcp_world_size: int,
                                  dcp_rank: int, params: AttnParams,
                                  workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """This rank's share (fp32 o [rows * heads, head_size], (m, l) [rows * heads, 2])
    of a decode whose sequences' tokens are spread over dcp_world_size ranks;
    seq_lens are the global lengths, kv_cache / block_tables the rank's own."""
    for t, n in ((query, "query"), (kv_cache, "kv_cache")):
        _need(t, n)
    _need(part_o, "part_o", torch.float32)
    _need(part_ml, "part_ml", torch.float32)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    nb = _cache_blocks(kv_cache, params)
    B = seq_lens.numel()
    rows = B * int(query_len)
    hd = params.num_heads * params.head_size
    if (query.numel() != rows * hd or part_o.numel() != rows * hd or
            part_ml.numel() != rows * params.num_heads * 2 or block_tables.shape[0] != B):
        raise ValueError("query/part_o/part_ml/block_tables sizes disagree")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _need(workspace, "workspace")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib().paged_attn_decode_dcp_partial(
        part_o.data_ptr(), part_ml.data_ptr(), query.data_ptr(), B, int(query_len),
        kv_cache.data_ptr(), nb, block_tables.data_ptr(), int(block_tables.shape[1]),
        seq_lens.data_ptr(), int(max_seq_len), int(dcp_world_size), int(dcp_rank),
        ctypes.byref(params), ws_ptr, ws_bytes, _stream(stream)), "paged_attn_decode_dcp_partial")


def paged_attn_dcp_combine(out: torch.Tensor, parts_o: torch.Tensor, parts_ml: torch.Tensor,
                           params: AttnParams, stream=None) -> None:
    """out [rows, heads * head_size] from the ranks' shares stacked rank-major:
    parts_o [P, rows * heads, head_size], parts_ml [P, rows * heads, 2]."""
    _need(out, "out")
    _need(parts_o, "parts_o", torch.float32)
    _need(parts_ml, "parts_ml", torch.float32)
    P = int(parts_o.shape[0])
    rh = params.num_heads
    rows = out.numel() // (rh * params.head_size)
    if (parts_o.numel() != P * rows * rh * params.head_size or
            parts_ml.numel() != P * rows * rh * 2):
        raise ValueError("parts_o/parts_ml sizes disagree with out")
    _check(lib().paged_attn_dcp_combine(out.data_ptr(), parts_o.data_ptr(), parts_ml.data_ptr(),
                                        P, rows, ctypes.byref(params), _stream(stream)),
           "paged_attn_dcp_combine")


def paged_attn_prefill_varlen(out: torch.Tensor, query: torch.Tensor, cu_seqlens_q: torch.Tensor,
                              cu_seqlens_k: torch.Tensor, max_query_len: int, max_seq_len: int,
                              kv_cache: torch.Tensor, block_tables: torch.Tensor,
                              params: AttnParams, stream=None) -> None:
    for t, n in ((out, "out"), (query, "query"), (kv_cache, "kv_cache")):
        _need(t, n)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    nb = _cache_blocks(kv_cache, params)
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1 or block_tables.shape[0] < B or out.shape != query.shape:
        raise ValueError("cu_seqlens/block_tables/out sizes disagree")
    rows = query.shape[0]
    if query.numel() != rows * params.num_heads * params.head_size:
        raise ValueError("query must be [num_query_tokens, num_heads * head_size]")
    _check(lib().paged_attn_prefill_varlen(out.data_ptr(), query.data_ptr(), rows, B,
                                           cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                           int(max_query_len), int(max_seq_len),
                                           kv_cache.data_ptr(), nb, block_tables.data_ptr(),
                                           int(block_tables.shape[1]), ctypes.byref(params),
                                           _stream(stream)),
           "paged_attn_prefill_varlen")


def kv_copy_blocks(kv_caches: Sequence[torch.Tensor], pairs: torch.Tensor, params: AttnParams,
                   stream=None) -> None:
    if len(kv_caches) == 0:
        return
    nb = None
    for k, c in enumerate(kv_caches):
        _need(c, f"kv_caches[{k}]")
        n = _cache_blocks(c, params)
        if nb is not None and n != nb:
            raise ValueError("all caches must have the same number of blocks")
        nb = n
    _need(pairs, "pairs", torch.int64, 2)
    arr = (ctypes.c_void_p * len(kv_caches))(*[c.data_ptr() for c in kv_caches])
    _check(lib().kv_copy_blocks(arr, len(kv_caches), nb, pairs.data_ptr(), int(pairs.shape[0]),
                                ctypes.byref(params), _stream(stream)),
           "kv_copy_blocks")


def kv_swap_blocks(src_cache: torch.Tensor, dst_cache: torch.Tensor, pairs: torch.Tensor,
                   params: AttnParams, stream=None) -> None:
    """pairs: CPU int64 [n, 2]; src/dst: CUDA tensors or pinned CPU tensors."""
    for t, n in ((src_cache, "src_cache"), (dst_cache, "dst_cache")):
        _need(t, n, cuda=False)
        if not t.is_cuda and not t.is_pinned():
            raise ValueError(f"{n} must be a CUDA tensor or pinned host memory")
    _need(pairs, "pairs", torch.int64, 2, cuda=False)
    if pairs.is_cuda:
        raise ValueError("swap pairs are read on the host: pass a CPU tensor")
    sb, db = _cache_blocks(src_cache, params), _cache_blocks(dst_cache, params)
    _check(lib().kv_swap_blocks(src_cache.data_ptr(), sb, dst_cache.data_ptr(), db,
                                pairs.data_ptr(), int(pairs.shape[0]), ctypes.byref(params),
                                _stream(stream)),
           "kv_swap_blocks")


# ---------------------------------------------------------------------------
# Block-sparse decode: cache write with the rotation, block bounds, block
# selection, attention over the selected blocks.  These calls run on the
# device that holds their tensors, whichever is current; a stream given by
# the caller must belong to it.
# ---------------------------------------------------------------------------
_Tensor = torch.Tensor
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no Stream object made on the way


def _current_stream(index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


@functools.lru_cache(maxsize=None)
def _one_gpu() -> bool:
    return torch.cuda.device_count() == 1


def _call_on(where: str, stream, tensors: Sequence[torch.Tensor], *args):
    """The entry point `where` on the device that holds `tensors`."""
    index = -1
    for t in tensors:
        at = t.get_device()
        if at != index or at < 0:
            if index >= 0 or at < 0:
                raise ValueError(f"{where}: tensors must be on one CUDA device, not "
                                 f"{tensors[0].device} and {t.device}")
            index = at
    if stream is None:
        handle = _current_stream(index)
    else:
        if getattr(stream, "device", tensors[0].device) != tensors[0].device:
            raise ValueError(f"{where}: a stream of {stream.device} for tensors on "
                             f"{tensors[0].device}")
        handle = _stream(stream)
    fn = getattr(lib(), where)
    if _one_gpu() or torch.cuda.current_device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != PKV_OK:
        raise PkvError(st, where)


_TORCH_DTYPES = {code: dtype for dtype, code in _DTYPES.items()}


@functools.lru_cache(maxsize=64)
def _facts_of(raw: bytes) -> tuple:
    p = AttnParams.from_buffer_copy(raw)
    dtype = _TORCH_DTYPES.get(p.dtype)
    if dtype is None:
        raise ValueError(f"unsupported params dtype {p.dtype}")
    return (dtype, torch.uint8 if p.kv_cache_dtype == PKV_CACHE_FP8_E4M3 else dtype,
            p.num_kv_heads, p.head_size, p.num_heads * p.head_size, p.num_kv_heads * p.head_size,
            p.block_size * p.num_kv_heads * p.head_size)


def _facts(p: AttnParams) -> tuple:
    """(dtype of queries, keys, values and outputs; dtype of the cache; KV
    heads; head size; elements of a query row, a key row, a cache block)."""
    return _facts_of(bytes(p))


def _is(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> tuple:
    """The sizes of a contiguous tensor of this type (its device is checked at the call)."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.is_contiguous():
        shape = t.shape
        if len(shape) == ndim:
            return shape
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} must be contiguous, {dtype}, of {ndim} dims; got "
                     f"{'contiguous' if t.is_contiguous() else 'strided'}, {t.dtype}, {list(t.shape)}")


def _int32(value, name: str) -> int:
    """ctypes would cut it to 32 bits."""
    value = int(value)
    if not -0x80000000 <= value <= 0x7fffffff:
        raise ValueError(f"{name} must fit in 32 bits, got {value}")
    return value


def _is_cache(t: torch.Tensor, dtype: torch.dtype, block: int) -> int:
    two, blocks, elems = _is(t, "kv_cache", dtype, 3)
    if two != 2 or elems != block:
        raise ValueError("kv_cache must be [2, num_blocks, block_size*num_kv_heads*head_size]")
    return blocks


def _is_batch(block_tables: torch.Tensor, seq_lens: torch.Tensor) -> tuple:
    n, wide = _is(block_tables, "block_tables", torch.int32, 2)
    if _is(seq_lens, "seq_lens", torch.int32, 1)[0] != n:
        raise ValueError("block_tables and seq_lens sizes disagree")
    return n, wide


def _row_stride(t: torch.Tensor, name: str, rows: int, row: int, dtype: torch.dtype) -> int:
    """Elements between the rows of a [rows, row] tensor whose rows may be
    slices of wider ones."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, row):
        raise ValueError(f"{name} must be [{rows}, {row}], got {list(t.shape)}")
    stride, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if rows <= 1:
        return row
    if stride < row or stride % 8 != 0:
        raise ValueError(f"{name}'s rows must not overlap and start a multiple of 8 elements apart")
    return stride


def rope_table(max_position: int, rot_dim: int, base: float = 10000.0, position_scale: float = 1.0,
               device="cuda") -> torch.Tensor:
    """The cos_sin table of kv_cache_write_rope: fp32 [max_position, rot_dim],
    row p = rot_dim / 2 cosines, then sines, of the angles position_scale * p *
    base^(-2i / rot_dim).  Angles are taken in 64 bits: in 32 those of far
    positions are off by more than the table's rounding."""
    if max_position <= 0 or rot_dim <= 0 or rot_dim % 2:
        raise ValueError("max_position and rot_dim must be positive, rot_dim even")
    f = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = (torch.arange(max_position, dtype=torch.float64, device=device) * position_scale)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32)


def kv_cache_write_rope(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                        value: torch.Tensor, kv_cache: torch.Tensor, slot_mapping: torch.Tensor,
                        positions: torch.Tensor, cos_sin: torch.Tensor, params: AttnParams,
                        interleaved: bool = False, stream=None) -> None:
    """kv_cache_write with queries and keys rotated by their positions: rows of
    query, key and value may be slices of one projection's output; query_out
    may be query."""
    dtype, cache_dtype, _, _, q_row, kv_row, block = _facts(params)
    nb = _is_cache(kv_cache, cache_dtype, block)
    T = _is(slot_mapping, "slot_mapping", torch.int64, 1)[0]
    if _is(positions, "positions", torch.int64, 1)[0] != T:
        raise ValueError("positions and slot_mapping sizes disagree")
    max_position, rot_dim = _is(cos_sin, "cos_sin", torch.float32, 2)
    so = _row_stride(query_out, "query_out", T, q_row, dtype)
    sq = _row_stride(query, "query", T, q_row, dtype)
    sk = _row_stride(key, "key", T, kv_row, dtype)
    sv = _row_stride(value, "value", T, kv_row, dtype)
    _call_on("kv_cache_write_rope", stream,
             (kv_cache, query_out, query, key, value, slot_mapping, positions, cos_sin),
             query_out.data_ptr(), so, query.data_ptr(), sq, key.data_ptr(), sk, value.data_ptr(),
             sv, T, positions.data_ptr(), cos_sin.data_ptr(), max_position, rot_dim,
             1 if interleaved else 0, kv_cache.data_ptr(), nb, slot_mapping.data_ptr(),
             ctypes.byref(params))


def _is_bounds(bounds: torch.Tensor, dtype: torch.dtype, kv_heads: int, head_size: int) -> int:
    blocks, heads, two, size = _is(bounds, "bounds", dtype, 4)
    if heads != kv_heads or two != 2 or size != head_size:
        raise ValueError("bounds must be [num_blocks, num_kv_heads, 2, head_size]")
    return blocks


def kv_block_bounds(bounds: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                    seq_lens: torch.Tensor, max_new_tokens: int, params: AttnParams,
                    context_lens: Optional[torch.Tensor] = None, stream=None) -> None:
    """Channelwise minima and maxima of the keys of the blocks that hold
    positions context_lens[b] .. seq_lens[b] - 1 (None: all of the sequence)."""
    _, cache_dtype, kv_heads, head_size, _, _, block = _facts(params)
    nb = _is_cache(kv_cache, cache_dtype, block)
    if _is_bounds(bounds, cache_dtype, kv_heads, head_size) != nb:
        raise ValueError("bounds and kv_cache must have the same number of blocks")
    n, wide = _is_batch(block_tables, seq_lens)
    tensors, ctx = (kv_cache, bounds, block_tables, seq_lens), None
    if context_lens is not None:
        if _is(context_lens, "context_lens", torch.int32, 1)[0] != n:
            raise ValueError("context_lens and seq_lens sizes disagree")
        tensors, ctx = tensors + (context_lens,), context_lens.data_ptr()
    _call_on("kv_block_bounds", stream, tensors, bounds.data_ptr(), kv_cache.data_ptr(), nb,
             block_tables.data_ptr(), wide, ctx, seq_lens.data_ptr(), n,
             _int32(max_new_tokens, "max_new_tokens"), ctypes.byref(params))


def _is_selected(selected: torch.Tensor, n: int, kv_heads: int) -> int:
    seqs, heads, k = _is(selected, "selected", torch.int32, 3)
    if seqs != n or heads != kv_heads:
        raise ValueError("selected must be [num_seqs, num_kv_heads, max_selected]")
    return k


def _is_rows(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, q_row: int) -> None:
    rows, row = _is(t, name, dtype, 2)
    if rows != n or row != q_row:
        raise ValueError(f"{name} must be [num_seqs, num_heads*head_size]")


def paged_attn_select_blocks(selected: torch.Tensor, query: torch.Tensor, bounds: torch.Tensor,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                             params: AttnParams, num_sink: int = 0, num_recent: int = 1,
                             stream=None) -> None:
    """selected [num_seqs, num_kv_heads, K]: each KV head's K blocks with the
    largest bound on q.k, the first num_sink and last num_recent among them,
    ascending, -1 behind."""
    dtype, cache_dtype, kv_heads, head_size, q_row, _, _ = _facts(params)
    nb = _is_bounds(bounds, cache_dtype, kv_heads, head_size)
    n, wide = _is_batch(block_tables, seq_lens)
    k = _is_selected(selected, n, kv_heads)
    _is_rows(query, "query", dtype, n, q_row)
    _call_on("paged_attn_select_blocks", stream, (bounds, selected, query, block_tables, seq_lens),
             selected.data_ptr(), k, query.data_ptr(), n, bounds.data_ptr(), nb,
             block_tables.data_ptr(), wide, seq_lens.data_ptr(), _int32(max_seq_len, "max_seq_len"),
             _int32(num_sink, "num_sink"), _int32(num_recent, "num_recent"), ctypes.byref(params))


def paged_attn_decode_sparse(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor,
                             selected: torch.Tensor, params: AttnParams, stream=None) -> None:
    """paged_attn_decode over the blocks that selected [num_seqs, num_kv_heads,
    K] names for each sequence and KV head (ascending, negative numbers behind)."""
    dtype, cache_dtype, kv_heads, _, q_row, _, block = _facts(params)
    nb = _is_cache(kv_cache, cache_dtype, block)
    n, wide = _is_batch(block_tables, seq_lens)
    k = _is_selected(selected, n, kv_heads)
    _is_rows(out, "out", dtype, n, q_row)
    _is_rows(query, "query", dtype, n, q_row)
    _call_on("paged_attn_decode_sparse", stream,
             (kv_cache, out, query, block_tables, seq_lens, selected), out.data_ptr(),
             query.data_ptr(), n, kv_cache.data_ptr(), nb, block_tables.data_ptr(), wide,
             seq_lens.data_ptr(), selected.data_ptr(), k, ctypes.byref(params))


# ---------------------------------------------------------------------------
# Speculative decoding over trees of drafted tokens: cache write with positions
# of several axes, attention, acceptance, commit of the accepted path.  As the
# calls above they run on the device that holds their tensors.
# ---------------------------------------------------------------------------
def rope_pair_axes(sections: Sequence[int], woven: bool = False) -> tuple:
    """The pair_axes of kv_cache_write_rope_axes for sections[a] pairs of axis
    a: behind one another, or woven, where axis 0 has all pairs but i = a,
    a + n, a + 2n, ... (n axes), of which axis a > 0 has the first sections[a]."""
    sections = [int(x) for x in sections]
    if not 1 <= len(sections) <= 4 or min(sections) < 0:
        raise ValueError("sections must be 1 to 4 counts of pairs")
    if not woven:
        return tuple(a for a, n in enumerate(sections) for _ in range(n))
    n = len(sections)
    return tuple(i % n if i < n * sections[i % n] else 0 for i in range(sum(sections)))


@functools.lru_cache(maxsize=64)
def _pair_axes(axes: bytes) -> tuple:
    """(array for the call, axes that it names)"""
    if not axes or max(axes) >= 4:
        raise ValueError("pair_axes must name an axis 0 .. 3 for every pair of channels")
    return (ctypes.c_uint8 * len(axes))(*axes), max(axes) + 1


def _positions(positions: torch.Tensor, T: int) -> tuple:
    """Axes, and elements from one axis to the next, of [axes, T] positions."""
    if not isinstance(positions, _Tensor):
        raise TypeError("positions must be a torch.Tensor")
    if positions.dtype is not torch.int64 or positions.dim() != 2 or positions.shape[1] != T:
        raise ValueError(f"positions must be {torch.int64} [axes, {T}], got {positions.dtype} "
                         f"{list(positions.shape)}")
    axes = positions.shape[0]
    if positions.is_contiguous():
        return axes, T
    stride, one = positions.stride()
    if (T > 1 and one != 1) or (axes > 1 and stride < T):
        raise ValueError("each axis's positions must be contiguous, and behind the one before")
    return axes, max(stride, T)


def kv_cache_write_rope_axes(query_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                             value: torch.Tensor, kv_cache: torch.Tensor, slot_mapping: torch.Tensor,
                             positions: torch.Tensor, cos_sin: torch.Tensor,
                             pair_axes: Sequence[int], params: AttnParams,
                             interleaved: bool = False, stream=None) -> None:
    """kv_cache_write_rope with positions [num_axes, T], whose rows may be slices
    of wider ones: pair i of a head turns by the position on axis pair_axes[i]
    (rope_pair_axes makes the list)."""
    dtype, cache_dtype, _, _, q_row, kv_row, block = _facts(params)
    nb = _is_cache(kv_cache, cache_dtype, block)
    T = _is(slot_mapping, "slot_mapping", torch.int64, 1)[0]
    axes, axis_stride = _positions(positions, T)
    max_position, rot_dim = _is(cos_sin, "cos_sin", torch.float32, 2)
    if type(pair_axes) not in (tuple, list, bytes):
        # bytes() of a number are as many zeros, of an array its memory
        pair_axes = tuple(map(operator.index, pair_axes))
    axis_array, named = _pair_axes(bytes(pair_axes))
    if len(axis_array) != rot_dim // 2 or named > axes:
        raise ValueError(f"pair_axes must name one of the {axes} axes for each of the "
                         f"{rot_dim // 2} pairs")
    so = _row_stride(query_out, "query_out", T, q_row, dtype)
    sq = _row_stride(query, "query", T, q_row, dtype)
    sk = _row_stride(key, "key", T, kv_row, dtype)
    sv = _row_stride(value, "value", T, kv_row, dtype)
    _call_on("kv_cache_write_rope_axes", stream,
             (kv_cache, query_out, query, key, value, slot_mapping, positions, cos_sin),
             query_out.data_ptr(), so, query.data_ptr(), sq, key.data_ptr(), sk, value.data_ptr(),
             sv, T, positions.data_ptr(), axis_stride, axes, axis_array, cos_sin.data_ptr(), max_position, rot_dim,
             1 if interleaved else 0, kv_cache.data_ptr(), nb, slot_mapping.data_ptr(),
             ctypes.byref(params))


def paged_attn_decode_tree_workspace_size(num_seqs: int, max_nodes: int, max_seq_len: int,
                                          params: AttnParams) -> int:
    return int(lib().paged_attn_decode_tree_workspace_size(
        _int32(num_seqs, "num_seqs"), _int32(max_nodes, "max_nodes"),
        _int32(max_seq_len, "max_seq_len"), ctypes.byref(params)))


def _is_trees(cu_nodes: torch.Tensor, n: int) -> None:
    if _is(cu_nodes, "cu_nodes", torch.int32, 1)[0] != n + 1:
        raise ValueError("cu_nodes must be [num_seqs + 1]")


def paged_attn_decode_tree(out: torch.Tensor, query: torch.Tensor, kv_cache: torch.Tensor,
                           block_tables: torch.Tensor, seq_lens: torch.Tensor,
                           cu_nodes: torch.Tensor, parents: torch.Tensor, max_nodes: int,
                           max_seq_len: int, params: AttnParams,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Every node of each sequence's tree of drafted tokens attends to the
    context, its ancestors and itself.  Node t of sequence b has row cu_nodes[b]
    + t of query and out, stands in the cache at position seq_lens[b] - nodes +
    t, and parents (numbers within the tree, -1: none) may be longer than the
    trees, as the rows may."""
    dtype, cache_dtype, _, _, q_row, _, block = _facts(params)
    nb = _is_cache(kv_cache, cache_dtype, block)
    n, wide = _is_batch(block_tables, seq_lens)
    _is_trees(cu_nodes, n)
    T = _is(query, "query", dtype, 2)[0]
    _is_rows(out, "out", dtype, T, q_row)
    _is_rows(query, "query", dtype, T, q_row)
    # rows behind the last tree have no parents
    T = min(T, _is(parents, "parents", torch.int32, 1)[0])
    tensors, ws_ptr, ws_bytes = (kv_cache, out, query, block_tables, seq_lens, cu_nodes, parents), None, 0
    if workspace is not None:
        _need(workspace, "workspace")
        tensors = tensors + (workspace,)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call_on("paged_attn_decode_tree", stream, tensors, out.data_ptr(), query.data_ptr(), T, n,
             cu_nodes.data_ptr(), parents.data_ptr(), _int32(max_nodes, "max_nodes"),
             kv_cache.data_ptr(), nb, block_tables.data_ptr(), wide, seq_lens.data_ptr(),
             _int32(max_seq_len, "max_seq_len"), ctypes.byref(params), ws_ptr, ws_bytes)


def paged_attn_tree_accept(accepted: torch.Tensor, num_accepted: torch.Tensor,
                           next_token: torch.Tensor, draft_tokens: torch.Tensor,
                           target_tokens: torch.Tensor, parents: torch.Tensor,
                           cu_nodes: torch.Tensor, max_nodes: int, stream=None) -> None:
    """accepted [num_seqs, K]: the path from node 0 along the children whose
    drafted token is the one sampled at their parent, -1 behind it; num_accepted
    [num_seqs] its nodes, next_token [num_seqs] the token sampled at its end."""
    n, most = _is(accepted, "accepted", torch.int32, 2)
    if (_is(num_accepted, "num_accepted", torch.int32, 1)[0] != n or
            _is(next_token, "next_token", torch.int64, 1)[0] != n):
        raise ValueError("accepted, num_accepted and next_token sizes disagree")
    _is_trees(cu_nodes, n)
    T = _is(draft_tokens, "draft_tokens", torch.int64, 1)[0]
    if (_is(target_tokens, "target_tokens", torch.int64, 1)[0] != T or
            _is(parents, "parents", torch.int32, 1)[0] != T):
        raise ValueError("draft_tokens, target_tokens and parents sizes disagree")
    _call_on("paged_attn_tree_accept", stream,
             (accepted, num_accepted, next_token, draft_tokens, target_tokens, parents, cu_nodes),
             accepted.data_ptr(), most, num_accepted.data_ptr(), next_token.data_ptr(),
             draft_tokens.data_ptr(), target_tokens.data_ptr(), parents.data_ptr(),
             cu_nodes.data_ptr(), n, T, _int32(max_nodes, "max_nodes"))


_get_dtype, _get_shape = operator.attrgetter("dtype"), operator.attrgetter("shape")
_is_contiguous, _get_device = torch.Tensor.is_contiguous, torch.Tensor.get_device
_data_ptr = torch.Tensor.data_ptr


def kv_commit_tree(kv_caches: Sequence[torch.Tensor], accepted: torch.Tensor,
                   block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_nodes: torch.Tensor,
                   params: AttnParams, stream=None) -> None:
    """In every layer's cache, each sequence's rows of the nodes accepted [num_seqs,
    K] (as paged_attn_tree_accept gives them) move behind its context."""
    if len(kv_caches) == 0:
        return
    _, cache_dtype, _, _, _, _, block = _facts(params)
    nb = _is_cache(kv_caches[0], cache_dtype, block)
    # a call a layer and check, without the interpreter between them
    if (set(map(_get_dtype, kv_caches)) != {cache_dtype} or not all(map(_is_contiguous, kv_caches)) or
            any(map(kv_caches[0].shape.__ne__, map(_get_shape, kv_caches)))):
        raise ValueError("all caches must be contiguous, of the cache's type and of one shape")
    if set(map(_get_device, kv_caches)) != {kv_caches[0].get_device()}:
        raise ValueError("kv_commit_tree: all caches must be on one CUDA device")
    n, wide = _is_batch(block_tables, seq_lens)
    seqs, most = _is(accepted, "accepted", torch.int32, 2)
    if seqs != n:
        raise ValueError("accepted must be [num_seqs, max_accepted]")
    _is_trees(cu_nodes, n)
    pointers = array.array("Q", map(_data_ptr, kv_caches))
    _call_on("kv_commit_tree", stream, (kv_caches[0], accepted, block_tables, seq_lens, cu_nodes),
             pointers.buffer_info()[0], len(kv_caches), nb, accepted.data_ptr(), most,
             block_tables.data_ptr(), wide, seq_lens.data_ptr(), cu_nodes.data_ptr(), n,
             ctypes.byref(params))


def check_wait_timeout(tag: int, stream=None) -> None:
    """Launch the bounded wait that nothing completes (pkv_check_wait_timeout)."""
    _check(lib().pkv_check_wait_timeout(int(tag), _stream(stream)), "pkv_check_wait_timeout")


def device_error() -> tuple[int, int]:
    """(status, detail) of the sticky device error word; reading clears it."""
    d = ctypes.c_int64(0)
    st = lib().pkv_device_error(ctypes.byref(d))
    return int(st), int(d.value)


def check_device_error(where: str = "device") -> None:
    st, d = device_error()
    if st != PKV_OK:
        raise PkvError(st, f"{where} (first bad index {d})")

"""Plain fp64 CPU restatement of the block-sparse decode over a paged cache:
the cache write with the rotary embedding, block bounds, block selection and
the decode over the selected blocks.

TEST INFRASTRUCTURE ONLY, like ``paged_attention``: it shares no code with the
CUDA path.  Readings taken:

* rotation: pair i < r / 2 of a head of which the first r channels rotate is
  (i, i + r / 2), or (2i, 2i + 1) interleaved; the pair turns by the angle whose
  cosine and sine stand in the position's table row.
* a padding token (slot < 0) is skipped: neither its query row nor the cache
  changes.
* block bounds: over the keys the sequence has in the block, slots past its
  end not read; NaN if any of them is NaN.
* a block's score is an upper bound of q.k for all its keys and all query
  heads of the KV head; equal scores go to the lower block; NaN counts as
  +infinity.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from .paged_attention import (F64, AttnParams, _dequant, _slope, alibi_bias, cache_row,
                              decode_position, kv_head_of, slot_location, window_lo)

__all__ = ["rope_pair", "rope_rotate", "kv_cache_write_rope", "kv_block_bounds", "block_score",
           "paged_attn_select_blocks", "paged_attn_decode_sparse"]


def rope_pair(i: int, rot_dim: int, interleaved: bool) -> tuple[int, int]:
    """The channels of pair i."""
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)


def rope_rotate(x: torch.Tensor, table_row: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """x [heads, D] fp64, turned by one position's [rot_dim] cosines and sines."""
    r = table_row.shape[0]
    y = x.clone()
    for i in range(r // 2):
        a, b = rope_pair(i, r, interleaved)
        c, s = float(table_row[i]), float(table_row[r // 2 + i])
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def kv_cache_write_rope(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                        slot_mapping: torch.Tensor, positions: torch.Tensor,
                        cos_sin: torch.Tensor, p: AttnParams, interleaved: bool):
    """Unrounded results per token: rotated queries [T, H * D], what the key
    slot and the value slot hold [T, KVH * D] (over an fp8 cache the quotients
    by the scales that the codes round); rows of padding tokens are NaN."""
    T, D = query.shape[0], p.head_size
    q = torch.full((T, p.num_heads * D), float("nan"), dtype=F64)
    k = torch.full((T, p.row_elems), float("nan"), dtype=F64)
    v = torch.full((T, p.row_elems), float("nan"), dtype=F64)
    fp8 = p.kv_cache_dtype == "fp8_e4m3"
    for t in range(T):
        if int(slot_mapping[t]) < 0:
            continue
        row = cos_sin[int(positions[t])]
        q[t] = rope_rotate(query[t].to(F64).view(-1, D), row, interleaved).reshape(-1)
        k[t] = rope_rotate(key[t].to(F64).view(-1, D), row, interleaved).reshape(-1)
        v[t] = value[t].to(F64)
        if fp8:
            k[t] /= torch.tensor(p.k_scale, dtype=torch.float32).to(F64)
            v[t] /= torch.tensor(p.v_scale, dtype=torch.float32).to(F64)
    return q, k, v


def _values(rows: torch.Tensor, p: AttnParams, scale: float = 1.0) -> torch.Tensor:
    return _dequant(rows, scale) if p.kv_cache_dtype == "fp8_e4m3" else rows.to(F64)


def kv_block_bounds(bounds: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                    seq_lens: torch.Tensor, p: AttnParams,
                    context_lens: Optional[torch.Tensor] = None) -> None:
    """bounds [num_blocks, KVH, 2, D] in fp64 (values; over an fp8 cache those
    of the codes), the blocks with positions context_len .. seq_len - 1 done,
    in place."""
    BS, KVH, D = p.block_size, p.num_kv_heads, p.head_size
    for b in range(seq_lens.numel()):
        L = int(seq_lens[b])
        ctx = 0 if context_lens is None else int(context_lens[b])
        for lb in sorted({j // BS for j in range(ctx, L)}):
            pb = int(block_tables[b, lb])
            rows = [_values(cache_row(kv_cache, 0, pb, t, p), p).view(KVH, D)
                    for t in range(min(BS, L - lb * BS))]
            lo, hi = rows[0].clone(), rows[0].clone()
            for r in rows[1:]:
                lo, hi = torch.minimum(lo, r), torch.maximum(hi, r)   # both keep NaN
            bounds[pb, :, 0], bounds[pb, :, 1] = lo, hi


def block_score(q: torch.Tensor, lo: torch.Tensor, hi: torch.Tensor) -> float:
    """max over heads h of sum_d max(q_hd lo_d, q_hd hi_d); q [heads, D], fp64."""
    s = torch.maximum(q * lo, q * hi).sum(1)
    return float("inf") if bool(torch.isnan(s).any()) else float(s.max())


def paged_attn_select_blocks(query: torch.Tensor, bounds: torch.Tensor,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor,
                             max_selected: int, num_sink: int, num_recent: int,
                             p: AttnParams) -> torch.Tensor:
    """int32 [num_seqs, KVH, max_selected]; bounds as values, any dtype."""
    BS, D, g = p.block_size, p.head_size, p.queries_per_kv
    out = torch.full((seq_lens.numel(), p.num_kv_heads, max_selected), -1, dtype=torch.int32)
    for b in range(seq_lens.numel()):
        L = int(seq_lens[b])
        if L == 0:
            continue
        blocks = range(window_lo(L - 1, p.sliding_window) // BS, (L - 1) // BS + 1)
        always = [j for j in blocks if j < num_sink or j > blocks[-1] - num_recent]
        for h in range(p.num_kv_heads):
            q = query[b].to(F64).view(-1, D)[h * g:(h + 1) * g]
            rest = [j for j in blocks if j not in always]
            room = max_selected - len(always)
            if len(rest) > room:
                def order(j):
                    pb = int(block_tables[b, j])
                    return -block_score(q, bounds[pb, h, 0].to(F64), bounds[pb, h, 1].to(F64)), j
                rest = sorted(rest, key=order)[:room]
            chosen = sorted(always + rest)
            out[b, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return out


def paged_attn_decode_sparse(query: torch.Tensor, kv_cache: torch.Tensor,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor,
                             selected: torch.Tensor, p: AttnParams,
                             seqs: Optional[Sequence[int]] = None):
    """(out, spread), fp64 [num_seqs, H * D]: the attention of each query head
    over the keys of its KV head's selected blocks, and sum_j p_j |v_j|, by
    which rounding the weights p_j may move it; rows not in ``seqs`` are NaN."""
    n, H, D, BS = seq_lens.numel(), p.num_heads, p.head_size, p.block_size
    out = torch.full((n, H * D), float("nan"), dtype=F64)
    spread = torch.full_like(out, float("nan"))
    for b in (range(n) if seqs is None else seqs):
        L = int(seq_lens[b])
        out[b] = spread[b] = 0.0
        i = decode_position(L)
        for h in range(H):
            g = kv_head_of(h, p.queries_per_kv)
            keys = [j for s in selected[b, g].tolist() if s >= 0
                    for j in range(s * BS, min((s + 1) * BS, L))
                    if j >= window_lo(i, p.sliding_window)]
            if not keys:
                continue
            k, v = (torch.stack([_values(cache_row(kv_cache, half, *slot_location(
                int(block_tables[b, j // BS]) * BS + j % BS, BS), p)[g * D:(g + 1) * D], p, scale)
                for j in keys]) for half, scale in ((0, p.k_scale), (1, p.v_scale)))
            s = p.scale * (k @ query[b, h * D:(h + 1) * D].to(F64))
            if _slope(p, h) is not None:
                s = s + alibi_bias(_slope(p, h), torch.tensor(keys, dtype=F64), i)
            w = torch.softmax(s, 0)
            out[b, h * D:(h + 1) * D] = w @ v
            spread[b, h * D:(h + 1) * D] = w @ v.abs()
    return out, spread

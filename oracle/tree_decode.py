"""Plain fp64 CPU restatement of a speculative step over trees of drafted
tokens: the cache write with positions of several axes, attention of the nodes,
acceptance of drafted tokens and the commit of the accepted path.

TEST INFRASTRUCTURE ONLY, like ``paged_attention``: it shares no code with the
CUDA path.  Readings taken:

* a tree's nodes are numbered so that parents come before their children; a
  node without a parent (-1) is a child of the context's last token.
* node t is stored at position context + t; its position for the rotary
  embedding, the window and ALiBi is context + depth, so that a path of the
  tree looks like the run of tokens that it would be.
* a node sees the context, its ancestors and itself, those of them that are
  inside its window.
* the walk of the acceptance starts at node 0, which holds the last sampled
  token, and prefers the lowest of several children with the right token.
"""
from __future__ import annotations

import torch

from .paged_attention import F64, AttnParams, _dequant, _slope, kv_head_of
from .sparse_decode import rope_rotate

__all__ = ["kv_cache_write_rope_axes", "tree_ancestors", "paged_attn_decode_tree",
           "paged_attn_tree_accept", "kv_commit_tree"]


def kv_cache_write_rope_axes(query, key, value, slot_mapping, positions, cos_sin, pair_axes,
                             p: AttnParams, interleaved: bool):
    """As kv_cache_write_rope, with positions [axes, T]: entry i of a token's
    row of cosines and sines comes from the table row of pair i's axis."""
    T, D = query.shape[0], p.head_size
    pairs = cos_sin.shape[1] // 2
    q = torch.full((T, p.num_heads * D), float("nan"), dtype=F64)
    k = torch.full((T, p.row_elems), float("nan"), dtype=F64)
    v = torch.full((T, p.row_elems), float("nan"), dtype=F64)
    for t in range(T):
        if int(slot_mapping[t]) < 0:
            continue
        row = torch.empty(2 * pairs)
        for i in range(pairs):
            at = int(positions[pair_axes[i], t])
            row[i], row[pairs + i] = cos_sin[at, i], cos_sin[at, pairs + i]
        q[t] = rope_rotate(query[t].to(F64).view(-1, D), row, interleaved).reshape(-1)
        k[t] = rope_rotate(key[t].to(F64).view(-1, D), row, interleaved).reshape(-1)
        v[t] = value[t].to(F64)
        if p.kv_cache_dtype == "fp8_e4m3":
            k[t] /= torch.tensor(p.k_scale, dtype=torch.float32).to(F64)
            v[t] /= torch.tensor(p.v_scale, dtype=torch.float32).to(F64)
    return q, k, v


def tree_ancestors(parents: list, t: int) -> list:
    """Node t and its ancestors, from the top."""
    path = []
    while t >= 0:
        path.append(t)
        t = parents[t]
    return path[::-1]


def paged_attn_decode_tree(query, kv_cache, block_tables, seq_lens, cu_nodes, parents,
                           p: AttnParams, rows=None):
    """(out, spread) [T, H * D] fp64: the outputs, and per element the sum of
    the weights' and values' magnitudes (what a relative error of the weights
    moves it by at most); rows of no tree are NaN.  `rows`: these only."""
    T, D = query.shape[0], p.head_size
    out = torch.full((T, p.num_heads, D), float("nan"), dtype=F64)
    spread = torch.full((T, p.num_heads, D), float("nan"), dtype=F64)
    fp8 = p.kv_cache_dtype == "fp8_e4m3"
    cache = kv_cache.view(2, -1, p.num_kv_heads, D)
    for b in range(seq_lens.numel()):
        first, n = int(cu_nodes[b]), int(cu_nodes[b + 1] - cu_nodes[b])
        if n == 0:
            continue
        up = parents[first:first + n].tolist()
        ctx = int(seq_lens[b]) - n
        slots = []
        for j in range(ctx + n):
            block, at = int(block_tables[b, j // p.block_size]), j % p.block_size
            slots.append(block * p.block_size + at)
        slots = torch.tensor(slots)
        for t in range(n):
            if rows is not None and first + t not in rows:
                continue
            path = tree_ancestors(up, t)
            here = ctx + len(path) - 1
            keys = [(j, j) for j in range(ctx)] + [(ctx + c, ctx + i) for i, c in enumerate(path)]
            if p.sliding_window > 0:
                keys = [(j, pos) for j, pos in keys if pos > here - p.sliding_window]
            at = slots[[j for j, _ in keys]]
            ago = torch.tensor([pos - here for _, pos in keys], dtype=F64)
            for h in range(p.num_heads):
                g = kv_head_of(h, p.queries_per_kv)
                k, v = cache[0, at, g], cache[1, at, g]
                k = _dequant(k, p.k_scale) if fp8 else k.to(F64)
                v = _dequant(v, p.v_scale) if fp8 else v.to(F64)
                s = p.scale * (k @ query[first + t].to(F64).view(-1, D)[h])
                if p.alibi_slopes is not None:
                    s = s + _slope(p, h) * ago
                w = torch.softmax(s, 0)
                # a weight of exactly zero meets no value: only what is seen is summed
                out[first + t, h] = w @ v
                spread[first + t, h] = w @ v.abs()
    return out.view(T, -1), spread.view(T, -1)


def paged_attn_tree_accept(draft, target, parents, cu_nodes, most: int):
    """(accepted [B, most], num_accepted [B], next_token [B]) as lists."""
    accepted, count, token = [], [], []
    for b in range(len(cu_nodes) - 1):
        first, n = int(cu_nodes[b]), int(cu_nodes[b + 1] - cu_nodes[b])
        path = [0] if n else []
        while path and len(path) < most:
            here = path[-1]
            fits = [c for c in range(n) if int(parents[first + c]) == here and
                    int(draft[first + c]) == int(target[first + here])]
            if not fits:
                break
            path.append(fits[0])
        accepted.append(path + [-1] * (most - len(path)))
        count.append(len(path))
        token.append(int(target[first + path[-1]]) if path else -1)
    return accepted, count, token


def kv_commit_tree(kv_caches, accepted, block_tables, seq_lens, cu_nodes, p: AttnParams) -> None:
    """In place, as if every row were read before any is written."""
    for cache in kv_caches:
        rows = cache.view(2, -1, p.row_elems)
        was = rows.clone()
        for b in range(seq_lens.numel()):
            ctx = int(seq_lens[b]) - int(cu_nodes[b + 1] - cu_nodes[b])
            for i, t in enumerate(accepted[b].tolist()):
                if t < 0:
                    break
                to, of = ctx + i, ctx + t
                slot = [int(block_tables[b, x // p.block_size]) * p.block_size + x % p.block_size
                        for x in (to, of)]
                rows[:, slot[0]] = was[:, slot[1]]

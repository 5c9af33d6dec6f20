"""The operators of a speculative step over a tree of drafted tokens, in their plain form and through the library: what is timed and
compared.

A verify step over a paged cache: ``kv_cache_write_rope_axes`` rotates the new queries and keys by positions of several axes (time,
height, width) and stores keys and values in their slots, ``paged_attn_decode_tree`` attends from every drafted token to the context
and to its ancestors, ``paged_attn_tree_accept`` follows the drafted tokens that the model would have taken, ``kv_commit_tree`` moves
their keys and values behind the context in every layer.  A case is one call of one of them.  `own` false: elementary torch
operations; true: the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_SCALE8 = 0.02  # k_scale and v_scale of the 8-bit caches: N(0, 1) keys use most of E4M3's range
_POSITIONS = 131072  # rows of the rotation table


def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "heads": 32, "kv_heads": 8, "head_size": 128, "block_size": 16, "fp8": False}
    if op == "tree":
        c.update(window=0, alibi=False, padding=0)
    c.update(kw)
    return c


def listed():
    return [
        # one sequence's drafted tree over an 8-bit cache, the batch padded to its graph's size; axes woven: latency
        _case("axes_64_fp8", "axes", tokens=64, rot=128, sections="24,20,20", woven=True, interleaved=False, packed=True, padding=3, fp8=True),
        # a scheduler step full of prompt tokens, text and images by turns; half of each head rotated, interleaved pairs
        _case("axes_16384", "axes", tokens=16384, rot=64, sections="8,12,12", woven=False, interleaved=True, packed=False, padding=0),
        # one sequence, a short context, a handful of drafted tokens: latency
        _case("tree_1_short", "tree", seqs=1, len_lo=500, len_hi=500, nodes_lo=6, nodes_hi=6),
        # one long sequence with a wide tree
        _case("tree_1", "tree", seqs=1, len_lo=32768, len_hi=32768, nodes_lo=61, nodes_hi=61),
        # a batch of ordinary trees over ragged contexts, rows for as many of the widest (a captured graph's size) and some more
        _case("tree_64", "tree", seqs=64, len_lo=4096, len_hi=16384, nodes_lo=20, nodes_hi=32, padding=24),
        # wide trees and many query heads per key head: as much arithmetic as reading
        _case("tree_16_wide", "tree", seqs=16, len_lo=16384, len_hi=32768, nodes_lo=64, nodes_hi=64, heads=64),
        # a large batch of small trees over an 8-bit cache, some contexts shorter than a tile
        _case("tree_128_fp8", "tree", seqs=128, len_lo=100, len_hi=4096, nodes_lo=4, nodes_hi=16, fp8=True),
        # one query head per key head, fp16, small heads, larger blocks, a sliding window
        _case("tree_32_mha", "tree", seqs=32, len_lo=4096, len_hi=16384, nodes_lo=48, nodes_hi=64, dtype="fp16", heads=16, kv_heads=16,
              head_size=64, block_size=32, window=4096),
        # the walk down one tree: latency
        _case("accept_1", "accept", seqs=1, nodes_lo=61, nodes_hi=61, most=8),
        # and down those of a large batch
        _case("accept_256", "accept", seqs=256, nodes_lo=1, nodes_hi=64, most=16),
        # one sequence's path in 32 layers
        _case("commit_1", "commit", seqs=1, layers=32, len_lo=2000, len_hi=2000, nodes_lo=61, nodes_hi=61, most=8),
        # those of a batch
        _case("commit_64", "commit", seqs=64, layers=32, len_lo=64, len_hi=300, nodes_lo=20, nodes_hi=32, most=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "tree", "tree", "accept", "commit"])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "heads": group * kv_heads, "kv_heads": kv_heads,
         "head_size": rng.choice([64, 128]), "block_size": rng.choice([16, 32]), "fp8": rng.random() < 0.4}
    if op == "axes":
        c["tokens"] = _log(rng, 1, 12000)
        c["rot"] = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= c["head_size"]])
        cut = sorted(rng.randrange(0, c["rot"] // 2 + 1) for _ in range(2))
        c["sections"] = "%d,%d,%d" % (cut[0], cut[1] - cut[0], c["rot"] // 2 - cut[1])
        c["woven"] = rng.random() < 0.5
        c["interleaved"] = rng.random() < 0.5
        c["packed"] = rng.random() < 0.5
        c["padding"] = rng.randrange(0, 1 + c["tokens"] // 4)
        return c
    c["nodes_hi"] = _log(rng, 1, 64) if rng.random() < 0.8 else _log(rng, 65, 256)
    c["nodes_lo"] = max(1, int(c["nodes_hi"] * rng.uniform(0.2, 1.0)))
    if op == "accept":
        c["seqs"] = _log(rng, 1, 256)
        c["most"] = rng.randrange(1, 20)
        return c
    if op == "commit":
        c["len_hi"] = _log(rng, 1, 300)
        c["len_lo"] = max(0, int(c["len_hi"] * rng.uniform(0.0, 1.0)))
        c["seqs"] = _log(rng, 1, max(1, min(64, 20000 // (c["len_hi"] + c["nodes_hi"]))))
        c["layers"] = rng.randrange(1, 33)
        c["most"] = rng.randrange(1, 12)
        return c
    # up to the listed cases' keys and half of their scores
    c["len_hi"] = _log(rng, 17, 65536)
    c["len_lo"] = int(c["len_hi"] * rng.uniform(0.2, 1.0))
    wide = c["len_hi"] + c["nodes_hi"]
    room = min(64 * 8 * 16384 // (wide * kv_heads), 1000000000 // (wide * c["heads"] * c["nodes_hi"]), 128)
    c["seqs"] = _log(rng, 1, max(1, room))
    c["padding"] = rng.choice([0, 0, 1, 7, 40])
    c["window"] = _log(rng, 1, c["len_hi"]) if rng.random() < 0.25 else 0
    c["alibi"] = rng.random() < 0.2
    return c


# ---- inputs ---------------------------------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _cache(g, c, *lead):
    """[...][block_size * kv_heads * head_size], the form that the library reads."""
    x = _normal(g, *lead, c["block_size"] * c["kv_heads"] * c["head_size"], dtype=_DTYPES[c["dtype"]])
    return x.div_(_SCALE8).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if c["fp8"] else x


def _trees(c, seed):
    """Node counts, where each tree's nodes start, and each node's parent within its tree (-1: the root, node 0)."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(c["nodes_lo"], c["nodes_hi"] + 1, (c["seqs"],), generator=g)
    if c["seqs"] > 2:
        n[1] = c["nodes_hi"]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    t = torch.arange(int(cu[-1])) - torch.repeat_interleave(cu[:-1], n)  # a node's number in its tree
    # any earlier node, the later ones more often: some ten levels of 64 nodes
    parents = torch.minimum((t * torch.rand(t.shape, generator=g) ** 0.7).long(), t - 1)
    return {"nodes": n.cuda(), "cu": cu.to(torch.int32).cuda(), "parents": parents.to(torch.int32).cuda(), "rows": int(cu[-1]),
            "max_nodes": int(n.max())}, g, n, t


def _batch(c, g, gen, nodes):
    """Lengths (context and nodes) and block tables of c["seqs"] sequences whose blocks lie in any order in one pool; the pool's last
    block is nobody's."""
    ctx = torch.randint(c["len_lo"], c["len_hi"] + 1, (c["seqs"],), generator=gen)
    if c["seqs"] > 2:
        ctx[1] = c["len_hi"]
    lens = ctx + nodes
    count = (lens + c["block_size"] - 1) // c["block_size"]
    wide, total = int(count.max()), c["seqs"] * -(-(c["len_hi"] + c["nodes_hi"]) // c["block_size"])  # room for the longest ones
    perm = torch.randperm(total, generator=g, device="cuda")
    start = (torch.cumsum(count, 0) - count).cuda()
    j = torch.arange(wide, device="cuda")
    held = j[None, :] < count.cuda()[:, None]
    tables = torch.where(held, perm[torch.where(held, start[:, None] + j[None, :], 0)], 0)
    return {"seq_lens": lens.to(torch.int32).cuda(), "max_len": int(lens.max()), "tables": tables.to(torch.int32), "blocks": total + 1}


def _axis_of_pair(c):
    """The axis (time, height, width) by which each pair of channels turns: sections behind one another, or height and width woven
    into time's pairs as long as theirs last."""
    t, h, w = (int(x) for x in c["sections"].split(","))
    if not c["woven"]:
        return [0] * t + [1] * h + [2] * w
    return [1 if i % 3 == 1 and i < 3 * h else 2 if i % 3 == 2 and i < 3 * w else 0 for i in range(c["rot"] // 2)]


def _rotation_table(rot):
    """cos | sin of position / 10000^(2 i / rot), made in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    H, KVH, D, BS, dt = c["heads"], c["kv_heads"], c["head_size"], c["block_size"], _DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "axes":
        T = c["tokens"]
        if c["packed"]:  # slices of one projection's output
            qkv = _normal(g, T, (H + 2 * KVH) * D, dtype=dt)
            s["query"], s["key"], s["value"] = qkv.split([H * D, KVH * D, KVH * D], 1)
        else:
            s["query"], s["key"], s["value"] = _normal(g, T, H * D, dtype=dt), _normal(g, T, KVH * D, dtype=dt), _normal(g, T, KVH * D, dtype=dt)
        # stretches of text, where the axes agree, and images of 32 x 32 patches by turns, somewhere in a long conversation
        i = torch.arange(T, device="cuda")
        first = torch.randint(0, _POSITIONS - 2 * T - 64, (1,), generator=g, device="cuda")
        turn = (i // 1024 + torch.randint(0, 2, (1,), generator=g, device="cuda")) % 2 == 1
        at, k = first + i, i % 1024
        s["positions"] = torch.stack([torch.where(turn, at - k, at), torch.where(turn, at - k + k // 32, at),
                                      torch.where(turn, at - k + k % 32, at)])
        s["axis"] = _axis_of_pair(c)
        blocks = (2 * T) // BS + 2
        s["slots"] = torch.randperm((blocks - 1) * BS, generator=g, device="cuda")[:T]
        s["slots"][T - c["padding"]:] = -1
        s["cache"] = _cache(g, c, 2, blocks)
        s["table"] = _rotation_table(c["rot"])
        s["rotated"] = torch.zeros(T, H * D, dtype=dt, device="cuda")
        return s
    tree, gen, n, t = _trees(c, seed)
    s.update(tree)
    if c["op"] == "accept":
        # three of four times the model goes on with a drafted token (the last of those that are tossed for)
        draft = torch.randint(0, 32000, (s["rows"],), generator=gen)
        target = torch.randint(0, 32000, (s["rows"],), generator=gen)
        tossed = ((torch.rand(s["rows"], generator=gen) < 0.75) & (t > 0)).nonzero()[:, 0]
        up = torch.arange(s["rows"]) - t + s["parents"].cpu().long()
        target.numpy()[up[tossed].numpy()] = draft[tossed].numpy()
        s["draft"], s["target"] = draft.cuda(), target.cuda()
        s["accepted"] = torch.full((c["seqs"], c["most"]), -1, dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
        s["token"] = torch.zeros(c["seqs"], dtype=torch.int64, device="cuda")
        return s
    s.update(_batch(c, g, gen, n))
    if c["op"] == "commit":
        s["caches"] = _cache(g, c, c["layers"], 2, s["blocks"])
        s["layers"] = list(s["caches"].unbind(0))
        # a path: the root, then nodes in ascending order, of some length
        r = torch.rand(c["seqs"], s["max_nodes"], generator=gen)
        r[torch.arange(s["max_nodes"]) >= n[:, None]] = -1.0
        r[:, 0] = 2.0
        most = min(c["most"], s["max_nodes"])
        v, i = r.topk(most, dim=1)
        take = (torch.arange(most) < torch.randint(1, most + 1, (c["seqs"], 1), generator=gen)) & (v >= 0)
        i = torch.where(take, i, s["max_nodes"]).sort(dim=1).values
        s["accepted"] = torch.full((c["seqs"], c["most"]), -1, dtype=torch.int32)
        s["accepted"][:, :most] = torch.where(i < s["max_nodes"], i, -1).to(torch.int32)
        s["accepted"] = s["accepted"].cuda()
        return s
    s["cache"] = _cache(g, c, 2, s["blocks"])
    # the nodes' rows, rows for as many nodes as the widest trees would have, and the case's padding
    T = c["seqs"] * c["nodes_hi"] + c["padding"]
    s["query"] = _normal(g, T, H * D, dtype=dt)
    s["room"] = torch.zeros(T + 1, H * D, dtype=dt, device="cuda")
    s["out"] = s["room"][:-1]
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H) if c["alibi"] else None
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------------------


def run(state):
    if own:
        return _run_own(state)
    return {"axes": _axes, "tree": _tree, "accept": _accept, "commit": _commit}[state["case"]["op"]](state)


def _values(t, c):
    """8-bit codes as the type whose values they are."""
    return t.view(torch.float8_e4m3fn) if c["fp8"] else t


def _run_own(s):
    from paged_kv_cache_246_gb300 import binding as B
    c = s["case"]
    if c["op"] == "accept":
        B.paged_attn_tree_accept(s["accepted"], s["count"], s["token"], s["draft"], s["target"], s["parents"], s["cu"], s["max_nodes"])
        return {"accepted": s["accepted"], "count": s["count"], "token": s["token"]}
    if "params" not in s:  # made once, as a program that serves with them keeps them
        s["params"] = B.make_params(c["heads"], c["kv_heads"], c["head_size"], c["block_size"], _DTYPES[c["dtype"]], c["head_size"] ** -0.5,
                                    s.get("slopes"), c.get("window", 0), kv_cache_dtype="fp8_e4m3" if c["fp8"] else "auto",
                                    k_scale=_SCALE8 if c["fp8"] else 1.0, v_scale=_SCALE8 if c["fp8"] else 1.0)
        if c["op"] == "tree":
            size = B.paged_attn_decode_tree_workspace_size(c["seqs"], s["max_nodes"], s["max_len"], s["params"])
            s["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    p = s["params"]
    if c["op"] == "axes":
        B.kv_cache_write_rope_axes(s["rotated"], s["query"], s["key"], s["value"], s["cache"], s["slots"], s["positions"], s["table"],
                                   s["axis"], p, interleaved=c["interleaved"])
        return {"query": s["rotated"], "cache": _values(s["cache"], c)}
    if c["op"] == "tree":
        B.paged_attn_decode_tree(s["out"], s["query"], s["cache"], s["tables"], s["seq_lens"], s["cu"], s["parents"], s["max_nodes"],
                                 s["max_len"], p, s["workspace"])
        return {"out": s["out"]}
    B.kv_commit_tree(s["layers"], s["accepted"], s["tables"], s["seq_lens"], s["cu"], p)
    return {"caches": _values(s["caches"], c)}


def _rotate(x, cos, sin, c):
    """x [T][heads][D] in 32 bits; cos, sin [T][1][rot / 2]."""
    y, r = x.clone(), c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return y


def _axes(s):
    c = s["case"]
    T, KVH, D = c["tokens"], c["kv_heads"], c["head_size"]
    held = (s["slots"] >= 0)[:, None]
    at = s["positions"][torch.tensor(s["axis"], device="cuda")].T  # [T][rot / 2]
    i = torch.arange(c["rot"] // 2, device="cuda")
    cos, sin = s["table"][at, i][:, None, :], s["table"][at, i + c["rot"] // 2][:, None, :]
    q = _rotate(s["query"].float().view(T, -1, D), cos, sin, c).view(T, -1)
    s["rotated"].copy_(torch.where(held, q.to(s["rotated"].dtype), s["rotated"]))
    k = _rotate(s["key"].float().view(T, KVH, D), cos, sin, c).view(T, -1)
    rows = s["cache"].view(2, -1, KVH * D)
    # padding tokens write the pool's last row, which no sequence has, as it was
    at = torch.where(held[:, 0], s["slots"], rows.shape[1] - 1)
    for half, x in ((0, k), (1, s["value"])):
        x = (x.float() / _SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if c["fp8"] else x.to(rows.dtype)
        rows[half].index_copy_(0, at, torch.where(held, x, rows[half, -1]))
    return {"query": s["rotated"], "cache": _values(s["cache"], c)}


def _padded(s):
    """Every tree at the widest one's size: which nodes there are, where they stand among the rows, their parents (-1: none)."""
    t = torch.arange(s["max_nodes"], device="cuda")
    there = t < s["nodes"][:, None]
    at = torch.where(there, s["cu"][:-1].long()[:, None] + t, 0)
    return there, at, torch.where(there, s["parents"].long()[at], -1)


def _ancestors(parents):
    """[trees][nodes][nodes] in 32 bits: 1 where the column's node is the row's or an ancestor of it."""
    n = parents.shape[1]
    step = torch.eye(n, device="cuda") + (parents[:, :, None] == torch.arange(n, device="cuda")).float()

    def twice(a):
        return (a @ a).clamp(max=1.0)

    return twice(twice(twice(twice(twice(twice(twice(twice(step))))))))  # chains of up to 256 steps


def _tree(s):
    c = s["case"]
    B, KVH, D, BS = c["seqs"], c["kv_heads"], c["head_size"], c["block_size"]
    group = c["heads"] // KVH
    there, at, parents = _padded(s)
    N = there.shape[1]
    above = _ancestors(parents)
    depth = above.sum(2).long() - 1
    ctx = s["seq_lens"].long() - s["nodes"]
    j = torch.arange(s["max_len"], device="cuda")
    node = j - ctx[:, None]  # [B][keys]: which node stands there, negative in the context
    place = torch.where(node < 0, j, ctx[:, None] + depth.gather(1, node.clamp(0, N - 1)))
    mine = ctx[:, None] + depth  # [B][N]
    index = node.clamp(0, N - 1)[:, None, :].expand(B, N, -1)
    seen = torch.where(node[:, None, :] < 0, True, above.gather(2, index) > 0) & (j < s["seq_lens"][:, None])[:, None, :]
    if c["window"]:
        seen = seen & (place[:, None, :] > mine[:, :, None] - c["window"])
    block = s["tables"].long().gather(1, (j // BS)[None, :].expand(B, -1).clamp(max=s["tables"].shape[1] - 1))
    rows = s["cache"].view(2, -1, KVH * D)
    scale = _SCALE8 if c["fp8"] else 1.0
    slot = block * BS + j % BS
    k, v = (_values(rows[x][slot], c).float().view(B, -1, KVH, D).transpose(1, 2) * scale for x in (0, 1))
    q = s["query"][at].float().view(B, N, KVH, group, D).permute(0, 2, 1, 3, 4).reshape(B, KVH, N * group, D)
    x = (q @ k.transpose(2, 3)).mul_(D ** -0.5).view(B, KVH, N, group, -1)
    if c["alibi"]:
        x += s["slopes"].view(1, KVH, 1, group, 1) * (place[:, None, :] - mine[:, :, None])[:, None, :, None, :]
    x.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p = (x - x.amax(4, keepdim=True)).exp_()
    total = p.sum(4, keepdim=True)
    out = ((p.view(B, KVH, N * group, -1) @ v).view(B, KVH, N, group, D) / total).permute(0, 2, 1, 3, 4).reshape(B * N, -1)
    # what is no node goes to the row behind the last one
    s["room"].index_copy_(0, torch.where(there, at, s["room"].shape[0] - 1).flatten(), out.to(s["room"].dtype))
    return {"out": s["out"]}


def _accept(s):
    c = s["case"]
    there, at, parents = _padded(s)
    N = there.shape[1]
    draft, target, t = s["draft"][at], s["target"][at], torch.arange(N, device="cuda")
    up = parents.clamp(min=0)
    taken = there & (parents >= 0) & (draft == target.gather(1, up))
    # of several children with the token the first
    first = torch.full_like(up, N).scatter_reduce_(1, up, torch.where(taken, t, N), "amin")
    taken = taken & (first.gather(1, up) == t) | (t == 0)
    above = _ancestors(parents)
    path = there & ((above @ (~taken).float()[:, :, None])[:, :, 0] == 0)
    level = above.sum(2).long() - 1
    path = path & (level < c["most"])
    s["accepted"].copy_(torch.full((c["seqs"], c["most"] + 1), -1, device="cuda")
                        .scatter_(1, torch.where(path, level, c["most"]), t.expand_as(level))[:, :-1])
    s["count"].copy_(path.sum(1))
    s["token"].copy_(target.gather(1, torch.where(path, level, -1).argmax(1, keepdim=True))[:, 0])
    return {"accepted": s["accepted"], "count": s["count"], "token": s["token"]}


def _commit(s):
    c = s["case"]
    BS, acc = c["block_size"], s["accepted"].long()
    ctx = (s["seq_lens"] - s["nodes"]).long()[:, None]
    rows = s["caches"].view(2 * c["layers"], -1, c["kv_heads"] * c["head_size"])

    def slot(pos):
        # what is not accepted moves the pool's last row, which no sequence has, to itself
        block = s["tables"].long().gather(1, (pos // BS).clamp(max=s["tables"].shape[1] - 1))
        return torch.where(acc >= 0, block * BS + pos % BS, rows.shape[1] - 1).flatten()

    src, dst = slot(ctx + acc.clamp(min=0)), slot(ctx + torch.arange(c["most"], device="cuda"))
    rows.index_copy_(1, dst, rows[:, src])
    return {"caches": _values(s["caches"], c)}


# ---- cost -----------------------------------------------------------------------------------------------------------------------


def work(case):
    c = case
    H, KVH, D = c["heads"], c["kv_heads"], c["head_size"]
    e8 = 1 if c["fp8"] else 2  # bytes of a cache element
    if c["op"] == "axes":
        T = c["tokens"] - c["padding"]
        return {"bytes": T * ((2 * H + 2 * KVH) * D * 2 + 2 * KVH * D * e8 + c["rot"] * 4 + 3 * 8 + 8), "flops": T * (H + KVH) * 3 * c["rot"]}
    n, nodes = c["seqs"], (c["nodes_lo"] + c["nodes_hi"]) / 2
    if c["op"] == "accept":
        return {"bytes": n * (nodes * 20 + c["most"] * 4 + 12), "flops": n * nodes}
    if c["op"] == "commit":
        moved = (min(c["most"], nodes) - 1) / 2
        return {"bytes": n * moved * 4 * c["layers"] * KVH * D * e8, "flops": 0}
    keys = (c["len_lo"] + c["len_hi"]) / 2 + nodes
    keys = min(keys, c["window"] + nodes) if c["window"] else keys
    return {"bytes": n * (keys * 2 * KVH * D * e8 + 2 * nodes * H * D * 2), "flops": n * keys * nodes * H * D * 4}


# ---- in 64 bits, from the definitions --------------------------------------------------------------------------------------------


def _walked(parents):
    """Each node's ancestors and itself, as a matrix of truth values, by walking up."""
    n = len(parents)
    rows = torch.zeros(n, n, dtype=torch.bool)
    for t, up in enumerate(parents):
        if up >= 0:
            rows[t] = rows[up]
        rows[t, t] = True
    return rows.cuda()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "accept":
        return None  # whole numbers
    KVH, D, BS = c["kv_heads"], c["head_size"], c["block_size"]
    scale = _SCALE8 if c["fp8"] else 1.0
    if c["op"] == "axes":
        # the rotation as a product of complex numbers
        r, kept = c["rot"], (s["slots"] >= 0).nonzero()[:, 0]
        turns = [torch.complex(s["table"][s["positions"][a], i].double(), s["table"][s["positions"][a], i + r // 2].double())
                 for i, a in enumerate(s["axis"])]
        w = torch.stack(turns, 1)[:, None, :]

        def turned(x):
            x = x.double().reshape(c["tokens"], -1, D)
            pairs = x[..., :r].unflatten(-1, (r // 2, 2) if c["interleaved"] else (2, r // 2))
            pairs = pairs if c["interleaved"] else pairs.transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
            y = y if c["interleaved"] else y.transpose(-1, -2)
            return torch.cat([y.flatten(-2), x[..., r:]], -1).flatten(1)

        query = torch.zeros(s["rotated"].shape, dtype=torch.float64, device="cuda")
        query[kept] = turned(s["query"])[kept]
        cache = _values(s["cache"], c).double().view(2, -1, KVH * D)
        cache[0, s["slots"][kept]] = turned(s["key"])[kept] / scale
        cache[1, s["slots"][kept]] = s["value"].double()[kept] / scale
        return {"query": query, "cache": cache.view(s["cache"].shape)}
    cu, parents, lens = s["cu"].tolist(), s["parents"].tolist(), s["seq_lens"].tolist()
    if c["op"] == "commit":
        out = _values(s["caches"], c).double().view(c["layers"], 2, -1, KVH * D)
        was = _values(s["caches"], c).view(c["layers"], 2, -1, KVH * D)
        tables = s["tables"].tolist()
        for b, path in enumerate(s["accepted"].tolist()):
            ctx = lens[b] - (cu[b + 1] - cu[b])
            for i, t in enumerate(path):
                if t >= 0:
                    to, of = ctx + i, ctx + t
                    out[:, :, tables[b][to // BS] * BS + to % BS] = was[:, :, tables[b][of // BS] * BS + of % BS].double()
        return {"caches": out.view(s["caches"].shape)}
    group = c["heads"] // KVH
    cache = s["cache"].view(2, -1, KVH, D)
    out = torch.zeros(s["out"].shape[0], c["heads"], D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        N = cu[b + 1] - cu[b]
        ctx, rows = n - N, _walked(parents[cu[b]:cu[b + 1]])
        place = torch.cat([torch.arange(ctx, device="cuda"), ctx + rows.sum(1) - 1])
        seen = torch.cat([torch.ones(N, ctx, dtype=torch.bool, device="cuda"), rows], 1)
        ago = place[ctx:, None] - place[None, :]
        if c["window"]:
            seen &= ago < c["window"]
        j = torch.arange(n, device="cuda")
        slot = s["tables"][b].long()[j // BS] * BS + j % BS
        for h in range(KVH):
            k, v = (_values(cache[x, slot, h], c).double() * scale for x in (0, 1))
            for i in range(h * group, (h + 1) * group):
                x = s["query"][cu[b]:cu[b + 1]].double().view(N, -1, D)[:, i] @ k.T / math.sqrt(D)
                if c["alibi"]:
                    x -= float(s["slopes"][i]) * ago
                out[cu[b]:cu[b + 1], i] = torch.softmax(x.masked_fill(~seen, float("-inf")), 1) @ v
    return {"out": out.view(s["out"].shape)}

"""The operators of a block-sparse decode step, in their plain form and through the library: what is timed and compared.

A decode step over a long paged cache: ``kv_cache_write_rope`` rotates the new queries and keys by their positions and stores keys
and values in their slots, ``kv_block_bounds`` keeps each block's channelwise smallest and largest key, ``paged_attn_select_blocks``
picks each sequence's blocks by the bounds, ``paged_attn_decode_sparse`` attends to the picked blocks.  A case is one call of one of
them.  `own` false: elementary torch operations; true: the library's calls.
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
    c.update(kw)
    return c


def listed():
    return [
        # the step of one running sequence: latency
        _case("append_1", "append", tokens=1, rot=128, interleaved=False, packed=True, padding=0),
        # a decode batch under a captured graph: 8-bit cache, the batch padded to its graph's size
        _case("append_256_fp8", "append", tokens=256, rot=128, interleaved=False, packed=True, padding=19, fp8=True),
        # a scheduler step full of prompt tokens; half of each head rotated, interleaved pairs
        _case("append_16384", "append", tokens=16384, rot=64, interleaved=True, packed=False, padding=0),
        # the blocks that a decode step's tokens fell in
        _case("bounds_64_decode", "bounds", seqs=64, len_lo=16384, len_hi=32768, new=1),
        # whole prompts, 8-bit cache
        _case("bounds_16_prompts_fp8", "bounds", seqs=16, len_lo=128, len_hi=8192, new=8192, fp8=True),
        # one long sequence: latency
        _case("select_1", "select", seqs=1, len_lo=32768, len_hi=32768, pick=128, sink=1, recent=2),
        # a batch of long sequences
        _case("select_64", "select", seqs=64, len_lo=16384, len_hi=32768, pick=128, sink=1, recent=2),
        # few very long sequences, 8-bit cache, larger blocks, many queries per key head, small fp16 heads
        _case("select_16_fp8", "select", seqs=16, len_lo=65536, len_hi=131072, pick=256, sink=4, recent=4, fp8=True, dtype="fp16",
              heads=64, head_size=64, block_size=32),
        # one long sequence: latency
        _case("sparse_1", "sparse", seqs=1, len_lo=32768, len_hi=32768, pick=128),
        # a batch of long sequences
        _case("sparse_64", "sparse", seqs=64, len_lo=16384, len_hi=32768, pick=128),
        # a large batch of ordinary lengths over an 8-bit cache, ragged: some sequences shorter than the pick
        _case("sparse_256_fp8", "sparse", seqs=256, len_lo=100, len_hi=4096, pick=96, fp8=True),
        # one query head per key head, fp16, small heads, larger blocks
        _case("sparse_32_mha", "sparse", seqs=32, len_lo=4096, len_hi=16384, pick=64, dtype="fp16", heads=16, kv_heads=16, head_size=64,
              block_size=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "bounds", "select", "sparse"])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "heads": group * kv_heads, "kv_heads": kv_heads,
         "head_size": rng.choice([64, 128]), "block_size": rng.choice([16, 32]), "fp8": rng.random() < 0.4}
    if op == "append":
        c["tokens"] = _log(rng, 1, 12000)
        c["rot"] = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= c["head_size"]])
        c["interleaved"] = rng.random() < 0.5
        c["packed"] = rng.random() < 0.5
        c["padding"] = rng.randrange(0, 1 + c["tokens"] // 4)
        return c
    # sequences times their longest length: up to the listed cases' million tokens
    c["len_hi"] = _log(rng, 17, 100000)
    c["len_lo"] = max(1, int(c["len_hi"] * rng.uniform(0.2, 1.0)))
    c["seqs"] = _log(rng, 1, max(1, min(200, 1000000 // c["len_hi"])))
    if op == "bounds":
        c["new"] = min(rng.choice([1, 1, 5, _log(rng, 1, c["len_hi"])]), 300000 // c["seqs"])
    else:
        c["pick"] = min(_log(rng, 5, 300), 190000 // (c["seqs"] * c["block_size"]))
        if op == "select":
            c["sink"] = rng.randrange(0, 3)
            c["recent"] = rng.randrange(1, 3)
    return c


# ---- inputs ---------------------------------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _cache(g, c, blocks):
    """[2][blocks][block_size * kv_heads * head_size], the form that the library reads."""
    shape = (2, blocks, c["block_size"] * c["kv_heads"] * c["head_size"])
    x = _normal(g, *shape, dtype=_DTYPES[c["dtype"]])
    return x.div_(_SCALE8).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if c["fp8"] else x


def _batch(c, seed, g):
    """Lengths and block tables of c["seqs"] sequences whose blocks lie in any order in one pool with room for the longest ones; the
    pool's last block is nobody's."""
    lens = torch.randint(c["len_lo"], c["len_hi"] + 1, (c["seqs"],), generator=torch.Generator().manual_seed(seed), dtype=torch.int64)
    if c["seqs"] > 2:
        lens[1] = c["len_hi"]
    count = (lens + c["block_size"] - 1) // c["block_size"]
    wide, total = int(count.max()), c["seqs"] * -(-c["len_hi"] // c["block_size"])
    perm = torch.randperm(total, generator=g, device="cuda")
    start = (torch.cumsum(count, 0) - count).cuda()
    j = torch.arange(wide, device="cuda")
    held = j[None, :] < count.cuda()[:, None]
    tables = torch.where(held, perm[torch.where(held, start[:, None] + j[None, :], 0)], 0)
    return {"seq_lens": lens.to(torch.int32).cuda(), "max_len": int(lens.max()), "tables": tables.to(torch.int32), "blocks": total + 1}


def _rotation_table(rot):
    """cos | sin of position / 10000^(2 i / rot), made in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(_POSITIONS, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    H, KVH, D, BS, dt = c["heads"], c["kv_heads"], c["head_size"], c["block_size"], _DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "append":
        T = c["tokens"]
        if c["packed"]:  # slices of one projection's output
            qkv = _normal(g, T, (H + 2 * KVH) * D, dtype=dt)
            s["query"], s["key"], s["value"] = qkv.split([H * D, KVH * D, KVH * D], 1)
        else:
            s["query"], s["key"], s["value"] = _normal(g, T, H * D, dtype=dt), _normal(g, T, KVH * D, dtype=dt), _normal(g, T, KVH * D, dtype=dt)
        s["positions"] = torch.randint(0, _POSITIONS, (T,), generator=g, device="cuda")
        blocks = (2 * T) // BS + 2
        s["slots"] = torch.randperm((blocks - 1) * BS, generator=g, device="cuda")[:T]
        s["slots"][T - c["padding"]:] = -1
        s["cache"] = _cache(g, c, blocks)
        s["table"] = _rotation_table(c["rot"])
        s["rotated"] = torch.zeros(T, H * D, dtype=dt, device="cuda")
        return s
    s.update(_batch(c, seed, g))
    B = c["seqs"]
    if c["op"] == "bounds":
        s["cache"] = _cache(g, c, s["blocks"])
        s["context"] = (s["seq_lens"] - c["new"]).clamp(min=0).to(torch.int32)
        s["bounds"] = torch.zeros(s["blocks"], KVH, 2, D, dtype=torch.uint8 if c["fp8"] else dt, device="cuda")
        return s
    s["query"] = _normal(g, B, H * D, dtype=dt)
    if c["op"] == "select":
        # neighbouring keys are alike, some channels are large throughout
        size = 1.0 + 4.0 * (torch.rand(KVH, D, generator=g, device="cuda") < 0.05)
        mid, half = _normal(g, s["blocks"], KVH, D), 0.3 + torch.rand(s["blocks"], KVH, D, generator=g, device="cuda")
        b = torch.stack([(mid - half) * size, (mid + half) * size], 2)
        s["bounds"] = (b / _SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if c["fp8"] else b.to(dt)
        s["selected"] = torch.full((B, KVH, c["pick"]), -1, dtype=torch.int32, device="cuda")
        return s
    s["cache"] = _cache(g, c, s["blocks"])
    # a choice as the selection makes it: any of the sequence's blocks, the last one among them, in order
    wide = s["tables"].shape[1]
    count = ((s["seq_lens"] + BS - 1) // BS).long()
    j = torch.arange(wide, device="cuda")
    r = torch.rand(B, KVH, wide, generator=g, device="cuda") + 1.0
    r = torch.where(j == count[:, None, None] - 1, 3.0, torch.where(j < count[:, None, None], r, 0.0))
    v, i = r.topk(min(c["pick"], wide), dim=2)
    i = torch.where(v > 0, i, wide).sort(dim=2).values
    picked = torch.full((B, KVH, c["pick"]), -1, dtype=torch.int32, device="cuda")
    picked[:, :, :i.shape[2]] = torch.where(i < wide, i, -1).to(torch.int32)
    s["selected"] = picked
    s["out"] = torch.zeros(B, H * D, dtype=dt, device="cuda")
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------------------


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "bounds": _bounds, "select": _select, "sparse": _sparse}[state["case"]["op"]](state)


def _values(t, c):
    """8-bit codes as the type whose values they are."""
    return t.view(torch.float8_e4m3fn) if c["fp8"] else t


def _run_own(s):
    from paged_kv_cache_246_gb300 import binding as B
    c = s["case"]
    if "params" not in s:  # made once, as a program that serves with them keeps them
        s["params"] = B.make_params(c["heads"], c["kv_heads"], c["head_size"], c["block_size"], _DTYPES[c["dtype"]], c["head_size"] ** -0.5,
                                    kv_cache_dtype="fp8_e4m3" if c["fp8"] else "auto", k_scale=_SCALE8 if c["fp8"] else 1.0,
                                    v_scale=_SCALE8 if c["fp8"] else 1.0)
    p = s["params"]
    if c["op"] == "append":
        B.kv_cache_write_rope(s["rotated"], s["query"], s["key"], s["value"], s["cache"], s["slots"], s["positions"], s["table"], p,
                              interleaved=c["interleaved"])
        return {"query": s["rotated"], "cache": _values(s["cache"], c)}
    if c["op"] == "bounds":
        B.kv_block_bounds(s["bounds"], s["cache"], s["tables"], s["seq_lens"], c["new"], p, context_lens=s["context"])
        return {"bounds": _values(s["bounds"], c)}
    if c["op"] == "select":
        B.paged_attn_select_blocks(s["selected"], s["query"], s["bounds"], s["tables"], s["seq_lens"], s["max_len"], p,
                                   num_sink=c["sink"], num_recent=c["recent"])
        return {"selected": s["selected"]}
    B.paged_attn_decode_sparse(s["out"], s["query"], s["cache"], s["tables"], s["seq_lens"], s["selected"], p)
    return {"out": s["out"]}


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


def _append(s):
    c = s["case"]
    T, KVH, D = c["tokens"], c["kv_heads"], c["head_size"]
    held = (s["slots"] >= 0)[:, None]
    cos, sin = s["table"][s["positions"]][:, None, :].chunk(2, 2)
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


def _bounds(s):
    c = s["case"]
    KVH, D, BS = c["kv_heads"], c["head_size"], c["block_size"]
    # the blocks from the first new position's to the last one's, as many columns as the widest sequence has
    first, L = (s["context"] // BS).long(), s["seq_lens"].long()
    last = (L - 1) // BS
    j = first[:, None] + torch.arange((min(c["new"], s["max_len"]) + BS - 2) // BS + 1, device="cuda")
    there = (j <= last[:, None]) & (s["context"] < s["seq_lens"])[:, None]
    at = torch.where(there, s["tables"].long().gather(1, j.clamp(max=s["tables"].shape[1] - 1)), s["blocks"] - 1).flatten()
    k = _values(s["cache"], c)[0].view(-1, BS * KVH * D)
    k = k.view(torch.uint8)[at].view(k.dtype) if c["fp8"] else k[at]
    k = k.float().view(-1, BS, KVH, D)
    written = ((j * BS)[:, :, None] + torch.arange(BS, device="cuda") < L[:, None, None]).flatten(0, 1)[:, :, None, None]
    lo = k.masked_fill(~written, float("inf")).amin(1)
    hi = k.masked_fill(~written, float("-inf")).amax(1)
    new = torch.stack([lo, hi], 2)
    new = new.to(torch.float8_e4m3fn).view(torch.uint8) if c["fp8"] else new.to(s["bounds"].dtype)
    s["bounds"].index_copy_(0, at, torch.where(there.flatten()[:, None, None, None], new, s["bounds"][-1]))
    return {"bounds": _values(s["bounds"], c)}


def _select(s):
    c = s["case"]
    B, KVH, D, BS, K = c["seqs"], c["kv_heads"], c["head_size"], c["block_size"], c["pick"]
    # in 64 bits: which of two blocks at the border scores higher shows in the last places
    b = s["bounds"][s["tables"].long()] if not c["fp8"] else s["bounds"][s["tables"].long()].view(torch.float8_e4m3fn).float()
    q = s["query"].double().view(B, KVH, -1, D)
    lo, hi = (b[:, :, :, x].permute(0, 2, 3, 1).double() for x in (0, 1))  # [B][KVH][D][blocks]
    score = (q.clamp(min=0) @ hi + q.clamp(max=0) @ lo).amax(2)  # [B][KVH][blocks]
    wide = score.shape[2]
    j = torch.arange(wide, device="cuda")
    count = ((s["seq_lens"].long() + BS - 1) // BS)[:, None, None]
    always = (j < c["sink"]) | (j >= count - c["recent"])
    score = torch.where(j < count, torch.where(always, float("inf"), score), float("-inf"))
    best, at = score.sort(dim=2, descending=True, stable=True)
    at = torch.where(best[:, :, :K] > float("-inf"), at[:, :, :K], wide).sort(dim=2).values
    s["selected"].fill_(-1)
    s["selected"][:, :, :at.shape[2]] = torch.where(at < wide, at, -1).to(torch.int32)
    return {"selected": s["selected"]}


def _sparse(s):
    c = s["case"]
    B, KVH, D, BS, K = c["seqs"], c["kv_heads"], c["head_size"], c["block_size"], c["pick"]
    sel = s["selected"].long()
    block = s["tables"].long().gather(1, sel.clamp(min=0).view(B, -1)).view(B, KVH, K)
    pos = (sel * BS)[..., None] + torch.arange(BS, device="cuda")
    seen = ((sel >= 0)[..., None] & (pos < s["seq_lens"].long()[:, None, None, None])).view(B, KVH, 1, K * BS)
    cache = s["cache"].view(2, -1, BS, KVH, D)
    h = torch.arange(KVH, device="cuda")[None, :, None]
    scale = _SCALE8 if c["fp8"] else 1.0
    k, v = (_values(cache[x][block, :, h], c).float().view(B, KVH, K * BS, D) * scale for x in (0, 1))
    q = s["query"].float().view(B, KVH, -1, D)
    x = (q @ k.transpose(2, 3) * D ** -0.5).masked_fill(~seen, float("-inf"))
    p = (x - x.amax(3, keepdim=True)).exp()
    s["out"].copy_(((p @ v) / p.sum(3, keepdim=True)).view(B, -1))
    return {"out": s["out"]}


# ---- cost -----------------------------------------------------------------------------------------------------------------------


def _mean_len(c):
    return (c["len_lo"] + c["len_hi"]) / 2


def work(case):
    c = case
    H, KVH, D, BS = c["heads"], c["kv_heads"], c["head_size"], c["block_size"]
    e8 = 1 if c["fp8"] else 2  # bytes of a cache element
    if c["op"] == "append":
        T = c["tokens"] - c["padding"]
        return {"bytes": T * ((2 * H + 2 * KVH) * D * 2 + 2 * KVH * D * e8 + c["rot"] * 4 + 16), "flops": T * (H + KVH) * 3 * c["rot"]}
    n = c["seqs"]
    if c["op"] == "bounds":
        rows = min(c["new"], _mean_len(c))
        # a decode step's block is half written on average
        rows = rows if rows > BS else rows + (BS - 1) / 2
        return {"bytes": n * KVH * D * e8 * (rows + 2 * max(1, rows / BS)), "flops": n * 2 * rows * KVH * D}
    if c["op"] == "select":
        blocks = _mean_len(c) / BS
        return {"bytes": n * (blocks * (2 * KVH * D * e8 + 4) + H * D * 2 + KVH * c["pick"] * 4), "flops": n * blocks * H * D * 4}
    keys = min(c["pick"] * BS, _mean_len(c))
    return {"bytes": n * (keys * 2 * KVH * D * e8 + 2 * H * D * 2 + KVH * c["pick"] * 4), "flops": n * keys * H * D * 4}


# ---- in 64 bits, from the definitions --------------------------------------------------------------------------------------------


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "select":
        return None  # whole numbers
    KVH, D, BS = c["kv_heads"], c["head_size"], c["block_size"]
    scale = _SCALE8 if c["fp8"] else 1.0
    if c["op"] == "append":
        # the rotation as a product of complex numbers
        w = torch.complex(*s["table"][s["positions"]].double().chunk(2, 1))[:, None, :]
        r, kept = c["rot"], (s["slots"] >= 0).nonzero()[:, 0]

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
    if c["op"] == "bounds":
        k = _values(s["cache"], c)[0].double().view(s["blocks"], BS, KVH, D)
        out = _values(s["bounds"], c).double()
        for b, (n, ctx) in enumerate(zip(s["seq_lens"].tolist(), s["context"].tolist())):
            if ctx >= n:
                continue
            first, last = ctx // BS, (n - 1) // BS
            at = s["tables"][b, first:last + 1].long()
            whole, tail = k[at[:-1]], k[at[-1], :n - last * BS]
            out[at[:-1], :, 0], out[at[:-1], :, 1] = whole.sort(dim=1).values[:, 0], whole.sort(dim=1).values[:, -1]
            out[at[-1], :, 0], out[at[-1], :, 1] = tail.sort(dim=0).values[0], tail.sort(dim=0).values[-1]
        return {"bounds": out}
    cache = s["cache"].view(2, -1, BS, KVH, D)
    out = torch.zeros(c["seqs"], c["heads"], D, dtype=torch.float64, device="cuda")
    group = c["heads"] // KVH
    for b, n in enumerate(s["seq_lens"].tolist()):
        for h in range(KVH):
            sel = s["selected"][b, h]
            sel = sel[sel >= 0].long()
            seen = ((sel * BS)[:, None] + torch.arange(BS, device="cuda") < n).flatten()
            k, v = (_values(cache[x, s["tables"][b, sel].long(), :, h], c).double().reshape(-1, D)[seen] * scale for x in (0, 1))
            q = s["query"][b].double().view(-1, D)[h * group:(h + 1) * group]
            out[b, h * group:(h + 1) * group] = torch.softmax(q @ k.T / math.sqrt(D), 1) @ v
    return {"out": out.view(c["seqs"], -1)}

"""GPU times of the block-sparse decode's and the speculative step's calls, without the host's: captured in a CUDA graph over three
sets of inputs and replayed (median of 7 replays of 30 calls).

    python perf/gpu_times.py [cases] [more] [data] [step] [tree] [tree_more]

cases: those of operators.py; more: forms of them that it does not list; data: the selection over scores of other kinds; step: the
four calls of a decode step against the dense cache write and decode; tree: the cases of more_operators.py; tree_more: forms of
them that it does not list, and the run of tokens that paged_attn_decode_multi takes.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import perf.more_operators as tree_ops  # noqa: E402
import perf.operators as ops  # noqa: E402
from paged_kv_cache_246_gb300 import binding as B  # noqa: E402

ops.own = tree_ops.own = True
LISTED = {c["name"]: c for c in ops.listed()}
TREES = {c["name"]: c for c in tree_ops.listed()}


def gpu_us(calls, reps=30):
    for f in calls:
        f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(reps):
            calls[i % len(calls)]()
    graph.replay()
    times = []
    for _ in range(7):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / reps)
    return sorted(times)[3]


def time_case(label, case, change=None, ops=ops):
    states = [ops.prepare(case, seed) for seed in range(3)]
    for s in states:
        if change:
            change(s)
    us = gpu_us([lambda s=s: ops.run(s) for s in states])
    print(f"{label:64s} {us:8.2f} us  {ops.work(case)['bytes'] / us / 1e6:5.2f} TB/s", flush=True)
    del states
    torch.cuda.empty_cache()


def cases():
    for name, case in LISTED.items():
        time_case(name, case)


def more():
    for name, kw in (("append_16384", dict(fp8=True)), ("append_16384", dict(rot=128, interleaved=False, packed=True)),
                     ("bounds_16_prompts_fp8", dict(fp8=False)),
                     ("sparse_64", dict(heads=64)), ("sparse_64", dict(heads=128)), ("sparse_64", dict(heads=256)),
                     ("sparse_256_fp8", dict(dtype="fp16")), ("sparse_256_fp8", dict(heads=64)),
                     ("sparse_256_fp8", dict(heads=64, dtype="fp16")), ("sparse_256_fp8", dict(heads=128)),
                     ("sparse_256_fp8", dict(heads=256))):
        time_case(f"{name} with {kw}", {**LISTED[name], **kw})
    # a captured step's bound on the lengths, far above them
    short = {**LISTED["select_64"], "len_lo": 2048, "len_hi": 4096}
    time_case("select_64 of 2048 .. 4096 tokens", short)
    time_case("the same, max_seq_len 524288", short, lambda s: s.update(max_len=524288))


def data():
    """How the selection's time depends on the scores: the border's bin of its histogram holds more blocks than it ranks at once
    where a few scores lie far from the rest, or where many are alike."""
    def first_block_outlies(s):
        s["bounds"][s["tables"][:, 0].long()] *= 64.0

    def alike(s):
        s["bounds"].copy_(s["bounds"][:1].clone().expand_as(s["bounds"]))
        s["bounds"][:, :, :, 0] += torch.randn(s["blocks"], s["bounds"].shape[1], 2, device="cuda").to(s["bounds"].dtype) * 0.01

    def equal(s):
        s["bounds"].copy_(s["bounds"][:1].clone().expand_as(s["bounds"]))

    for name in ("select_1", "select_64"):
        for label, change, sink in (("as listed", None, 1), ("no block outlies, num_sink 0", None, 0),
                                    ("the first block outlies, num_sink 0", first_block_outlies, 0),
                                    ("the first block outlies, num_sink 1", first_block_outlies, 1),
                                    ("alike in all but a channel", alike, 1), ("equal", equal, 1)):
            time_case(f"{name}, {label}", {**LISTED[name], "sink": sink}, change)


def step():
    for n, lo, hi, fp8 in ((1, 32768, 32768, False), (8, 32768, 32768, False), (64, 16384, 32768, False), (64, 16384, 32768, True)):
        s = ops.prepare({**LISTED["sparse_64"], "seqs": n, "len_lo": lo, "len_hi": hi, "fp8": fp8}, 1)
        kw = dict(kv_cache_dtype="fp8_e4m3", k_scale=0.02, v_scale=0.02) if fp8 else {}
        p = B.make_params(32, 8, 128, 16, torch.bfloat16, 128 ** -0.5, **kw)
        cache, tables, lens, top = s["cache"], s["tables"], s["seq_lens"], s["max_len"]
        bounds = torch.zeros(s["blocks"], 8, 2, 128, dtype=cache.dtype, device="cuda")
        B.kv_block_bounds(bounds, cache, tables, lens, top, p)
        q, k, v = torch.randn(n, 48 * 128, device="cuda").bfloat16().split([4096, 1024, 1024], 1)
        kc, vc = k.contiguous(), v.contiguous()
        rot, out = (torch.zeros(n, 4096, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pos, ctx, table = (lens - 1).long(), lens - 1, B.rope_table(32768, 128)
        slots = tables.long().gather(1, pos[:, None] // 16)[:, 0] * 16 + pos % 16
        sel = torch.zeros(n, 8, 128, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(16, B.paged_attn_decode_workspace_size(n, top, p)), dtype=torch.uint8, device="cuda")

        def sparse():
            B.kv_cache_write_rope(rot, q, k, v, cache, slots, pos, table, p)
            B.kv_block_bounds(bounds, cache, tables, lens, 1, p, context_lens=ctx)
            B.paged_attn_select_blocks(sel, rot, bounds, tables, lens, top, p, num_sink=1, num_recent=2)
            B.paged_attn_decode_sparse(out, rot, cache, tables, lens, sel, p)

        def dense():
            B.kv_cache_write(kc, vc, cache, slots, p)
            B.paged_attn_decode(out, rot, cache, tables, lens, top, p, ws)

        print(f"{n} sequences of {lo} .. {hi} tokens, {'8' if fp8 else '16'}-bit cache: sparse step {gpu_us([sparse]):.1f} us, "
              f"dense write and decode {gpu_us([dense]):.1f} us", flush=True)
        del s, cache, bounds
        torch.cuda.empty_cache()


def tree():
    for name, case in TREES.items():
        time_case(name, case, ops=tree_ops)


def tree_more():
    for name, kw in (("axes_16384", dict(woven=True)), ("axes_16384", dict(fp8=True)),
                     ("axes_16384", dict(rot=128, sections="16,24,24", interleaved=False, packed=True)),
                     ("tree_1_short", dict(len_lo=250, len_hi=250)), ("tree_1_short", dict(len_lo=4000, len_hi=4000)),
                     ("tree_64", dict(nodes_lo=1, nodes_hi=1)), ("tree_64", dict(nodes_lo=2, nodes_hi=40)),
                     ("tree_64", dict(nodes_lo=64, nodes_hi=64)), ("tree_64", dict(alibi=True)), ("tree_64", dict(fp8=True)),
                     ("tree_64", dict(len_lo=100, len_hi=600)), ("tree_128_fp8", dict(fp8=False)),
                     ("tree_128_fp8", dict(dtype="fp16")), ("tree_32_mha", dict(window=0)),
                     ("tree_32_mha", dict(nodes_lo=200, nodes_hi=256))):
        time_case(f"{name} with {kw}", {**TREES[name], **kw}, ops=tree_ops)
    # a captured step's bound on the nodes, far above them
    time_case("tree_64, max_nodes 256", TREES["tree_64"], lambda s: s.update(max_nodes=256), tree_ops)
    # a run of tokens through both calls
    for tokens in (4, 8, 16, 32):
        s = tree_ops.prepare({**TREES["tree_64"], "nodes_lo": tokens, "nodes_hi": tokens, "padding": 0}, 1)
        p = B.make_params(32, 8, 128, 16, torch.bfloat16, 128 ** -0.5)
        n, top = s["seq_lens"].numel(), s["max_len"]
        s["parents"].copy_((torch.arange(n * tokens, device="cuda") % tokens - 1).int())
        ws, multi = (torch.empty(max(16, size), dtype=torch.uint8, device="cuda") for size in (
            B.paged_attn_decode_tree_workspace_size(n, tokens, top, p),
            B.paged_attn_decode_multi_workspace_size(n, tokens, top, p)))
        t = gpu_us([lambda: B.paged_attn_decode_tree(s["out"], s["query"], s["cache"], s["tables"], s["seq_lens"], s["cu"],
                                                     s["parents"], tokens, top, p, ws)])
        m = gpu_us([lambda: B.paged_attn_decode_multi(s["out"], s["query"], s["cache"], s["tables"], s["seq_lens"], tokens, top, p,
                                                      multi)])
        print(f"64 runs of {tokens} tokens behind 4096 .. 16384: tree {t:.1f} us, multi {m:.1f} us", flush=True)
        del s
        torch.cuda.empty_cache()


if __name__ == "__main__":
    for what in sys.argv[1:] or ["cases", "more", "data", "step", "tree", "tree_more"]:
        {"cases": cases, "more": more, "data": data, "step": step, "tree": tree, "tree_more": tree_more}[what]()

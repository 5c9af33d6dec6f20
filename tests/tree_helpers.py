"""Scenes for the tests of speculative decoding over trees: trees, caches and
tables on the CPU, with their params on both sides."""
from __future__ import annotations

import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8, codes

BF, FP = torch.bfloat16, torch.float16


def random_tree(n, g, shape="bushy"):
    """Parents of n nodes: "chain", "star" (all under node 0), "forest" (several
    without a parent), "bushy"."""
    if shape == "chain":
        return [t - 1 for t in range(n)]
    if shape == "star":
        return [-1] + [0] * (n - 1)
    low = -1 if shape == "forest" else 0
    return [-1] + [int(torch.randint(low, t, (1,), generator=g)) for t in range(1, n)]


class TreeScene:
    """Sequences of `ctx` cached tokens and `nodes` nodes each."""

    def __init__(self, ctx, nodes, heads=8, kv_heads=2, D=128, BS=16, dtype=BF, fp8=False, window=0,
                 alibi=False, shape="bushy", seed=0, padding=0, extra_blocks=2, table_slack=0):
        self.gen = g = torch.Generator().manual_seed(seed)
        self.H, self.KVH, self.D, self.BS, self.dtype, self.fp8 = heads, kv_heads, D, BS, dtype, fp8
        self.row, self.ctx, self.nodes, self.window = kv_heads * D, list(ctx), list(nodes), window
        self.lens = torch.tensor([c + n for c, n in zip(ctx, nodes)], dtype=torch.int32)
        self.cu = torch.tensor([0] + list(nodes)).cumsum(0).int()
        self.trees = [random_tree(n, g, shape) if n else [] for n in nodes]
        self.parents = torch.tensor([p for t in self.trees for p in t], dtype=torch.int32)
        self.rows = int(self.cu[-1])
        n = len(self.nodes)
        self.wide = max(1, max((int(L) + BS - 1) // BS for L in self.lens)) + table_slack
        self.blocks = n * self.wide + extra_blocks
        self.tables = torch.randperm(self.blocks, generator=g)[:n * self.wide].view(n, -1).int()
        x = torch.randn(2, self.blocks, BS * self.row, generator=g)
        self.cache = codes(x) if fp8 else x.to(dtype)
        self.query = torch.randn(self.rows + padding, heads * D, generator=g).to(dtype)
        self.slopes = [2.0 ** -(1 + h % 7) for h in range(heads)] if alibi else None
        self.k = dict(kv_cache_dtype="fp8_e4m3" if fp8 else "auto", k_scale=SCALE8 if fp8 else 1.0,
                      v_scale=SCALE8 if fp8 else 1.0)
        self.op = O.AttnParams(heads, kv_heads, D, BS, D ** -0.5, self.slopes, window, True, **self.k)

    def params(self, dev="cuda:0"):
        self.dev_slopes = None if self.slopes is None else torch.tensor(self.slopes, device=dev)
        return B.make_params(self.H, self.KVH, self.D, self.BS, self.dtype, self.D ** -0.5,
                             self.dev_slopes, self.window, **self.k)

    def slot(self, b, pos):
        return int(self.tables[b, pos // self.BS]) * self.BS + pos % self.BS

    def depths(self, b):
        return [len(O.tree_ancestors(self.trees[b], t)) - 1 for t in range(self.nodes[b])]

    def decode(self, dev="cuda:0", out=None, workspace=None, max_nodes=None, max_len=None, stream=None,
               query=None, cache=None, params=None):
        """The library's output on the device (rows of no tree hold 7)."""
        p = self.params(dev) if params is None else params
        query = (self.query if query is None else query).to(dev)
        cache = (self.cache if cache is None else cache).to(dev)
        out = torch.full_like(query, 7.0) if out is None else out
        max_nodes = max(1, max(self.nodes)) if max_nodes is None else max_nodes
        max_len = int(self.lens.max()) if max_len is None else max_len
        if workspace is None:
            size = B.paged_attn_decode_tree_workspace_size(len(self.nodes), max_nodes, max_len, p)
            # what a workspace holds does not matter
            workspace = torch.full((max(16, size),), 0xFF, dtype=torch.uint8, device=dev)
        B.paged_attn_decode_tree(out, query, cache, self.tables.to(dev), self.lens.to(dev),
                                 self.cu.to(dev), self.parents.to(dev), max_nodes, max_len, p, workspace,
                                 stream=stream)
        return out

    def expect(self, rows=None, query=None, cache=None):
        return O.paged_attn_decode_tree(self.query if query is None else query,
                                        self.cache if cache is None else cache, self.tables, self.lens,
                                        self.cu, self.parents, self.op, rows)


def tolerance(s: TreeScene, out, spread, query=None):
    """How far a decode may be from (out, spread), elementwise.  The output is
    rounded once: half a step of its type.  Each softmax weight enters the
    product with V rounded to 16 bits, half a step of that type (fp16 over an
    8-bit cache), which moves the output by as much of spread.  A score off by d
    moves its weight by 2 d of itself at most (its own and the sum's); d is that
    of fp32 sums of D products of at most max|q| max|k| (over an 8-bit cache also
    the queries' 8-bit terms: a row is scaled to a largest component of 2^7 or
    more, its terms of 4 bits hold a component's 8 or 11 but for what lies below
    half of E4M3's smallest step 2^-9, 2^-17 of the largest), ALiBi's slope times
    distance in fp32, and 2^x of the special-function unit (2^-22)."""
    half = torch.finfo(s.dtype).eps / 2
    weights = torch.finfo(FP).eps / 2 if s.fp8 else half
    q = (s.query if query is None else query).double().nan_to_num(0.0, 0.0, 0.0).abs().max().item()
    k = 448 * SCALE8 if s.fp8 else s.cache[0].double().nan_to_num(0.0, 0.0, 0.0).abs().max().item()
    per = s.D * 2.0 ** -24 + (2.0 ** -17 if s.fp8 else 0.0)
    d = s.D ** -0.5 * s.D * q * k * per
    far = float(s.lens.max()) if s.slopes is not None else 0.0
    d += (2 * far + 64.0) * 2.0 ** -22
    tiny = 2.0 ** -25 if s.dtype == FP else 1e-30   # fp16 below its normal range
    return (half * 1.01) * out.abs() + (weights + 2 * d) * 1.01 * spread + 1e-7 + tiny

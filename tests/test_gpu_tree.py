"""paged_attn_decode_tree against the fp64 oracle: sizes, masks and values
where it can go wrong, bad indices, streams and graphs."""
import dataclasses
import os
import subprocess
import sys

import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8, codes
from tree_helpers import BF, FP, TreeScene, tolerance

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def error():
    torch.cuda.synchronize()
    return B.device_error()


def clean(where):
    st, d = error()
    assert st == B.PKV_OK, f"{where}: {B.status_string(st)} at {d}"


def within(got, want, tol, what):
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    ok = torch.isfinite(want)
    off = ((got - want).abs() - tol)[ok]
    assert not (off > 0).any(), f"{what}: {int((off > 0).sum())} off, worst by {float(off.max())}"


def check(s: TreeScene, what="tree", got=None, rows=None, **kw):
    got = s.decode(**kw) if got is None else got
    clean(what)
    got = got.cpu()
    assert (got[s.rows:] == 7.0).all(), "rows behind the last tree"
    want, spread = s.expect(rows)
    at = list(range(s.rows)) if rows is None else sorted(rows)
    within(got[at].double(), want[at], tolerance(s, want, spread)[at], what)
    return got


KINDS = [(BF, 128, 16, 8, 2, False), (FP, 64, 32, 3, 3, False), (BF, 64, 16, 5, 1, True),
         (FP, 128, 32, 12, 2, True), (FP, 128, 16, 6, 2, False)]


@pytest.mark.parametrize("dtype,D,BS,heads,kv_heads,fp8", KINDS)
def test_small_trees(dtype, D, BS, heads, kv_heads, fp8):
    s = TreeScene([0, 1, 30, 127, 128, 129], [1, 3, 7, 2, 1, 12], heads, kv_heads, D, BS, dtype, fp8,
                  padding=3, seed=D + BS)
    check(s)


@pytest.mark.parametrize("dtype,D,BS,heads,kv_heads,fp8", KINDS)
@pytest.mark.parametrize("window,alibi", [(1, False), (9, True), (150, False), (0, True)])
def test_windows_and_alibi(dtype, D, BS, heads, kv_heads, fp8, window, alibi):
    s = TreeScene([0, 5, 200, 300], [9, 4, 20, 33], heads, kv_heads, D, BS, dtype, fp8, window, alibi,
                  seed=window)
    check(s)


@pytest.mark.parametrize("shape", ["chain", "star", "forest", "bushy"])
@pytest.mark.parametrize("n", [64, 130, 256])
def test_wide_trees(shape, n):
    # trees that span several key tiles and several groups of rows
    s = TreeScene([70, 1], [n, n - 1], 4, 2, 64, 16, FP, shape=shape, seed=n, window=0 if n == 64 else 100)
    check(s)
    s = TreeScene([33], [n], 4, 1, 64, 16, BF, fp8=True, shape=shape, seed=n)
    check(s)


@pytest.mark.parametrize("heads,kv_heads,n", [(1, 1, 40), (2, 2, 129), (7, 1, 64), (16, 1, 17), (33, 1, 9),
                                              (100, 1, 3), (128, 1, 5), (24, 3, 100)])
def test_groups_of_heads(heads, kv_heads, n):
    check(TreeScene([100], [n], heads, kv_heads, 64, 16, FP, seed=heads))
    check(TreeScene([40], [n], heads, kv_heads, 128, 16, BF, fp8=True, seed=heads))


@pytest.mark.parametrize("fp8", [False, True])
def test_long_contexts(fp8):
    # split over many CTAs, ragged; a sample of the rows against the oracle
    s = TreeScene([5000, 17, 9000, 0, 3001], [20, 1, 33, 5, 64], 8, 2, 128, 16, BF, fp8, seed=4)
    check(s, rows={0, 19, 20, 21, 53, 54, 59, 122})
    s = TreeScene([12000], [64], 8, 2, 64, 32, FP, fp8, seed=5)
    check(s, rows={0, 1, 33, 63})


def test_one_long_sequence_in_many_parts():
    s = TreeScene([20000], [40], 4, 1, 128, 16, BF, seed=6)
    check(s, rows={0, 39})


def test_a_chain_is_the_multi_token_decode():
    s = TreeScene([300, 64, 7], [5, 5, 5], 8, 2, shape="chain", window=120, alibi=True)
    got = check(s).double()
    p, q = s.params(), s.query.to(DEV)
    out = torch.empty_like(q)
    size = B.paged_attn_decode_multi_workspace_size(3, 5, 400, p)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    B.paged_attn_decode_multi(out, q, s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV), 5, 400, p, ws)
    want, spread = s.expect()
    assert ((out.cpu().double() - got).abs() <= 2 * tolerance(s, want, spread)).all()


def test_no_nodes_and_empty_calls():
    s = TreeScene([50, 40, 0, 9], [3, 0, 0, 2], 4, 2, 64)
    check(s, max_nodes=5)
    s = TreeScene([50, 40], [0, 0], 4, 2, 64, padding=4)
    s.parents = torch.zeros(4, dtype=torch.int32)
    check(s)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    q = torch.zeros(0, 4 * 64, dtype=BF, device=DEV)
    B.paged_attn_decode_tree(q, q, s.cache.to(DEV), torch.zeros(0, 1, dtype=torch.int32, device=DEV), e,
                             torch.zeros(1, dtype=torch.int32, device=DEV), e, 4, 16, s.params())
    clean("empty")


@pytest.mark.parametrize("fp8", [False, True])
def test_bounds_far_above_the_sizes(fp8):
    s = TreeScene([600, 20], [7, 3], 8, 2, fp8=fp8, table_slack=40)
    a = check(s)
    b = check(s, max_nodes=B.PKV_TREE_MAX_NODES, max_len=100000)
    assert torch.isfinite(b[:s.rows]).all() and a.shape == b.shape


@pytest.mark.parametrize("seqs", [1, 3, 40, 400])
def test_batches(seqs):
    g = torch.Generator().manual_seed(seqs)
    ctx = torch.randint(0, 200, (seqs,), generator=g).tolist()
    nodes = torch.randint(0, 4, (seqs,), generator=g).tolist()
    nodes[0] = 3
    check(TreeScene(ctx, nodes, 4, 2, 64, 16, BF, seed=seqs, padding=1))


def test_many_sequences():
    g = torch.Generator().manual_seed(1)
    nodes = torch.randint(0, 3, (3000,), generator=g).tolist()
    ctx = torch.randint(0, 5, (3000,), generator=g).tolist()
    nodes[17], ctx[17] = 2, 250
    s = TreeScene(ctx, nodes, 1, 1, 64, 16, FP, seed=2)
    rows = set(range(0, s.rows, 37)) | {int(s.cu[17]), int(s.cu[17]) + 1}
    check(s, rows=rows)


@pytest.mark.parametrize("fp8", [False, True])
def test_mixed_trees(fp8):
    # some trees of several row tiles among small and empty ones: the row tiles' lists differ
    s = TreeScene([600, 40, 0, 333, 129, 70, 2], [3, 200, 1, 33, 0, 90, 64], 8, 2, 64, 16, BF, fp8, seed=31, padding=2)
    check(s, rows={0, 2, 3, 4, 130, 202, 203, 204, 236, 237, 290, 326, 327, 390})
    check(s, max_nodes=B.PKV_TREE_MAX_NODES, max_len=20000, rows={0, 202, 203, 236, 326, 390})


@pytest.mark.parametrize("seed", range(24))
def test_drawn_scenes(seed):
    g = torch.Generator().manual_seed(1000 + seed)
    pick = lambda *v: v[int(torch.randint(len(v), (1,), generator=g))]
    n = int(torch.randint(1, 7, (1,), generator=g))
    top = pick(1, 5, 20, 70)
    ctx = torch.randint(0, pick(3, 130, 700), (n,), generator=g).tolist()
    nodes = torch.randint(0, top + 1, (n,), generator=g).tolist()
    nodes[-1] = max(1, nodes[-1])
    kv = pick(1, 2, 3)
    s = TreeScene(ctx, nodes, kv * pick(1, 2, 4, 5, 8), kv, pick(64, 128), pick(16, 32), pick(BF, FP), pick(False, True),
                  pick(0, 0, 1, 30, 200), pick(False, False, True), pick("bushy", "chain", "star", "forest"), seed,
                  padding=pick(0, 3))
    rows = set(torch.randint(0, s.rows, (12,), generator=g).tolist())
    check(s, rows=rows)


# ---- values ----------------------------------------------------------------------


@pytest.mark.parametrize("dtype,D,fp8", [(BF, 128, False), (FP, 64, False), (BF, 128, True), (FP, 64, True)])
@pytest.mark.parametrize("window", [0, 6])
def test_what_a_row_does_not_see_does_not_touch_it(dtype, D, fp8, window):
    """NaN and infinities in siblings' keys and values, in slots past the end
    and before the window: only rows that see them change."""
    s = TreeScene([20, 133], [9, 12], 4, 2, D, 16, dtype, fp8, window, seed=9, table_slack=9)
    rows = s.cache.view(2, -1, s.row)
    bad = 0x7F if fp8 else float("nan")
    for b in range(2):
        n, L = s.nodes[b], s.ctx[b] + s.nodes[b]
        rows[0, s.slot(b, L - 2), 1] = bad               # a node's key
        rows[1, s.slot(b, L - 4), 3] = bad               # a node's value
        rows[1, s.slot(b, L - 5), 5] = 0xFF if fp8 else float("inf")
        rows[1, s.slot(b, L - 6), s.D + 2] = 0xFF if fp8 else float("-inf")
        for pos in range(L, min(L + 40, s.wide * s.BS)):  # past the end
            rows[:, s.slot(b, pos)] = bad
        if window:
            for pos in range(max(0, s.ctx[b] - window - 12), max(0, s.ctx[b] - window + 3)):
                rows[:, s.slot(b, pos)] = bad
    check(s)


@pytest.mark.parametrize("fp8", [False, True])
def test_queries_that_are_not_finite(fp8):
    s = TreeScene([40, 3], [6, 5], 4, 2, 64, 16, FP, fp8, seed=3)
    s.query[2, 70] = float("nan")
    s.query[4, 3] = float("inf")
    s.query[8, 130] = float("-inf")
    got = s.decode().cpu().double()
    clean("values")
    # the formula's rows: a NaN score anywhere, or +inf, makes the head NaN; what
    # an infinite component makes of all-negative products is NaN too
    want, spread = s.expect()
    hit = torch.zeros(s.rows, s.H, dtype=torch.bool)
    hit[2, 1] = hit[4, 0] = hit[8, 2] = True
    hit = hit.repeat_interleave(s.D, 1)
    assert torch.isnan(got[hit[:s.rows]]).all() and torch.isfinite(got[~hit]).all()
    q = s.query.double().nan_to_num(0.0, 0.0, 0.0)
    tol = tolerance(s, want, spread, q)
    assert ((got - want).abs() <= tol)[~hit].all()


def test_infinite_scores():
    # a key whose products overflow, or are -inf for all rows
    s = TreeScene([10], [3], 2, 1, 64, 16, BF, shape="chain")
    rows = s.cache.view(2, -1, s.row)
    s.query[:, :64] = s.query[:, :64].abs()
    rows[0, s.slot(0, 4), :] = 0.0
    rows[0, s.slot(0, 4), 7] = float("-inf")          # head 0: weight 0; head 1: by the query's sign
    got = s.decode().cpu().double()
    clean("values")
    want, spread = s.expect()
    q = s.query[:3].double().view(3, 2, 64)[:, 1, 7]
    s.cache[:] = s.cache.nan_to_num(0.0, 0.0, 0.0)
    within(got[:, :64], want[:, :64], tolerance(s, want, spread)[:, :64], "head 0")
    for t in range(3):
        row = got[t, 64:]
        assert torch.isnan(row).all() if q[t] < 0 else torch.isfinite(row).all()


def test_nothing_but_minus_infinity():
    s = TreeScene([0], [2], 2, 1, 64, 16, BF, shape="chain")
    rows = s.cache.view(2, -1, s.row)
    rows[0, s.slot(0, 0), :] = rows[0, s.slot(0, 1), :] = 0.0
    rows[0, s.slot(0, 0), 3] = rows[0, s.slot(0, 1), 3] = float("-inf")
    s.query[:] = s.query.abs()
    got = s.decode().cpu()
    clean("values")
    assert torch.isnan(got).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_large_and_small_scores(fp8):
    # scores of several hundred: the weights lie on single keys; and of nearly zero
    for factor in (60.0, 2.0 ** -9):
        s = TreeScene([300, 40], [16, 9], 8, 2, 128, 16, BF, fp8, seed=8)
        s.query = (s.query.float() * factor).to(BF)
        check(s)


def test_rising_scores():
    # every key scores above all before it: the running maximum moves all the time
    s = TreeScene([700], [5], 2, 1, 64, 16, FP, shape="chain")
    rows = s.cache.view(2, -1, s.row)
    for pos in range(705):
        rows[0, s.slot(0, pos)] = pos / 700.0
    s.query[:] = 8.0
    check(s)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_weights_keep_their_low_terms(dtype):
    """Values of alternating sign that cancel but for what the weights have
    beyond 16 bits: a weight rounded to the model's type would show."""
    s = TreeScene([256], [4], 2, 1, 64, 16, dtype, shape="chain", seed=12)
    rows = s.cache.view(2, -1, s.row)
    for pos in range(256):
        rows[1, s.slot(0, pos)] = 1.0
    for pos in range(256, 260):
        rows[1, s.slot(0, pos)] = -64.0
    got = s.decode().cpu().double()
    clean("weights")
    want, spread = s.expect()
    # the output's rounding, weights of two 16-bit terms (2^-16 of a bf16 one), the scores' errors
    d = 64 ** 0.5 * s.query.abs().max().double() * s.cache[0].abs().max().double() * 64 * 2.0 ** -24 + 2.0 ** -16
    tol = torch.finfo(dtype).eps / 2 * 1.01 * want.abs() + (2.0 ** -16 + 2 * d) * spread
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (FP, False), (BF, True), (FP, True)])
def test_many_small_weights_beside_a_large_one(dtype, fp8):
    """One key whose value is 0, and 2000 keys of weight 2^-26 beside it, whose
    value is 1: together they are the output."""
    s = TreeScene([2000] * 40, [2] * 40, 4, 4, 64, 16, dtype, fp8, seed=5)
    rows = s.cache.view(2, -1, s.row)
    one = 0x38                                      # 1.0 in E4M3
    rows[0] = 0
    rows[1] = one if fp8 else 1.0
    for b in range(40):
        rows[0, s.slot(b, 0)] = one if fp8 else 1.0
        rows[1, s.slot(b, 0)] = 0
    # 64 channels of q k / 8 are 18 nats
    s.query[:] = 2.25 / (SCALE8 if fp8 else 1.0)
    got = s.decode().cpu().double()
    clean("small weights")
    want, spread = s.expect()
    # beside the usual, an fp16 weight is off by 2^-30 of the row's largest at most
    tol = tolerance(s, want, spread) + 2002 * 2.0 ** -30 * (SCALE8 if fp8 else 1.0)
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("dtype,fp8", [(BF, False), (FP, True)])
def test_a_scale_that_vanishes(dtype, fp8, alibi):
    """scale * k_scale below what fp32 holds: the scores are 0, not 0 * infinity
    where they are hidden."""
    s = TreeScene([70, 3], [9, 4], 4, 2, 64, 16, dtype, fp8, alibi=alibi, seed=6)
    s.op = dataclasses.replace(s.op, scale=1e-44, k_scale=1e-30)
    p = s.params()
    p.scale, p.k_scale = 1e-44, 1e-30
    got = s.decode(params=p).cpu().double()
    clean("scale")
    want, spread = s.expect()
    assert ((got - want).abs() <= tolerance(s, want, spread)).all()


def test_both_types_errors_are_cleared_together():
    for dtype in (BF, FP):
        s = TreeScene([20], [3], 2, 1, 64, 16, dtype)
        s.tables[0, 0] = -3
        s.decode()
    torch.cuda.synchronize()
    assert B.device_error()[0] == B.PKV_ERR_BOUNDS
    clean("cleared")


# ---- indices ---------------------------------------------------------------------


def test_bad_sequences_are_skipped():
    base = TreeScene([50, 60, 70], [4, 5, 6], 4, 2, 64, 16, FP, seed=1)
    good = base.decode().cpu()
    clean("good")

    def run(detail, hit, **change):
        s = TreeScene([50, 60, 70], [4, 5, 6], 4, 2, 64, 16, FP, seed=1)
        kw = {}
        for k, v in change.items():
            if k in ("max_nodes", "max_len"):
                kw[k] = v
            else:
                setattr(s, k, v)
        got = s.decode(**kw).cpu()
        st, at = error()
        assert st == B.PKV_ERR_BOUNDS and at in detail
        for b in range(3):
            r = slice(int(base.cu[b]), int(base.cu[b + 1]))
            if b not in hit:
                assert torch.equal(got[r], good[r]), (change, b)
            else:
                assert (got[r] == 7.0).all(), (change, b)

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    run({1}, {1}, lens=i32(54, 4, 76))                   # fewer tokens than nodes
    run({1}, {1}, lens=i32(54, -3, 76))
    run({2}, {2}, lens=i32(54, 65, 100000))              # beyond the table
    run({2}, {2}, max_len=70)
    run({2}, {2}, max_nodes=5)
    run({0, 1}, {0, 1}, cu=i32(0, 9999, 9, 15))          # outside the rows, then descending


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_parents_and_tables(fp8):
    for up in (3, 2, -2, 1 << 30):
        s = TreeScene([50, 60], [4, 5], 4, 2, 64, 16, FP, fp8, seed=1)
        s.parents[4 + 2] = up                            # node 2 of the second tree
        got = s.decode().cpu()
        assert error() == (B.PKV_ERR_BOUNDS, 6)
        s.parents[6], s.trees[1][2] = -1, -1             # counts as having none
        check(s, got=got)
    for entry in (-1, 10000):
        s = TreeScene([50, 60], [4, 5], 4, 2, 64, 16, FP, fp8, seed=1)
        s.tables[0, 1] = entry
        got = s.decode().cpu()
        assert error() == (B.PKV_ERR_BOUNDS, 1)
        want, spread = s_expect_second(s)
        within(got[4:9].double(), want, spread, "the other sequence")


def s_expect_second(s):
    s.tables[0, 1] = 0
    want, spread = s.expect(set(range(4, 9)))
    return want[4:9], tolerance(s, want, spread)[4:9]


# ---- streams, graphs -------------------------------------------------------------


def test_other_stream_and_repeats():
    s = TreeScene([3000, 100, 40], [30, 8, 1], 8, 2, seed=2)
    first = check(s, rows={0, 30, 38})
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            again = s.decode()
        side.synchronize()
        assert torch.equal(again.cpu(), first)
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(s.query, 7.0).to(DEV)
    torch.cuda.synchronize()
    s.decode(out=out, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), first)


def test_two_workspaces_at_once():
    a, b = (TreeScene([4000, 900], [20, 31], 8, 2, seed=x) for x in (1, 2))
    want = [check(s, rows={0, 25}) for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                outs.append(s.decode())
    torch.cuda.synchronize()
    clean("two streams")
    for i, o in enumerate(outs):
        assert torch.equal(o.cpu(), want[i % 2])


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_replays_new_trees(fp8):
    s = TreeScene([2000, 300, 60], [20, 12, 3], 8, 2, fp8=fp8, seed=5, padding=8)
    p = s.params()
    dev = {k: getattr(s, k).to(DEV) for k in ("cache", "query", "tables", "lens", "cu")}
    parents = torch.zeros(s.rows + 8, dtype=torch.int32, device=DEV)
    parents[:s.rows] = s.parents.to(DEV)
    out = torch.full_like(dev["query"], 7.0)
    size = B.paged_attn_decode_tree_workspace_size(3, 32, 2100, p)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)

    def call():
        B.paged_attn_decode_tree(out, dev["query"], dev["cache"], dev["tables"], dev["lens"], dev["cu"],
                                 parents, 32, 2100, p, ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    check(s, got=out, rows={0, 19, 20, 34})
    # other trees, lengths and queries in the same buffers
    n = TreeScene([100, 1500, 0], [30, 2, 11], 8, 2, fp8=fp8, seed=6)
    n.tables, n.wide = s.tables, s.wide
    n.blocks, n.cache = s.blocks, s.cache
    out.fill_(7.0)
    dev["query"][:n.rows] = n.query.to(DEV)
    dev["lens"].copy_(n.lens)
    dev["cu"].copy_(n.cu)
    parents[:n.rows] = n.parents.to(DEV)
    # a captured call and an eager one between its replays share the workspace, in order
    graph.replay()
    a = out.clone()
    call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)
    n.tables = n.tables.clone()
    n.query = torch.cat([n.query, s.query[n.rows:]])
    b = {"n": n}
    assert n.lens.max() <= n.wide * n.BS
    check(n, got=out, rows={0, 29, 30, 31, 32, 42})
    del b


_FIRST = """
import sys
sys.path[:0] = sys.argv[1:]
import torch
from paged_kv_cache_246_gb300 import binding as B
from tree_helpers import BF, TreeScene, tolerance
s = TreeScene([500, 20], [7, 3], 8, 2, dtype=BF)
p, t = s.params(), [x.to("cuda:0") for x in (s.query, s.cache, s.tables, s.lens, s.cu, s.parents)]
out = torch.zeros_like(t[0])
ws = torch.empty(max(16, B.paged_attn_decode_tree_workspace_size(2, 7, 507, p)), dtype=torch.uint8, device="cuda:0")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    B.paged_attn_decode_tree(out, *t, 7, 507, p, ws)
graph.replay()
torch.cuda.synchronize()
want, spread = s.expect()
assert B.device_error()[0] == B.PKV_OK
assert ((out.cpu().double() - want).abs() <= tolerance(s, want, spread)).all()
print("captured")
"""


def test_the_first_call_of_a_process_is_captured():
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", _FIRST, os.path.dirname(here), here], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("fp8", [False, True])
def test_sequences_that_share_context_blocks(fp8):
    s = TreeScene([160, 160, 165], [9, 20, 3], 8, 2, fp8=fp8, seed=8)
    s.tables[1, :10] = s.tables[0, :10]
    s.tables[2, :10] = s.tables[0, :10]
    check(s)


def test_workspace_is_refused_when_too_small():
    s = TreeScene([3000], [64], 8, 1, 128, 16)
    need = B.paged_attn_decode_tree_workspace_size(1, 64, 3064, s.params())
    if need == 0:
        pytest.skip("no workspace")
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device=DEV),
               torch.empty(need + 256, dtype=torch.uint8, device=DEV)[16:]):
        with pytest.raises(B.PkvError) as e:
            s.decode(workspace=ws)
        assert e.value.status == B.PKV_ERR_INVALID


def test_finite_8_bit_extremes():
    s = TreeScene([200], [10], 4, 1, 128, 16, BF, True)
    s.cache = torch.randint(0, 256, s.cache.shape, generator=s.gen).to(torch.uint8)
    s.cache[(s.cache & 0x7F) == 0x7F] = 0x7E
    check(s)
    s.cache = codes(torch.randn(s.cache.shape, generator=s.gen) * 2.0 ** -9)
    check(s)

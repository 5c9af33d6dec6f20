"""paged_attn_decode_tree over values that are not finite deep in the context,
against the fp64 oracle: what a row sees goes into it as the formula says,
wherever the key lies and however small its weight."""
import random

import pytest
import torch

import oracle as O

from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8
from test_gpu_tree import DEV, check, clean, within
from tree_helpers import BF, FP, TreeScene, tolerance

pytestmark = pytest.mark.gpu

INF = float("inf")


def put(s: TreeScene, b, pos, head, channel, value, half=1):
    s.cache.view(2, -1, s.row)[half, s.slot(b, pos), head * s.D + channel] = value


TYPES = [(BF, 128), (FP, 128), (BF, 64), (FP, 64)]


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("ctx,window,alibi", [(200, 0, False), (1500, 0, False), (1500, 0, True), (1500, 900, False)])
def test_infinite_values_in_the_context(dtype, D, ctx, window, alibi):
    """In tiles that all rows see whole, in both halves of a tile and of a row;
    200: sequences that are not cut, 1500: cut into parts."""
    s = TreeScene([ctx, ctx + 5, ctx - 3], [6, 20, 3], 4, 2, D, 16, dtype, window=window, alibi=alibi, seed=ctx + D)
    for b in range(3):
        far = s.ctx[b] - min(window or ctx, ctx) + 40      # inside every row's window
        put(s, b, far, 0, 3, INF)
        put(s, b, far + 70, 0, D - 2, -INF)
        put(s, b, far + 1, 1, 5, INF)                      # both in one channel: NaN
        put(s, b, far + 30, 1, 5, -INF)
        put(s, b, far + 64, 1, D // 2, float("nan"))
    got = check(s)
    assert torch.isinf(got).any() and torch.isnan(got).any() and torch.isfinite(got).any()


@pytest.mark.parametrize("dtype,D", TYPES)
def test_infinite_values_of_small_weight(dtype, D):
    """Scores spread over some hundred: most weights vanish beside the largest
    in 32 bits, and the formula's product with infinity does not."""
    s = TreeScene([700, 130], [5, 9], 4, 2, D, 16, dtype, seed=D)
    s.query = (s.query.float() * 12).to(dtype)
    for b in range(2):
        for i, pos in enumerate(range(3, 120, 13)):
            put(s, b, pos, i % 2, i, INF if i % 3 else -INF)
    check(s)


@pytest.mark.parametrize("dtype,D", TYPES)
@pytest.mark.parametrize("where", ["context", "node"])
def test_infinite_values_of_no_weight(dtype, D, where):
    """A score of -infinity leaves a weight of exactly zero, and 0 * infinity is NaN."""
    s = TreeScene([300], [4], 2, 1, D, 16, dtype, shape="chain", seed=3)
    at = 40 if where == "context" else 300
    s.query[:, 7] = 1.0                                    # head 0: -infinity at the key; head 1 by sign
    s.cache.view(2, -1, s.row)[0, s.slot(0, at)] = 0.0
    put(s, 0, at, 0, 7, -INF, half=0)
    s.query[:, D + 7] = torch.tensor([-1.0, -2.0, -1.0, -0.5])[:4].to(dtype)    # +infinity: NaN rows
    put(s, 0, at, 0, 2, INF)
    put(s, 0, 60, 0, 9, -INF)
    got = s.decode().cpu()
    clean("no weight")
    want, spread = s.expect()
    assert torch.isinf(want[:, 9]).all() and torch.isnan(want[:, D:]).all()
    want[:, 2] = float("nan")      # said here: a library's product may pass over a factor of zero
    s.cache[:] = s.cache.nan_to_num(0.0, 0.0, 0.0)         # for the tolerance
    within(got.double(), want, tolerance(s, want, spread), "no weight")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("query", [1.0, -INF])
@pytest.mark.parametrize("ctx", [150, 1500])
def test_infinite_values_and_nothing_but_minus_infinity(dtype, query, ctx):
    s = TreeScene([ctx], [3], 2, 1, 64, 16, dtype, shape="chain", seed=4)
    rows = s.cache.view(2, -1, s.row)
    s.query[:] = 0.5
    s.query[:, 3] = s.query[:, 64 + 3] = query
    rows[0] = 0.25
    rows[0, :, 3] = 1.0 if query < 0 else -INF
    rows[1, :, 5] = INF
    put(s, 0, ctx // 2, 0, 6, -INF)
    put(s, 0, ctx, 0, 7, INF)
    got = s.decode().cpu()
    clean("minus infinity")
    assert torch.isnan(got).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinite_values_of_some_sequences(dtype):
    """Several segments a CTA, every third sequence with one: the others keep
    every bit."""
    s = TreeScene([500] * 90, [3] * 90, 4, 2, 64, 16, dtype, seed=6)
    clear = s.decode().cpu()
    clean("finite")
    hit = torch.zeros(s.rows, s.H, s.D, dtype=torch.bool)
    for b in range(0, 90, 3):
        put(s, b, 11 + 4 * b, b % 2, b % 64, INF if b % 2 else -INF)
        hit[3 * b:3 * b + 3, 2 * (b % 2):2 * (b % 2) + 2, b % 64] = True
    hit = hit.view(s.rows, -1)
    got = s.decode().cpu()
    clean("some")
    sign = torch.cat([torch.full((3,), INF if b % 2 else -INF, dtype=dtype) for b in range(90)])
    assert torch.equal(got[hit], sign[:, None].expand_as(got)[hit])
    assert torch.equal(got[~hit], clear[~hit])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinite_values_with_several_row_tiles_and_shared_blocks(dtype):
    s = TreeScene([640, 640], [130, 70], 4, 2, 64, 16, dtype, seed=7, padding=1)
    s.tables[1, :40] = s.tables[0, :40]
    put(s, 0, 77, 0, 1, INF)
    put(s, 0, 333, 1, 63, -INF)
    put(s, 1, 640, 0, 5, INF)                              # and in a node's
    check(s, rows={0, 31, 32, 33, 64, 129, 130, 131, 162, 199})


def test_a_long_context_full_of_them():
    # every key's value is infinite in one channel: the look through them ends in time
    s = TreeScene([40000], [3], 2, 1, 64, 16, BF, seed=8)
    s.cache.view(2, -1, s.row)[1, :, 10] = INF
    got = s.decode().cpu().view(3, 2, 64)
    clean("long")
    assert torch.equal(got[:, :, 10], torch.full((3, 2), INF, dtype=BF))
    assert torch.isfinite(got[:, :, 11:]).all() and torch.isfinite(got[:, :, :10]).all()


def test_not_finite_codes_in_the_context():
    # over an 8-bit cache a value is finite or NaN, and NaN is NaN at any weight
    s = TreeScene([700, 90], [5, 9], 4, 2, 64, 16, FP, True, seed=9)
    s.cache.view(2, -1, s.row)[1, s.slot(0, 50), 3] = 0x7F
    s.cache.view(2, -1, s.row)[1, s.slot(1, 20), 64] = 0xFF
    check(s)
    torch.cuda.synchronize(DEV)
    assert B.device_error()[0] == B.PKV_OK


def by_class(s: TreeScene):
    """The formula, what is not finite said by cases: a row whose scores hold a
    NaN or +infinity, or nothing but -infinity, is NaN; an infinite value makes
    its channel infinite in the rows that see it, NaN where the weight is 0 (a
    score of -infinity) or the other infinity is there too."""
    out = torch.full((s.rows, s.H, s.D), float("nan"), dtype=torch.float64)
    cache = s.cache.view(2, -1, s.KVH, s.D)
    cache = cache.view(torch.float8_e4m3fn).double() * float(torch.tensor(SCALE8)) if s.fp8 else cache.double()
    for b, (n, ctx) in enumerate(zip(s.nodes, s.ctx)):
        if n == 0:
            continue
        slots = torch.tensor([s.slot(b, j) for j in range(ctx + n)])
        depth = torch.tensor(s.depths(b))
        place = torch.cat([torch.arange(ctx), ctx + depth])
        ago = place - (ctx + depth)[:, None]
        seen = torch.zeros(n, ctx + n, dtype=torch.bool)
        seen[:, :ctx] = True
        for t in range(n):
            seen[t, [ctx + c for c in O.tree_ancestors(s.trees[b], t)]] = True
        if s.window > 0:
            seen &= ago > -s.window
        rows = slice(int(s.cu[b]), int(s.cu[b + 1]))
        for h in range(s.H):
            k, v = cache[:, slots, h // (s.H // s.KVH)]
            q = s.query[rows].double().view(n, s.H, s.D)[:, h]
            x = (q[:, None] * k[None]).sum(2) * s.D ** -0.5 + (s.slopes[h] * ago if s.slopes else 0.0)
            none = (seen & (x.isnan() | (x == INF))).any(1) | ~(seen & (x > -INF)).any(1)
            w = torch.softmax(torch.where(seen, x.nan_to_num(0.0, 0.0, -INF), -INF), 1).nan_to_num(0.0)
            both = (seen & (x == -INF)).double() @ (~v.isfinite()).double() > 0
            up = (seen.double() @ (v.isnan() | (v == INF)).double() > 0) | both
            down = (seen.double() @ (v.isnan() | (v == -INF)).double() > 0) | both
            o = w @ v.nan_to_num(0.0, 0.0, 0.0)
            o = torch.where(up & down, float("nan"), torch.where(up, INF, torch.where(down, -INF, o)))
            o[none] = float("nan")
            out[rows, h] = o
    return out.view(s.rows, -1)


@pytest.mark.parametrize("seed", range(40))
def test_drawn_values_that_are_not_finite(seed):
    """Anywhere in keys, values and queries, seen by all, by some or by none."""
    r = random.Random(seed)
    n, longest, widest = r.randint(1, 4), r.choice([20, 200, 400, 900]), r.choice([3, 20, 80])
    ctx, nodes = [r.randint(0, longest) for _ in range(n)], [r.randint(0, widest) for _ in range(n)]
    nodes[-1] = max(1, nodes[-1])
    kv, fp8 = r.choice([1, 2]), r.random() < 0.3
    s = TreeScene(ctx, nodes, kv * r.choice([1, 2, 4, 5]), kv, r.choice([64, 128]), r.choice([16, 32]), r.choice([BF, FP]),
                  fp8, r.choice([0, 0, 1, 30, 200, 300]), r.random() < 0.25,
                  r.choice(["bushy", "chain", "star", "forest"]), seed)
    rows = s.cache.view(2, -1, s.row)
    kinds = [0x7F, 0xFF] if fp8 else [INF, -INF, INF, -INF, float("nan")]
    for _ in range(r.randint(1, 12)):
        b = r.randrange(n)
        at = s.slot(b, r.randrange(ctx[b] + nodes[b])) if ctx[b] + nodes[b] and r.random() < 0.8 else r.randrange(rows.shape[1])
        half, c = r.choice([0, 1, 1, 1]), r.randrange(s.row)
        rows[half, at, c] = r.choice(kinds)
        if r.random() < 0.3:                               # key and value of one token
            rows[1 - half, at, c // s.D * s.D + r.randrange(s.D)] = r.choice(kinds)
    if r.random() < 0.3:
        s.query[r.randrange(s.rows), r.randrange(s.H * s.D)] = r.choice([INF, -INF, float("nan")])
    got = s.decode().cpu().double()
    clean("drawn")
    want = by_class(s)
    if not s.fp8:
        s.cache[:] = s.cache.nan_to_num(0.0, 0.0, 0.0)     # for the tolerance
    else:
        s.cache[(s.cache & 0x7F) == 0x7F] = 0
    s.query = s.query.nan_to_num(0.0, 0.0, 0.0)
    _, spread = s.expect()                                 # of the finite values alone
    within(got, want, tolerance(s, want.nan_to_num(0.0, 0.0, 0.0), spread), "drawn")

"""The write with positions of several axes, acceptance and commit against the
oracle, and a whole speculative step."""
import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8, values
from tree_helpers import BF, FP, TreeScene, random_tree, tolerance

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def error():
    torch.cuda.synchronize()
    return B.device_error()


def clean(where):
    st, d = error()
    assert st == B.PKV_OK, f"{where}: {B.status_string(st)} at {d}"


def within(got, want, tol, what):
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float(((got - want).abs() - tol).max())}"


# ---- kv_cache_write_rope_axes ----------------------------------------------------


def axes_scene(T, dtype, D, BS, heads, kv_heads, fp8, seed):
    return TreeScene([T], [1], heads, kv_heads, D, BS, dtype, fp8, seed=seed)


def check_axes(s, T, rot, inter, packed, axes, num_axes, in_place=False, seed=0):
    p, g = s.params(), torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, s.H * s.D + 2 * s.row, generator=g).to(s.dtype)
    split = [s.H * s.D, s.row, s.row]
    q, k, v = qkv.split(split, 1)
    dq, dk, dv = qkv.to(DEV).split(split, 1)
    if not packed:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    slots = torch.randperm(s.blocks * s.BS, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.2] = -1
    pos = torch.randint(0, 200, (num_axes, T), generator=g)
    pos[:, slots < 0] = -5                               # of a padding token: not looked at
    table, cache = B.rope_table(200, rot, device=DEV), s.cache.to(DEV)
    out = dq if in_place else torch.full((T, s.H * s.D), 7.0, dtype=s.dtype, device=DEV)
    B.kv_cache_write_rope_axes(out, dq, dk, dv, cache, slots.to(DEV), pos.to(DEV), table, axes, p,
                               interleaved=inter)
    clean("axes")
    eq, ek, ev = O.kv_cache_write_rope_axes(q, k, v, slots, pos, table.cpu(), axes, s.op, inter)
    kept = slots >= 0
    half = torch.finfo(s.dtype).eps / 2
    # fp32: two products and their sum, each off by 2^-24 of |x1| + |x2| <= 12, then one rounding
    # (fp16 below its normal range: half of 2^-24)
    slop = 3 * 2.0 ** -24 * 12
    got = out.cpu().double()
    within(got[kept], eq[kept], half * eq[kept].abs() * 1.001 + slop + 2.0 ** -25, "query")
    before = q.double() if in_place else torch.full_like(got, 7.0)
    assert torch.equal(got[~kept], before[~kept])
    rows, old = (values(c, s.fp8).view(2, -1, s.row) for c in (cache.cpu(), s.cache))
    for i, want in ((0, ek), (1, ev)):
        have = rows[i, slots[kept]]
        if s.fp8:
            # the nearest code: half a step (2^-4 of the value, 2^-10 below 2^-6), saturating
            e = want[kept].clamp(-448, 448)
            within(have, e, e.abs() * 2.0 ** -4 * 1.001 + 2.0 ** -10 + slop / SCALE8, "codes")
        elif i:
            assert torch.equal(have, want[kept])         # values: a copy
        else:
            within(have, want[kept], half * want[kept].abs() * 1.001 + slop + 2.0 ** -25, "key")
        rest = torch.ones(old.shape[1], dtype=torch.bool)
        rest[slots[kept]] = False
        assert torch.equal(rows[i, rest], old[i, rest])


@pytest.mark.parametrize("T", [1, 2, 37])
@pytest.mark.parametrize("dtype,D,BS,heads,kv_heads,rot,inter,fp8,packed,sections,woven", [
    (BF, 128, 16, 32, 8, 128, False, False, True, (16, 24, 24), False),
    (BF, 128, 16, 8, 2, 128, False, True, True, (24, 20, 20), True),
    (FP, 64, 32, 4, 4, 64, True, False, False, (8, 12, 12), False),
    (FP, 64, 16, 5, 1, 32, True, True, True, (5, 5, 6), True),
    (BF, 64, 32, 6, 2, 16, False, True, True, (3, 5), False),
    (FP, 128, 16, 6, 2, 96, False, False, False, (12, 13, 13, 10), True),
    (BF, 128, 16, 1, 1, 48, True, False, True, (0, 0, 24), False),
])
def test_axes_write(T, dtype, D, BS, heads, kv_heads, rot, inter, fp8, packed, sections, woven):
    s = axes_scene(100, dtype, D, BS, heads, kv_heads, fp8, T)
    check_axes(s, T, rot, inter, packed, B.rope_pair_axes(sections, woven), len(sections), seed=T)


@pytest.mark.parametrize("dtype,D,heads,kv_heads,rot,inter,fp8", [
    (BF, 128, 4, 1, 128, True, False), (FP, 64, 3, 3, 32, False, False), (FP, 64, 2, 1, 64, True, True),
    (BF, 128, 2, 2, 64, False, True)])
def test_axes_bulk(dtype, D, heads, kv_heads, rot, inter, fp8):
    # more tokens than 6 per SM: the streaming form
    s = axes_scene(1400, dtype, D, 16, heads, kv_heads, fp8, 1)
    check_axes(s, 1111, rot, inter, True, B.rope_pair_axes((rot // 8, rot // 8, rot // 4)), 3)


@pytest.mark.parametrize("T", [1, 30, 1000])
def test_axes_rows_of_a_wider_tensor(T):
    s = axes_scene(1100, FP, 64, 16, 4, 2, False, seed=T)
    g, axes = torch.Generator().manual_seed(1), B.rope_pair_axes([8, 12, 12])
    q, k, v = (torch.randn(T, w, generator=g).to(FP).to(DEV) for w in (s.H * s.D, s.row, s.row))
    slots = torch.randperm(s.blocks * s.BS, generator=g)[:T].to(DEV)
    wide = torch.full((3, 1200), -9, dtype=torch.int64)         # none of these is looked at
    wide[:, 5:5 + T] = torch.randint(0, 200, (3, T), generator=g)
    pos, table, outs = wide.to(DEV)[:, 5:5 + T], B.rope_table(200, 64, device=DEV), []
    for positions in (pos, pos.contiguous()):
        out, cache = torch.zeros_like(q), s.cache.to(DEV)
        B.kv_cache_write_rope_axes(out, q, k, v, cache, slots, positions, table, axes, s.params())
        clean("axes")
        outs.append((out, cache))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_axes_in_place():
    s = axes_scene(600, BF, 128, 16, 8, 2, False, 2)
    check_axes(s, 500, 128, False, True, B.rope_pair_axes((16, 24, 24)), 3, in_place=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [3, 1200])
def test_axes_that_agree_are_the_rotating_write(fp8, T):
    s = axes_scene(1300, BF, 128, 16, 4, 2, fp8, 3)
    p, g = s.params(), torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, n, generator=g).to(BF).to(DEV) for n in (s.H * s.D, s.row, s.row))
    slots = torch.randperm(s.blocks * s.BS, generator=g)[:T].to(DEV)
    pos = torch.randint(0, 300, (T,), generator=g).to(DEV)
    table = B.rope_table(300, 64, device=DEV)
    for inter in (False, True):
        a, b = s.cache.to(DEV), s.cache.to(DEV)
        qa, qb = torch.zeros_like(q), torch.zeros_like(q)
        B.kv_cache_write_rope(qa, q, k, v, a, slots, pos, table, p, interleaved=inter)
        B.kv_cache_write_rope_axes(qb, q, k, v, b, slots, pos.expand(3, T).contiguous(), table,
                                   B.rope_pair_axes((16, 8, 8), woven=True), p, interleaved=inter)
        clean("both")
        assert torch.equal(a, b) and torch.equal(qa, qb)


@pytest.mark.parametrize("T", [4, 1000])
def test_axes_bad_tokens(T):
    s = axes_scene(1100, FP, 64, 16, 4, 2, False, 4)
    p, g = s.params(), torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(T, n, generator=g).to(FP).to(DEV) for n in (s.H * s.D, s.row, s.row))
    table = B.rope_table(50, 32, device=DEV)
    axes = B.rope_pair_axes((8, 8, 0))
    good_slots = torch.randperm(s.blocks * s.BS, generator=g)[:T]

    def run(pos, slots):
        out, cache = torch.full_like(q, 7.0), s.cache.to(DEV)
        B.kv_cache_write_rope_axes(out, q, k, v, cache, slots.to(DEV), pos.to(DEV), table, axes, p)
        return out.cpu(), cache.cpu()

    pos = torch.randint(0, 50, (3, T), generator=g)
    want = run(pos, good_slots)
    clean("good")
    for axis, slot, value in ((0, None, 50), (1, None, -1), (1, None, 1 << 40), (None, s.blocks * s.BS, 0)):
        bad, slots = pos.clone(), good_slots.clone()
        if axis is None:
            slots[2] = slot
        else:
            bad[axis, 2] = value
        out, cache = run(bad, slots)
        assert error() == (B.PKV_ERR_BOUNDS, 2)
        keep = torch.arange(T) != 2
        assert torch.equal(out[keep], want[0][keep]) and (out[2] == 7.0).all()
        rows, old, new = (c.view(2, -1, s.row) for c in (cache, s.cache, want[1]))
        assert torch.equal(rows[:, good_slots[2]], old[:, good_slots[2]])
        assert torch.equal(rows[:, good_slots[keep]], new[:, good_slots[keep]])
    # an axis that no pair turns by may hold anything
    free = pos.clone()
    free[2] = -7
    out, cache = run(free, good_slots)
    clean("unused axis")
    assert torch.equal(out, want[0]) and torch.equal(cache, want[1])


# ---- paged_attn_tree_accept ------------------------------------------------------


def trees(nodes, seed, vocabulary, shape="bushy"):
    g = torch.Generator().manual_seed(seed)
    cu = torch.tensor([0] + list(nodes)).cumsum(0).int()
    up = torch.tensor([p for n in nodes for p in (random_tree(n, g, shape) if n else [])], dtype=torch.int32)
    T = int(cu[-1])
    draft, target = (torch.randint(0, vocabulary, (T,), generator=g) for _ in range(2))
    return cu, up, draft, target


def accept(cu, up, draft, target, most, max_nodes):
    n = cu.numel() - 1
    acc = torch.full((n, most), 99, dtype=torch.int32, device=DEV)
    num = torch.full((n,), 99, dtype=torch.int32, device=DEV)
    tok = torch.full((n,), 99, dtype=torch.int64, device=DEV)
    B.paged_attn_tree_accept(acc, num, tok, draft.to(DEV), target.to(DEV), up.to(DEV), cu.to(DEV), max_nodes)
    return acc.tolist(), num.tolist(), tok.tolist()


@pytest.mark.parametrize("vocabulary", [1, 2, 4, 1 << 40])
@pytest.mark.parametrize("most", [1, 3, 40, 300])
def test_accept(vocabulary, most):
    nodes = [1, 0, 5, 64, 33, 256, 31, 32, 2]
    for shape in ("bushy", "chain", "star", "forest"):
        args = trees(nodes, most, vocabulary, shape)
        got = accept(*args, most, 256)
        clean("accept")
        cu, up, draft, target = args
        assert got == O.paged_attn_tree_accept(draft, target, up, cu, most)


def test_accept_bad_trees():
    cu, up, draft, target = trees([6, 7, 8], 3, 1)
    good = accept(cu, up, draft, target, 4, 8)
    clean("good")
    bad = up.clone()
    bad[6 + 3] = 3
    got = accept(cu, bad, draft, target, 4, 8)
    assert error() == (B.PKV_ERR_BOUNDS, 9)
    assert [x[0] for x in got] == [x[0] for x in good] and [x[2] for x in got] == [x[2] for x in good]
    bad[9] = -1
    assert got == accept(cu, bad, draft, target, 4, 8)
    clean("as none")
    for cu_bad, hit, most in ((cu, 2, 7), (torch.tensor([0, 6, 13, 22], dtype=torch.int32), 2, 9),
                              (torch.tensor([0, 6, 5, 21], dtype=torch.int32), 1, 16),
                              (torch.tensor([-1, 6, 13, 21], dtype=torch.int32), 0, 8)):
        got = accept(cu_bad, up, draft, target, 4, most)
        assert error()[0] == B.PKV_ERR_BOUNDS
        assert got[0][hit] == [-1] * 4 and got[1][hit] == 0 and got[2][hit] == -1


# ---- kv_commit_tree --------------------------------------------------------------


def commit(s, caches, accepted):
    dev = [c.to(DEV) for c in caches]
    B.kv_commit_tree(dev, accepted.to(DEV), s.tables.to(DEV), s.lens.to(DEV), s.cu.to(DEV), s.params())
    return [c.cpu() for c in dev]


@pytest.mark.parametrize("dtype,D,BS,kv_heads,fp8,layers", [(BF, 128, 16, 8, False, 1), (FP, 64, 32, 1, False, 3),
                                                            (BF, 64, 16, 2, True, 2), (FP, 128, 16, 24, True, 40)])
@pytest.mark.parametrize("most", [1, 5, 17])
def test_commit(dtype, D, BS, kv_heads, fp8, layers, most):
    nodes = [1, 30, 0, 17, 64]
    s = TreeScene([0, 5, 40, 15, 33], nodes, kv_heads, kv_heads, D, BS, dtype, fp8, seed=most)
    g = s.gen
    accepted = torch.full((5, most), -1, dtype=torch.int32)
    for b, n in enumerate(nodes):
        m = min(most, n)
        if m:
            path = torch.randperm(n, generator=g)[:m].sort().values
            accepted[b, :m] = path.int()
            if b == 3:
                accepted[b, m // 2:] = -2                # any negative number ends it
    caches = [s.cache] + [s.cache.roll(i + 1, 1) for i in range(layers - 1)]
    got = commit(s, caches, accepted)
    clean("commit")
    want = [c.clone() for c in caches]
    O.kv_commit_tree(want, accepted, s.tables, s.lens, s.cu, s.op)
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_commit_of_the_longest_paths():
    s = TreeScene([9, 3], [256, 256], 2, 2, 64, 16, FP, seed=2)
    accepted = torch.full((2, 256), -1, dtype=torch.int32)
    accepted[0] = torch.arange(256)                       # nothing moves
    accepted[1, :255] = torch.arange(1, 256)              # everything by one
    got = commit(s, [s.cache], accepted)[0]
    clean("commit")
    want = s.cache.clone()
    O.kv_commit_tree([want], accepted, s.tables, s.lens, s.cu, s.op)
    assert torch.equal(got, want)


def test_commit_bad_paths():
    for change, hit in ((dict(a=(1, 2, 2)), 1), (dict(a=(1, 1, 9)), 1), (dict(a=(1, 0, 40)), 1),
                        (dict(a=(1, 0, 17)), 1), (dict(t=(1, 1, -1)), 1), (dict(t=(1, 2, 5000)), 1),
                        (dict(lens=(0, 3)), 0), (dict(lens=(2, 1 << 20)), 2), (dict(lens=(2, -1)), 2),
                        (dict(cu=(3, 9)), 2), (dict(a=(1, 0, -1)), 1)):
        s = TreeScene([30, 20, 7], [9, 17, 6], 2, 2, 64, 16, FP, seed=1)
        accepted = torch.tensor([[0, 3, 5, -1], [0, 2, 9, 16], [0, 1, 4, 5]], dtype=torch.int32)
        good = commit(s, [s.cache], accepted)[0]
        clean("good")
        if "a" in change:
            b, i, v = change["a"]
            accepted[b, i] = v
        if "t" in change:
            b, i, v = change["t"]
            s.tables[b, i] = v
        if "lens" in change:
            s.lens[change["lens"][0]] = change["lens"][1]
        if "cu" in change:
            s.cu[change["cu"][0]] = change["cu"][1]
        got = commit(s, [s.cache], accepted)[0]
        assert error() == (B.PKV_ERR_BOUNDS, hit), change
        fresh = TreeScene([30, 20, 7], [9, 17, 6], 2, 2, 64, 16, FP, seed=1)
        for b in range(3):
            src = s.cache if b == hit else good
            for pos in range(fresh.ctx[b] + fresh.nodes[b]):
                at = fresh.slot(b, pos)
                assert torch.equal(got.view(2, -1, s.row)[:, at], src.view(2, -1, s.row)[:, at]), (change, b, pos)


# ---- the step --------------------------------------------------------------------


@pytest.mark.parametrize("dtype,D,BS,heads,kv_heads,fp8,window", [(BF, 128, 16, 8, 2, False, 0),
                                                                  (FP, 64, 32, 4, 4, True, 50)])
def test_a_step_of_all_calls(dtype, D, BS, heads, kv_heads, fp8, window):
    """Prompts with image positions, a tree's nodes written and attended to, a
    path accepted and committed in two layers, and the next step's attention over
    the result: captured in one graph and against the oracle, step by step."""
    ctx, nodes = [70, 33, 5], [12, 7, 9]
    s = TreeScene(ctx, nodes, heads, kv_heads, D, BS, dtype, fp8, window, seed=21, table_slack=2)
    p, g, T = s.params(), s.gen, s.rows
    axes = B.rope_pair_axes((D // 8, D // 8, D // 4))
    table = B.rope_table(200, D, device=DEV)
    qkv = torch.randn(T, (heads + 2 * kv_heads) * D, generator=g).to(dtype)
    place = torch.tensor([c + d for b, c in enumerate(ctx) for d in s.depths(b)])
    pos = torch.stack([place, place + 3, place + 40])        # text behind an image: the axes differ
    slots = torch.tensor([s.slot(b, ctx[b] + t) for b in range(3) for t in range(nodes[b])])
    _, _, draft, target = trees(nodes, 5, 2)
    d = {k: v.to(DEV) for k, v in dict(qkv=qkv, pos=pos, slots=slots, draft=draft, target=target, lens=s.lens,
                                       cu=s.cu, up=s.parents, tables=s.tables).items()}
    layers = [s.cache.to(DEV), s.cache.flip(1).contiguous().to(DEV)]
    rot, out = (torch.zeros(T, heads * D, dtype=dtype, device=DEV) for _ in range(2))
    acc = torch.zeros(3, 6, dtype=torch.int32, device=DEV)
    num, tok = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    max_len = int(s.lens.max())
    ws = torch.empty(max(16, B.paged_attn_decode_tree_workspace_size(3, 12, max_len, p)), dtype=torch.uint8,
                     device=DEV)
    q, k, v = d["qkv"].split([heads * D, kv_heads * D, kv_heads * D], 1)

    def step():
        for cache in layers:
            B.kv_cache_write_rope_axes(rot, q, k, v, cache, d["slots"], d["pos"], table, axes, p)
            B.paged_attn_decode_tree(out, rot, cache, d["tables"], d["lens"], d["cu"], d["up"], 12, max_len, p, ws)
        B.paged_attn_tree_accept(acc, num, tok, d["draft"], d["target"], d["up"], d["cu"], 12)
        B.kv_commit_tree(layers, acc, d["tables"], d["lens"], d["cu"], p)

    keep = [c.clone() for c in layers]
    step()
    torch.cuda.synchronize()
    eager = [x.clone() for x in (rot, out, acc, num, tok, *layers)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c, x in zip(layers, keep):
        c.copy_(x)
    for x in (rot, out, acc, num, tok):
        x.zero_()
    graph.replay()
    clean("step")
    for x, y in zip(eager, (rot, out, acc, num, tok, *layers)):
        assert torch.equal(x.view(torch.uint8) if x.dtype == torch.uint8 else x, y)

    # the last layer against the oracle: what the library wrote is what it attends to
    half = torch.finfo(dtype).eps / 2
    hq, hk, hv = qkv.split([heads * D, kv_heads * D, kv_heads * D], 1)
    eq, _, _ = O.kv_cache_write_rope_axes(hq, hk, hv, slots, pos, table.cpu(), axes, s.op, False)
    within(rot.cpu().double(), eq, half * eq.abs() * 1.001 + 3 * 2.0 ** -24 * 12 + 2.0 ** -25, "query")
    written = keep[1].clone()
    again = torch.zeros_like(rot)
    B.kv_cache_write_rope_axes(again, q, k, v, written, d["slots"], d["pos"], table, axes, p)
    s.cache, s.query = written.cpu(), rot.cpu()
    want, spread = s.expect()
    within(out.cpu().double(), want, tolerance(s, want, spread), "attention")
    want_acc = O.paged_attn_tree_accept(draft, target, s.parents, s.cu, 6)
    assert (acc.tolist(), num.tolist(), tok.tolist()) == want_acc
    moved = [s.cache.clone()]
    O.kv_commit_tree(moved, acc.cpu(), s.tables, s.lens, s.cu, s.op)
    assert torch.equal(layers[1].cpu().view(torch.uint8), moved[0].view(torch.uint8))

    # the next step: one new node each behind the committed path
    n = TreeScene([c + m for c, m in zip(ctx, num.tolist())], [1, 1, 1], heads, kv_heads, D, BS, dtype, fp8, window,
                  seed=22)
    n.tables, n.cache = s.tables, layers[1].cpu()
    got = n.decode().cpu().double()
    clean("next step")
    want, spread = n.expect()
    within(got, want, tolerance(n, want, spread), "next step")

"""The block-sparse decode's kernels against the fp64 oracle: sizes and masks
where they can go wrong, bad indices, streams, graphs, and a run of them
together."""
import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8, Scene, attention_tolerance, codes, values

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


def error():
    torch.cuda.synchronize()
    return B.device_error()


def clean(where):
    st, d = error()
    assert st == B.PKV_OK, f"{where}: {B.status_string(st)} at {d}"


# ---- kv_cache_write_rope -------------------------------------------------------


def rope_inputs(s: Scene, T, packed, seed, positions=200):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, s.H * s.D + 2 * s.row, generator=g).to(s.dtype)
    q, k, v = qkv.split([s.H * s.D, s.row, s.row], 1)
    dev = qkv.to(DEV)
    dq, dk, dv = dev.split([s.H * s.D, s.row, s.row], 1)
    if not packed:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    slots = torch.randperm(s.blocks * s.BS, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.2] = -1
    pos = torch.randint(0, positions, (T,), generator=g)
    return (q, k, v), (dq, dk, dv), slots, pos


def within(got, want, tol, what):
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float(((got - want).abs() - tol).max())}"


def check_rope(s, T, rot, inter, packed, seed=0, in_place=False):
    p = s.params()
    (q, k, v), (dq, dk, dv), slots, pos = rope_inputs(s, T, packed, seed)
    table = B.rope_table(200, rot, device=DEV)
    cache = s.cache.to(DEV)
    out = dq if in_place else torch.full((T, s.H * s.D), 7.0, dtype=s.dtype, device=DEV)
    B.kv_cache_write_rope(out, dq, dk, dv, cache, slots.to(DEV), pos.to(DEV), table, p,
                          interleaved=inter)
    clean("rope")
    eq, ek, ev = O.kv_cache_write_rope(q, k, v, slots, pos, table.cpu(), s.op, inter)
    kept = slots >= 0
    half = torch.finfo(s.dtype).eps / 2
    # fp32: two products and a sum of them, each off by 2^-24 of |x1| + |x2| <= 12,
    # then one rounding; fp16 below its normal range by half of 2^-24
    slop = 3 * 2.0 ** -24 * 12
    got = out.cpu().double()
    within(got[kept], eq[kept], half * eq[kept].abs() * 1.001 + slop + 2.0 ** -25, "query")
    before = q.double() if in_place else torch.full_like(got, 7.0)
    assert torch.equal(got[~kept], before[~kept])
    rows = values(cache.cpu(), s.fp8).view(2, -1, s.row)
    old = values(s.cache, s.fp8).view(2, -1, s.row)
    for half_i, want in ((0, ek), (1, ev)):
        have = rows[half_i, slots[kept]]
        if s.fp8:
            # nearest code: half a step (2^-4 of the value, or 2^-10 below 2^-6),
            # saturating; the quotient is off by fp32's errors
            e = want[kept].clamp(-448, 448)
            within(have, e, e.abs() * 2.0 ** -4 * 1.001 + 2.0 ** -10 + slop / SCALE8, "codes")
        elif half_i:
            assert torch.equal(have, want[kept])       # values: a copy
        else:
            within(have, want[kept], half * want[kept].abs() * 1.001 + slop + 2.0 ** -25, "key")
        rest = torch.ones(old.shape[1], dtype=torch.bool)
        rest[slots[kept]] = False
        assert torch.equal(rows[half_i, rest], old[half_i, rest])


@pytest.mark.parametrize("T", [1, 2, 37])
@pytest.mark.parametrize("dtype,D,BS,heads,kv_heads,rot,inter,fp8,packed", [
    (BF, 128, 16, 32, 8, 128, False, False, True),
    (FP, 128, 32, 4, 4, 64, True, False, False),
    (BF, 64, 16, 5, 1, 64, True, True, True),
    (FP, 64, 32, 6, 2, 16, False, True, True),
    (BF, 128, 16, 6, 2, 96, False, True, False),
    (FP, 128, 16, 9, 3, 48, True, False, True),
])
def test_rope_write(T, dtype, D, BS, heads, kv_heads, rot, inter, fp8, packed):
    s = Scene([64, 64], heads, kv_heads, D, BS, dtype, fp8)
    check_rope(s, T, rot, inter, packed, seed=T)


def test_rope_in_place_and_many_tokens():
    s = Scene([5000], 8, 2, 128, 16)
    check_rope(s, 500, 128, False, True, in_place=True)
    check_rope(s, 500, 64, True, False, in_place=True)
    check_rope(s, 3001, 128, False, True)


@pytest.mark.parametrize("dtype,D,heads,kv_heads,rot,inter,fp8", [
    (BF, 128, 4, 1, 128, True, False), (FP, 64, 3, 3, 32, False, False), (FP, 64, 2, 1, 64, True, True),
    (BF, 128, 2, 2, 64, False, True)])
def test_rope_bulk(dtype, D, heads, kv_heads, rot, inter, fp8):
    # more tokens than 6 per SM: the streaming form
    check_rope(Scene([1400], heads, kv_heads, D, 16, dtype, fp8), 1111, rot, inter, True)


def test_rope_without_rotation_is_the_cache_write():
    s = Scene([100], 8, 2, 128, 16)
    p = s.params()
    _, (dq, dk, dv), slots, pos = rope_inputs(s, 50, False, 3)
    a, b, out = s.cache.to(DEV), s.cache.to(DEV), torch.zeros_like(dq)
    still = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).to(DEV)
    B.kv_cache_write(dk, dv, a, slots.to(DEV), p)
    B.kv_cache_write_rope(out, dq, dk, dv, b, slots.to(DEV), torch.zeros_like(pos).to(DEV), still, p)
    clean("rope")
    assert torch.equal(a, b) and torch.equal(out.cpu()[slots >= 0], dq.cpu()[slots >= 0])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale", [0.02, 1.0, 0.37, 300.0, 2.0 ** -110, 1e-40, 1e35])
@pytest.mark.parametrize("T", [1024, 512])   # the streaming form and the other
def test_rope_codes_are_the_cache_write_s(dtype, scale, T):
    # every 16-bit value as a value row, every finite one as a key row, unrotated:
    # bit for bit the codes of the plain cache write, which divides
    s = Scene([8], 1, 1, 64, 16, dtype, fp8=True, extra_blocks=64)
    p = B.make_params(1, 1, 64, 16, dtype, 0.125, kv_cache_dtype="fp8_e4m3", k_scale=scale, v_scale=scale)
    v = (torch.arange(1024 * 64, device=DEV) - 32768).to(torch.int16).view(dtype).view(1024, 64)[:T].contiguous()
    k = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    slots = torch.randperm(s.blocks * 16, generator=s.gen)[:T].to(DEV)
    still = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).to(DEV)
    a, b = s.cache.to(DEV), s.cache.to(DEV)
    B.kv_cache_write(k, v, a, slots, p)
    B.kv_cache_write_rope(torch.zeros_like(v), v, k, v, b, slots, torch.zeros_like(slots), still, p)
    clean("rope")
    # (-0 turned by 0 is +0)
    same = (a == b) | ((a == 0x80) & (b == 0))
    assert same[0].all() and torch.equal(a[1], b[1])


@pytest.mark.parametrize("what", ["slot", "position", "negative position"])
def test_rope_bad_index(what):
    s = Scene([100], 8, 2, 128, 16)
    p = s.params()
    _, (dq, dk, dv), slots, pos = rope_inputs(s, 9, False, 3)
    slots = torch.arange(9)
    if what == "slot":
        slots[4] = s.blocks * s.BS
    else:
        pos[4] = 200 if what == "position" else -1
    cache, out = s.cache.to(DEV), torch.full_like(dq, 7.0)
    B.kv_cache_write_rope(out, dq, dk, dv, cache, slots.to(DEV), pos.to(DEV),
                          B.rope_table(200, 128, device=DEV), p)
    assert error() == (B.PKV_ERR_BOUNDS, 4)
    assert (out[4] == 7).all() and not (out[5] == 7).any()
    if what != "slot":
        assert torch.equal(cache.cpu().view(2, -1, s.row)[:, 4], s.cache.view(2, -1, s.row)[:, 4])


# ---- kv_block_bounds -----------------------------------------------------------


def check_bounds(s, new, ctx=None, nan=False):
    p = s.params()
    if nan:
        flat = s.cache.view(2, -1, s.row)
        flat[0, torch.randint(0, flat.shape[1], (20,), generator=s.gen)] = 0x7f if s.fp8 else float("nan")
    start = codes(torch.full((s.blocks, s.KVH, 2, s.D), 2.0)) if s.fp8 else \
        torch.full((s.blocks, s.KVH, 2, s.D), 7.0, dtype=s.dtype)
    got = start.to(DEV)
    want = values(start, s.fp8).clone()
    ctx_t = None if ctx is None else torch.tensor(ctx, dtype=torch.int32)
    B.kv_block_bounds(got, s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV), new, p,
                      context_lens=None if ctx is None else ctx_t.to(DEV))
    clean("bounds")
    O.kv_block_bounds(want, s.cache, s.tables, s.lens, s.op, ctx_t)
    have = values(got.cpu(), s.fp8)
    assert torch.equal(torch.isnan(have), torch.isnan(want))
    assert torch.equal(have.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("dtype,D,BS,kv_heads,fp8", [(BF, 128, 16, 8, False), (FP, 64, 32, 3, False),
                                                     (BF, 64, 16, 1, True), (FP, 128, 32, 5, True)])
def test_bounds(dtype, D, BS, kv_heads, fp8):
    lens = [0, 1, BS - 1, BS, BS + 1, 5 * BS, 77]
    mk = lambda: Scene(lens, kv_heads, kv_heads, D, BS, dtype, fp8)  # noqa: E731
    check_bounds(mk(), max(lens))                                    # whole prompts
    check_bounds(mk(), 1, [max(0, L - 1) for L in lens])             # a decode step
    check_bounds(mk(), 1, lens)                                      # nothing new
    check_bounds(mk(), BS + 2, [max(0, L - BS - 2) for L in lens])   # over a block's border
    check_bounds(mk(), max(lens), nan=True)


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (FP, False), (BF, True)])
def test_bounds_bulk(dtype, fp8):
    # tables and a bound on the new tokens wide enough for the streaming form
    s = Scene([100, 0, 37], 8, 8, 128, 16, dtype, fp8)
    s.tables = torch.cat([s.tables, torch.zeros(3, 2200, dtype=torch.int32)], 1)
    check_bounds(s, 35000)
    check_bounds(s, 35000, [90, 0, 16], nan=True)


def test_bounds_leave_unwritten_slots_out():
    s = Scene([17, 40], 2, 2, 64, 16)
    flat = s.cache.view(2, -1, 16, s.row)
    for b, L in enumerate(s.lens.tolist()):
        flat[0, int(s.tables[b, L // 16]), L % 16:] = float("nan")
    check_bounds(s, 40)


@pytest.mark.parametrize("lens,ctx,new,bad", [([20, -1], [0, 0], 99, 1), ([20, 33], [0, 0], 99, 1),
                                              ([20, 20], [-1, 0], 99, 0), ([20, 20], [0, 21], 99, 1),
                                              ([20, 20], [0, 10], 19, 0)])
def test_bounds_bad_lengths(lens, ctx, new, bad):
    s = Scene([20, 20], 2, 2, 64, 16)
    got = torch.full((s.blocks, 2, 2, 64), 7.0, dtype=BF, device=DEV)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    B.kv_block_bounds(got, s.cache.to(DEV), s.tables.to(DEV), i(lens), new, s.params(), context_lens=i(ctx))
    assert error() == (B.PKV_ERR_BOUNDS, bad)
    assert (got[s.tables[bad].long()] == 7).all() and not (got[s.tables[1 - bad].long()] == 7).any()


def test_bounds_bad_table():
    s = Scene([40, 40], 2, 2, 64, 16)
    t = s.tables.clone()
    t[1, 1] = s.blocks
    got = torch.full((s.blocks, 2, 2, 64), 7.0, dtype=BF, device=DEV)
    B.kv_block_bounds(got, s.cache.to(DEV), t.to(DEV), s.lens.to(DEV), 40, s.params())
    assert error() == (B.PKV_ERR_BOUNDS, t.shape[1] + 1)
    assert not (got[t[1, 2]] == 7).any()


# ---- paged_attn_select_blocks ---------------------------------------------------


def run_select(s, bounds, k, sink=0, recent=1, max_len=None, tables=None, query=None):
    out = torch.full((s.lens.numel(), s.KVH, k), 99, dtype=torch.int32, device=DEV)
    B.paged_attn_select_blocks(out, (s.query if query is None else query).to(DEV), bounds.to(DEV),
                               (s.tables if tables is None else tables).to(DEV), s.lens.to(DEV),
                               int(s.lens.max()) if max_len is None else max_len, s.params(),
                               num_sink=sink, num_recent=recent)
    return out


def check_select(s, bounds, k, sink=0, recent=1, **kw):
    got = run_select(s, bounds, k, sink, recent, **kw)
    clean("select")
    want = O.paged_attn_select_blocks(s.query, values(bounds, s.fp8), s.tables, s.lens, k, sink, recent, s.op)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("heads,kv_heads,D,BS,dtype,fp8,window", [
    (4, 1, 128, 16, BF, False, 0), (8, 8, 64, 32, FP, False, 0), (10, 2, 128, 16, FP, True, 0),
    (16, 2, 64, 16, BF, True, 333), (12, 1, 128, 32, BF, False, 500), (17, 1, 64, 16, FP, False, 0),
    (33, 1, 128, 16, BF, True, 0)])
def test_select(heads, kv_heads, D, BS, dtype, fp8, window):
    s = Scene([0, 1, BS, BS + 1, 9 * BS, 1000, 1777], heads, kv_heads, D, BS, dtype, fp8, window)
    b = s.random_bounds()
    check_select(s, b, 7)
    check_select(s, b, 9, sink=2, recent=3)
    check_select(s, b, 4, sink=3, recent=1)     # nothing left to choose
    check_select(s, b, 1)
    check_select(s, b, 60, sink=1, max_len=5000)
    check_select(s, b, 300)                     # all


@pytest.mark.parametrize("heads,kv_heads,D,BS,dtype,fp8", [
    (4, 4, 128, 16, BF, False), (8, 4, 64, 16, FP, False), (4, 4, 64, 32, FP, True), (8, 4, 128, 16, BF, True),
    (44, 4, 64, 16, BF, False)])
def test_select_many_pairs(heads, kv_heads, D, BS, dtype, fp8):
    # more (sequence, KV head) pairs than two per SM; one sequence to a CTA
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 700, (90,), generator=g).tolist()
    s = Scene(lens, heads, kv_heads, D, BS, dtype, fp8)
    b = s.random_bounds()
    check_select(s, b, 9, sink=1, recent=2)
    s.query.zero_()
    check_select(s, b, 5)
    t = torch.randint(-1, 2, (s.blocks, kv_heads, 1, D), generator=g) * 0.5
    t[:, :, :, 3:] = 0.0
    t = torch.cat([t, t], 2)
    s.query = torch.randint(-2, 3, s.query.shape, generator=g).to(dtype)
    check_select(s, codes(t) if fp8 else t.to(dtype), 12)


def test_select_long():
    s = Scene([40000, 39999, 123], 4, 2, 64, 16)
    check_select(s, s.random_bounds(), 100, sink=1, recent=2)
    check_select(s, s.random_bounds(), 1500)


@pytest.mark.parametrize("fp8", [False, True])
def test_select_ties(fp8):
    # scores of few different values: the lowest blocks of the border's score
    s = Scene([3000, 2999, 500, 80], 6, 2, 64, 16, fp8=fp8)
    b = torch.randint(-1, 2, (s.blocks, 2, 1, 64), generator=s.gen) * 0.5
    b[:, :, :, 2:] = 0.0
    b = torch.cat([b, b], 2)
    b = codes(b) if fp8 else b.to(s.dtype)
    s.query = torch.randint(-2, 3, s.query.shape, generator=s.gen).to(s.dtype)
    for k in (2, 17, 50, 120):
        check_select(s, b, k, sink=1)
    s.query.zero_()
    check_select(s, b, 20)


@pytest.mark.parametrize("what", ["ties", "nan"])
def test_select_border_of_more_blocks_than_keys_are_kept_for(what):
    # 12400 blocks whose scores take few values (or one of which is NaN, which
    # sends all of them through the exact scores): more than the first CTA has
    # room for in 64 bits, so they are made again for every digit
    s = Scene([198400], 1, 1, 64, 16)
    b = torch.randint(-1, 2, (s.blocks, 1, 1, 64), generator=s.gen) * 0.5
    b[:, :, :, 2:] = 0.0
    b = torch.cat([b, b], 2).to(s.dtype)
    s.query = torch.randint(1, 3, s.query.shape, generator=s.gen).to(s.dtype)
    if what == "nan":
        b[s.tables[0, 3000].long(), :, 1, 9] = float("nan")
    check_select(s, b, 40)
    check_select(s, b, 2500, sink=2)


def test_select_zeros_and_bad_entries():
    s = Scene([500], 2, 2, 64, 16)
    b = s.random_bounds()
    s.query.zero_()
    check_select(s, b, 12)
    t = s.tables.clone()
    t[0, 0] = t[0, 4] = s.blocks          # equal scores: bad ones last all the same
    got = run_select(s, b, 30, tables=t)
    assert error()[0] == B.PKV_ERR_BOUNDS
    assert got[0, 0].tolist() == [j for j in range(32) if j not in (0, 4)]
    got = run_select(s, b, 31, tables=t)
    assert error()[0] == B.PKV_ERR_BOUNDS
    assert got[0, 0].tolist() == [j for j in range(32) if j != 4]


def test_select_tells_scores_apart_that_fp32_cannot():
    # a large sum hides differences of its last place: scores 2^20 + i * 2^-12
    s = Scene([2400], 2, 2, 64, 16)
    n = 150
    b = torch.zeros(s.blocks, 2, 2, 64)
    order = torch.randperm(n, generator=s.gen)
    for j in range(n):
        b[s.tables[0, j].long(), :, :, 0] = 1024.0
        b[s.tables[0, j].long(), :, :, 1] = float(order[j]) * 2.0 ** -12
    s.query.zero_()
    q = s.query.view(2, 64)
    q[:, 0], q[:, 1] = 1024.0, 1.0
    assert torch.equal(b.to(BF).float(), b)
    check_select(s, b.to(BF), 40)
    q[:, 0] = -1024.0
    check_select(s, b.to(BF), 40)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_select_non_finite(dtype):
    s = Scene([1600, 700], 4, 2, 64, 16, dtype)
    b = s.random_bounds().float()
    at = s.tables[0].long()
    b[at[5], 0, :, 3] = float("nan")
    b[at[60], 1, 1, 7] = float("inf")
    b[at[61], 1, 0, 7] = float("-inf")
    b[at[9], 0, 0, 1], b[at[9], 0, 1, 1] = float("-inf"), float("inf")
    check_select(s, b.to(dtype), 10)
    s.query[1, 5] = float("nan")
    check_select(s, b.to(dtype), 10)


@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_select_huge_and_tiny(scale):
    # sums beyond fp32 and products below it
    s = Scene([1600], 4, 2, 64, 16)
    b = (s.random_bounds().double() * scale).to(BF)
    s.query = (s.query.double() * scale).to(BF)
    check_select(s, b, 10)


def test_select_bad_entries():
    s = Scene([500, 500], 2, 2, 64, 16)
    b = s.random_bounds()
    t = s.tables.clone()
    t[1, 3] = -1
    got = run_select(s, b, 31, tables=t)      # of 32 blocks the bad one is left
    assert error() == (B.PKV_ERR_BOUNDS, t.shape[1] + 3)
    assert got[1, 0].tolist() == [j for j in range(32) if j != 3]
    for lens, ml in (([500, -1], 500), ([500, 500], 499), ([500, 5000], 5000)):
        s.lens = torch.tensor(lens, dtype=torch.int32)
        got = run_select(s, b, 8, max_len=ml)
        st, d = error()
        assert st == B.PKV_ERR_BOUNDS and d in (0, 1)
        assert (got[1] == -1).all()


def test_select_large_offsets():
    # bounds past 2^32 bytes
    blocks, kvh = 1100000, 8
    bounds = torch.zeros(blocks, kvh, 2, 128, dtype=BF, device=DEV)
    s = Scene([640], 8, 8, 128, 16)
    s.tables = (blocks - 1 - torch.arange(40)).view(1, 40).int()
    small = Scene([640], 8, 8, 128, 16, seed=4).random_bounds()[:40]
    bounds[s.tables[0].long().to(DEV)] = small.to(DEV)
    got = run_select(s, bounds, 10)
    clean("select")
    want = O.paged_attn_select_blocks(s.query, small, torch.arange(40).view(1, 40), s.lens, 10, 0, 1, s.op)
    assert torch.equal(got.cpu(), want)


# ---- paged_attn_decode_sparse ---------------------------------------------------


def run_sparse(s, sel, tables=None, cache=None, query=None):
    q = (s.query if query is None else query).to(DEV)
    out = torch.full_like(q, float("nan"))
    B.paged_attn_decode_sparse(out, q, (s.cache if cache is None else cache).to(DEV),
                               (s.tables if tables is None else tables).to(DEV), s.lens.to(DEV),
                               sel.to(DEV), s.params())
    return out


def check_sparse(s, sel, seqs=None):
    got = run_sparse(s, sel)
    clean("sparse")
    want, spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel, s.op, seqs)
    rows = list(range(s.lens.numel())) if seqs is None else seqs
    assert torch.isfinite(got).all()
    within(got.cpu().double()[rows], want[rows], attention_tolerance(s, want, spread)[rows], "sparse")


@pytest.mark.parametrize("heads,kv_heads,D,BS,dtype,fp8,window,alibi", [
    (4, 1, 128, 16, BF, False, 0, False), (8, 8, 64, 32, FP, False, 0, True),
    (10, 2, 128, 16, FP, True, 0, False), (16, 2, 64, 16, BF, True, 100, True),
    (12, 1, 128, 32, BF, False, 70, False), (17, 1, 64, 16, FP, False, 0, False),
    (40, 1, 128, 32, BF, True, 0, False), (3, 1, 64, 32, FP, True, 0, False)])
def test_sparse(heads, kv_heads, D, BS, dtype, fp8, window, alibi):
    s = Scene([0, 1, BS - 1, BS, BS + 1, 9 * BS, 400], heads, kv_heads, D, BS, dtype, fp8, window, alibi)
    check_sparse(s, s.selection(1))
    check_sparse(s, s.selection(5))
    check_sparse(s, s.selection(11, short=True))     # rows with nothing selected
    check_sparse(s, s.selection(30))                 # every block


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_sparse_many_blocks(fp8, D):
    # long enough for the keys to be spread over CTAs
    s = Scene([9000, 8999, 40, 5000], 8, 2, D, 16, fp8=fp8)
    check_sparse(s, s.selection(300), seqs=[0, 2])


@pytest.mark.parametrize("seqs", [80, 160])
@pytest.mark.parametrize("heads,kv_heads,D,BS,dtype,fp8", [
    (4, 2, 128, 16, BF, False), (18, 2, 128, 32, FP, False), (4, 2, 64, 32, FP, False), (24, 2, 64, 16, BF, False),
    (8, 2, 128, 16, BF, True), (20, 2, 128, 16, FP, True), (12, 2, 64, 16, FP, True), (34, 2, 64, 32, BF, True)])
def test_sparse_many_pairs(heads, kv_heads, D, BS, dtype, fp8, seqs):
    # more (sequence, KV head) pairs than SMs: smaller CTAs, two parts or one
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 130, (seqs,), generator=g).tolist()
    s = Scene(lens, heads, kv_heads, D, BS, dtype, fp8, window=100)
    check_sparse(s, s.selection(6, short=True), seqs=list(range(0, seqs, 7)))


def test_sparse_of_all_blocks_is_the_decode():
    s = Scene([900, 333, 16], 8, 2, 128, 16)
    p = s.params()
    sel = s.selection(s.wide).to(DEV)
    q, cache, t, lens = s.query.to(DEV), s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.empty(max(16, B.paged_attn_decode_workspace_size(3, 900, p)), dtype=torch.uint8, device=DEV)
    B.paged_attn_decode(a, q, cache, t, lens, 900, p, ws)
    B.paged_attn_decode_sparse(b, q, cache, t, lens, sel, p)
    clean("sparse")
    # both round the same weights to bf16 and the output once: two half steps
    # of the output apart, and the weights' rounding on either side
    spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel.cpu(), s.op)[1]
    within(b.cpu().double(), a.cpu().double(), 2 * attention_tolerance(s, a.cpu().double(), spread), "decode")


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_reads_nothing_else(fp8):
    # every slot that no query may see holds NaN
    s = Scene([100, 47, 300], 4, 2, 128, 16, fp8=fp8, window=150)
    sel = s.selection(4)
    seen = torch.zeros(s.blocks * 16, 2, dtype=torch.bool)
    for b, L in enumerate(s.lens.tolist()):
        for h in range(2):
            for j in (j for c in sel[b, h].tolist() if c >= 0 for j in range(16 * c, 16 * c + 16)):
                if max(0, L - 150) <= j < L:
                    seen[int(s.tables[b, j // 16]) * 16 + j % 16, h] = True
    flat = s.cache.view(2, -1, 2, 128)
    clean_cache = s.cache.clone()
    flat[:, ~seen] = 0x7f if fp8 else float("nan")
    got = run_sparse(s, sel)
    clean("sparse")
    want, spread = O.paged_attn_decode_sparse(s.query, clean_cache, s.tables, s.lens, sel, s.op)
    s.cache = clean_cache
    within(got.cpu().double(), want, attention_tolerance(s, want, spread), "sparse")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [2, 8, 16])
@pytest.mark.parametrize("dtype,low", [(FP, 2.0 ** -10), (BF, 2.0 ** -7)])
def test_sparse_every_bit_of_a_query_counts_over_fp8(dtype, low, heads, D):
    # q = (1 + low, ..., 1, ...) against keys (c, ..., -c, ...): the ones cancel
    # and the score is that of the queries' last bits
    s = Scene([32], heads, 1, D, 16, dtype, fp8=True)
    q = torch.ones(heads, D)
    q[:, :D // 2] += low
    s.query = q.to(dtype).view(1, -1)
    assert torch.equal(s.query.float().view(heads, D), q)
    k = torch.zeros(32, D)
    k[:7, :D // 2], k[:7, D // 2:] = 448.0, -448.0
    for j in range(2):
        s.cache[0, int(s.tables[0, j])] = k[16 * j:16 * j + 16].reshape(-1).to(torch.float8_e4m3fn).view(torch.uint8)
    sel = s.selection(2)
    got = run_sparse(s, sel)
    clean("sparse")
    want, spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel, s.op)
    # products and their fp32 sums are exact here (powers of two times 7 bits);
    # the softmax's own arithmetic is fp32: 2^-16 is ample
    half, weights = torch.finfo(dtype).eps / 2, torch.finfo(FP).eps / 2
    within(got.cpu().double(), want, 1.01 * (half * want.abs() + (weights + 2.0 ** -16) * spread), "sparse")


def test_sparse_climbing_scores():
    # the running maximum moves at every block, by far more than any slack
    s = Scene([640], 2, 1, 64, 16)
    k = s.cache[0].view(-1, 16, 64)
    for j in range(40):
        k[int(s.tables[0, j])] *= 0.5 * j
    check_sparse(s, s.selection(40))


@pytest.mark.parametrize("row,bad", [([3, 3, -1, -1], 1), ([4, 2, 9, -1], 1), ([2, -1, 5, -1], 2),
                                     ([1, 2, 3, 10], 3), ([1, 2, 3, 1 << 30], 3)])
def test_sparse_bad_selection(row, bad):
    s = Scene([160, 160], 2, 1, 64, 16)     # 10 blocks each
    sel = torch.tensor([[row], [[0, 4, 9, -1]]], dtype=torch.int32)
    got = run_sparse(s, sel)
    assert error() == (B.PKV_ERR_BOUNDS, bad)
    want, spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel, s.op, [1])
    within(got.cpu().double()[1], want[1], attention_tolerance(s, want, spread)[1], "other row")


def test_sparse_bad_lengths_and_tables():
    s = Scene([160, 160], 2, 1, 64, 16)
    sel = s.selection(4)
    t = s.tables.clone()
    t[1, int(sel[1, 0, 2])] = s.blocks
    run_sparse(s, sel, tables=t)
    assert error() == (B.PKV_ERR_BOUNDS, t.shape[1] + int(sel[1, 0, 2]))
    for bad in (-3, 161):
        s.lens = torch.tensor([160, bad], dtype=torch.int32)
        got = run_sparse(s, sel)
        assert error() == (B.PKV_ERR_BOUNDS, 1)
        assert (got[1] == 0).all()


def test_sparse_large_offsets():
    # cache rows past 2^32 bytes of each half
    blocks = 140000
    cache = torch.zeros(2, blocks, 16 * 8 * 128, dtype=BF, device=DEV)
    s = Scene([320], 8, 8, 128, 16)
    big = (blocks - 1 - torch.arange(20)).view(1, 20).int()
    cache[:, big[0].long().to(DEV)] = s.cache[:, s.tables[0].long()].to(DEV)
    sel = s.selection(6)
    got = run_sparse(s, sel, tables=big, cache=cache)
    clean("sparse")
    want, spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel, s.op)
    within(got.cpu().double(), want, attention_tolerance(s, want, spread), "sparse")
    # and the write and the bounds at the same place
    p = s.params()
    slot = torch.tensor([blocks * 16 - 1])
    _, (dq, dk, dv), _, _ = rope_inputs(s, 1, False, 3)
    still = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).to(DEV)
    B.kv_cache_write_rope(torch.empty_like(dq), dq, dk, dv, cache, slot.to(DEV), torch.zeros(1, dtype=torch.int64, device=DEV), still, p)
    assert torch.equal(cache.view(2, -1, 1024)[0, -1], dk[0]) and torch.equal(cache.view(2, -1, 1024)[1, -1], dv[0])
    bounds = torch.zeros(blocks, 8, 2, 128, dtype=BF, device=DEV)
    B.kv_block_bounds(bounds, cache, big.to(DEV), s.lens.to(DEV), 320, p)
    clean("bounds")
    k = cache.view(2, blocks, 16, 8, 128)[0, big[0].long().to(DEV)]
    assert torch.equal(bounds[big[0].long().to(DEV)], torch.stack([k.amin(1), k.amax(1)], 2))


# ---- together --------------------------------------------------------------------


class Step:
    """A sequence batch that decodes token after token: the four calls on
    buffers that stay."""

    def __init__(self, lens, fp8=False, k=6, seed=0):
        s = self.s = Scene([L + 40 for L in lens], 8, 2, 128, 16, fp8=fp8, seed=seed)
        self.p, n = s.params(), len(lens)
        self.cache, self.tables = s.cache.to(DEV), s.tables.to(DEV)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.max_len = max(lens) + 40
        self.bounds = torch.zeros(s.blocks, 2, 2, 128, dtype=self.cache.dtype, device=DEV)
        self.table = B.rope_table(4096, 128, device=DEV)
        self.qkv = torch.zeros(n, (8 + 4) * 128, dtype=s.dtype, device=DEV)
        self.rot, self.out = (torch.zeros(n, 1024, dtype=s.dtype, device=DEV) for _ in range(2))
        self.sel = torch.zeros(n, 2, k, dtype=torch.int32, device=DEV)
        B.kv_block_bounds(self.bounds, self.cache, self.tables, self.lens, self.max_len, self.p)

    def __call__(self):
        q, k, v = self.qkv.split([1024, 256, 256], 1)
        ctx = self.lens.clone()
        self.lens += 1
        pos = (self.lens - 1).long()
        slots = self.tables.long().gather(1, pos[:, None] // 16)[:, 0] * 16 + pos % 16
        B.kv_cache_write_rope(self.rot, q, k, v, self.cache, slots, pos, self.table, self.p)
        B.kv_block_bounds(self.bounds, self.cache, self.tables, self.lens, 1, self.p, context_lens=ctx)
        B.paged_attn_select_blocks(self.sel, self.rot, self.bounds, self.tables, self.lens, self.max_len,
                                   self.p, num_sink=1, num_recent=2)
        B.paged_attn_decode_sparse(self.out, self.rot, self.cache, self.tables, self.lens, self.sel, self.p)


def new_tokens(step, t):
    g = torch.Generator().manual_seed(100 + t)
    step.qkv.copy_(torch.randn(step.qkv.shape, generator=g).to(step.qkv.dtype))


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_together(fp8):
    step = Step([300, 31, 95, 128], fp8)
    s = step.s
    for t in range(18):                       # over a block's border for every sequence
        new_tokens(step, t)
        step()
        clean("step")
        if t % 4:
            continue
        # each call's result from what the calls before it left
        s.cache, s.lens, s.query = step.cache.cpu(), step.lens.cpu(), step.rot.cpu()
        want = torch.zeros(step.bounds.shape, dtype=torch.float64)
        O.kv_block_bounds(want, s.cache, s.tables, s.lens, s.op)
        for b, L in enumerate(s.lens.tolist()):
            at = s.tables[b, :(L + 15) // 16].long()
            assert torch.equal(values(step.bounds.cpu(), fp8)[at], want[at])
        sel = O.paged_attn_select_blocks(s.query, want, s.tables, s.lens, 6, 1, 2, s.op)
        assert torch.equal(step.sel.cpu(), sel)
        out, spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel, s.op)
        within(step.out.cpu().double(), out, attention_tolerance(s, out, spread), "step")


def test_steps_captured_and_replayed():
    lens = [300, 31, 95, 128, 2000]
    a, b, eager = Step(lens), Step(lens, seed=5), Step(lens)
    eager_b = Step(lens, seed=5)
    graphs = []
    for st in (a, b):                         # first calls outside the capture
        keep = (st.cache.clone(), st.lens.clone(), st.bounds.clone())
        st()
        for t, k in zip((st.cache, st.lens, st.bounds), keep):
            t.copy_(k)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st()
        graphs.append(g)
    for t in range(3):
        for st, g, e in ((a, graphs[0], eager), (b, graphs[1], eager_b)):
            new_tokens(st, t)
            new_tokens(e, t)
            g.replay()
        eager()
        eager_b()
        clean("replay")
        for st, e in ((a, eager), (b, eager_b)):
            for x, y in ((st.out, e.out), (st.sel, e.sel), (st.cache, e.cache), (st.bounds, e.bounds)):
                assert torch.equal(x, y)


def test_two_streams_at_once():
    lens = [1500, 700]
    ref = [Step(lens, seed=k) for k in range(2)]
    got = [Step(lens, seed=k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for t in range(4):
        for r in ref:
            new_tokens(r, t)
            r()
    torch.cuda.synchronize()
    for t in range(4):
        for g, st in zip(got, streams):
            with torch.cuda.stream(st):
                new_tokens(g, t)
                g()
    clean("streams")
    for r, g in zip(ref, got):
        assert torch.equal(r.out, g.out) and torch.equal(r.sel, g.sel) and torch.equal(r.cache, g.cache)


def test_explicit_stream():
    s = Scene([900, 333], 8, 2, 128, 16)
    p, sel = s.params(), s.selection(20).to(DEV)
    q, cache, t, lens = s.query.to(DEV), s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    B.paged_attn_decode_sparse(a, q, cache, t, lens, sel, p)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    B.paged_attn_decode_sparse(b, q, cache, t, lens, sel, p, stream=st)
    st.synchronize()
    clean("stream")
    assert torch.equal(a, b)
    B.paged_attn_decode_sparse(b.zero_(), q, cache, t, lens, sel, p, stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(a, b)


def test_empty_batches():
    s = Scene([40], 4, 2, 64, 16)
    p, e = s.params(), dict(device=DEV)
    cache, i32 = s.cache.to(DEV), torch.zeros(0, dtype=torch.int32, **e)
    none = torch.zeros(0, 256, dtype=BF, **e)
    kv, i64 = torch.zeros(0, 128, dtype=BF, **e), torch.zeros(0, dtype=torch.int64, **e)
    t, sel = torch.zeros(0, 3, dtype=torch.int32, **e), torch.zeros(0, 2, 4, dtype=torch.int32, **e)
    bounds = s.random_bounds().to(DEV)
    B.kv_cache_write_rope(none, none, kv, kv, cache, i64, i64, B.rope_table(8, 64), p)
    B.kv_block_bounds(bounds, cache, t, i32, 5, p)
    B.paged_attn_select_blocks(sel, none, bounds, t, i32, 40, p)
    B.paged_attn_decode_sparse(none, none, cache, t, i32, sel, p)
    clean("empty")
    assert torch.equal(cache.cpu(), s.cache)


def test_repeats_bit_for_bit():
    s = Scene([9000, 40, 777], 8, 2, 128, 16)
    sel = s.selection(200)
    first = run_sparse(s, sel)
    for _ in range(3):
        assert torch.equal(run_sparse(s, sel), first)


def test_binding_refusals():
    s = Scene([40, 40], 4, 2, 64, 16)
    p, cache, q = s.params(), s.cache.to(DEV), s.query.to(DEV)
    t, lens, sel = s.tables.to(DEV), s.lens.to(DEV), s.selection(2).to(DEV)
    ok = (torch.zeros_like(q), q, cache, t, lens, sel, p)
    B.paged_attn_decode_sparse(*ok)
    for i, bad in ((0, ok[0].half()), (1, q[:1]), (2, cache[:, :, ::2]), (3, t[:1]), (4, lens.long()),
                   (5, sel[:, :1]), (5, sel.long()), (5, sel.transpose(0, 1)), (1, q.cpu())):
        with pytest.raises(ValueError):
            B.paged_attn_decode_sparse(*ok[:i], bad, *ok[i + 1:])
    with pytest.raises(B.PkvError):
        B.paged_attn_decode_sparse(*ok[:5], sel[:, :, :0].contiguous(), p)
    bounds = s.random_bounds().to(DEV)
    ok = (sel, q, bounds, t, lens, 40, p)
    for i, bad in ((2, bounds.half()), (2, bounds[:, :1]), (1, q.half()), (0, sel[:1])):
        with pytest.raises(ValueError):
            B.paged_attn_select_blocks(*ok[:i], bad, *ok[i + 1:])
    with pytest.raises(B.PkvError):
        B.paged_attn_select_blocks(*ok, num_sink=2)
    with pytest.raises(ValueError):
        B.kv_block_bounds(bounds[1:], cache, t, lens, 40, p)
    with pytest.raises(ValueError):
        B.kv_block_bounds(bounds, cache, t, lens, 40, p, context_lens=lens[:1])
    _, (dq, dk, dv), slots, pos = rope_inputs(s, 6, True, 1)
    table = B.rope_table(200, 64, device=DEV)
    ok = [torch.zeros(6, 256, dtype=BF, device=DEV), dq, dk, dv, cache, slots.to(DEV), pos.to(DEV), table, p]
    B.kv_cache_write_rope(*ok)
    for i, bad in ((0, ok[0][:5]), (1, dq.t()), (2, dk.half()), (5, ok[5].int()), (6, ok[6][:5]), (7, table.half()),
                   (3, torch.zeros(6, 130, dtype=BF, device=DEV)[:, 1:129].as_strided((6, 128), (129, 1)))):
        with pytest.raises(ValueError):
            B.kv_cache_write_rope(*ok[:i], bad, *ok[i + 1:])
    clean("refusals")

"""The sparse decode over values out of the ordinary, against the fp64 oracle:
queries that are not finite, heads of very different size in one group, keys
that are not finite, and weights whose last bits show."""
import dataclasses

import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8, Scene

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def decode(s, sel):
    p = B.make_params(s.H, s.KVH, s.D, s.BS, s.dtype, s.op.scale, None, s.window, **s._k)
    q = s.query.to(DEV)
    out = torch.full_like(q, 7.0)
    B.paged_attn_decode_sparse(out, q, s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV), sel.to(DEV), p)
    torch.cuda.synchronize()
    st, d = B.device_error()
    assert st == B.PKV_OK, f"{B.status_string(st)} at {d}"
    return out.cpu().double().view(q.shape[0], s.H, s.D)


def expected(s, sel):
    """The first four sequences' and the last one's (NaN in the rows between)."""
    n = s.lens.numel()
    want, spread = O.paged_attn_decode_sparse(s.query, s.cache, s.tables, s.lens, sel, s.op,
                                              sorted({*range(min(n, 4)), n - 1}))
    shape = (s.lens.numel(), s.H, s.D)
    return want.view(shape), spread.view(shape)


def score_error(s):
    """[seqs, H, 1]: how far a head's scores may be off, from its own largest |q|:
    fp32 sums of D products (2^-24 of each per step) and, over an fp8 cache, E4M3
    terms of the query that cut it at 2^-17 of the head's largest component."""
    q = s.query.double().view(s.lens.numel(), s.H, s.D).abs().amax(2, keepdim=True)
    k = 448 * SCALE8 if s.fp8 else s.cache[0].double().nan_to_num(0.0, 0.0, 0.0).abs().max().item()
    per = s.D * 2.0 ** -24 + (2.0 ** -17 if s.fp8 else 0.0)
    return s.op.scale * s.D * q * k * per + 64.0 * 2.0 ** -22


def near(s, got, want, spread, rows, what):
    """Half a step of the output, the weights' rounding (half a step of 16 bits at
    most) and a weight's 2 d for scores that are off by d, at the heads `rows`
    [seqs, H]."""
    half = torch.finfo(s.dtype).eps / 2
    weights = torch.finfo(FP).eps / 2 if s.fp8 else half
    tol = 1.01 * (half * want.abs() + (weights + 2 * score_error(s)) * spread) + 1e-7
    seen = torch.zeros_like(rows)
    seen[[*range(min(4, len(rows))), -1]] = True      # those that `expected` gives
    bad = ~((got - want).abs() <= tol) & (rows & seen)[:, :, None]
    assert not bad.any(), f"{what}: heads {sorted(set(bad.nonzero()[:, 1].tolist()))}"


# (heads, KV heads, head size, type, 8-bit cache): 1 .. 17 query heads to a KV head
SHAPES = [(4, 1, 128, BF, True), (8, 2, 64, FP, True), (7, 1, 64, BF, True), (16, 2, 128, FP, True),
          (12, 1, 128, BF, True), (17, 1, 64, FP, True), (4, 1, 128, BF, False), (8, 1, 64, FP, False),
          (12, 1, 64, BF, False), (17, 1, 128, FP, False)]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("heads,kv_heads,D,dtype,fp8", SHAPES)
def test_a_head_that_is_not_finite_stays_alone(heads, kv_heads, D, dtype, fp8, bad, many):
    # many: more (sequence, KV head) pairs than SMs; else parts of a cluster
    lens = [90, 0, 400, 33] + ([16] * 170 if many else [])
    s = Scene(lens, heads, kv_heads, D, 16, dtype, fp8)
    sel = s.selection(9)
    sel[3] = -1                                # nothing selected: zeros, whatever the query holds
    q = s.query.view(len(lens), heads, D)
    group = heads // kv_heads
    at = [0, group - 1] if group > 1 else [0]
    clean = s.query.clone()
    want, spread = expected(s, sel)
    hit = torch.zeros(len(lens), heads, dtype=torch.bool)
    for b in range(4):
        h = at[b % len(at)]
        q[b, h, (17 * b + 5) % D] = bad
        hit[b, h] = True
    got = decode(s, sel)
    s.query = clean
    near(s, got, want, spread, ~hit, "the other heads")
    for b, h in hit.nonzero().tolist():
        assert torch.isnan(got[b, h]).all() if b in (0, 2) else (got[b, h] == 0).all(), (b, h)


@pytest.mark.parametrize("ratio", [-6, -12, -20])
@pytest.mark.parametrize("heads,kv_heads,D,dtype,fp8", [x for x in SHAPES if x[4]])
def test_a_head_is_as_exact_beside_a_larger_one(heads, kv_heads, D, dtype, fp8, ratio):
    # the largest head of the group is 2^-ratio of the others, whose scores have
    # an ordinary size
    s = Scene([90, 500, 16], heads, kv_heads, D, 16, dtype, fp8)
    group = heads // kv_heads
    if dtype is FP:
        s.query /= 16                          # 2^20 times 4 does not fit
    up = 2.0 ** (-ratio if dtype is BF else min(-ratio, 16))
    s.op = dataclasses.replace(s.op, scale=D ** -0.5 * (16 if dtype is FP else 1))
    q = s.query.view(3, heads, D)
    big = torch.zeros(3, heads, dtype=torch.bool)
    big[:, group // 2::group] = True
    q[big] = (q[big].double() * up).to(dtype)
    assert torch.isfinite(q).all()
    sel = s.selection(20)
    got = decode(s, sel)
    want, spread = expected(s, sel)
    assert torch.isfinite(got).all()
    near(s, got, want, spread, ~big if group > 1 else big, "the smaller heads")


@pytest.mark.parametrize("power", [100, 70, -100, -60])
@pytest.mark.parametrize("heads,D,fp8", [(4, 128, True), (8, 64, True), (16, 64, True), (4, 64, False)])
def test_huge_and_tiny_queries(heads, D, fp8, power):
    s = Scene([90, 300], heads, 1, D, 16, BF, fp8)
    s.query = (s.query.double() * 2.0 ** power).to(BF)
    s.op = dataclasses.replace(s.op, scale=D ** -0.5 * 2.0 ** -power)
    sel = s.selection(20)
    got = decode(s, sel)
    want, spread = expected(s, sel)
    near(s, got, want, spread, torch.ones(2, heads, dtype=torch.bool), "all heads")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("heads,kv_heads,D,dtype,fp8", [
    (8, 2, 128, BF, True), (8, 2, 64, FP, False), (24, 2, 64, BF, True), (24, 2, 128, FP, False)])
def test_visible_keys_and_values_that_are_nan(heads, kv_heads, D, dtype, fp8, many):
    # a NaN in a key: every head of that KV head is NaN; in a value: one channel
    # is; KV head 1 has neither
    lens = [100, 100, 800, 40] + ([16] * 90 if many else [])
    s = Scene(lens, heads, kv_heads, D, 16, dtype, fp8)
    sel = s.selection(7)
    want, spread = expected(s, sel)
    nan = 0x7f if fp8 else NAN
    flat = s.cache.view(2, s.blocks, 16, kv_heads, D)
    place = lambda b, k: int(s.tables[b, int(sel[b, 0, k])])  # noqa: E731
    flat[0, place(0, 2), 3, 0, 1] = nan        # a key
    flat[1, place(1, 4), 9, 0, 5] = nan        # a value
    for k in range(7):
        flat[0, place(2, k), :, 0, 7] = nan    # every key
    flat[0, place(3, 2), 40 % 16:, 0] = nan   # keys and values past the end are not seen
    flat[1, place(3, 2), 40 % 16:, 0] = nan
    assert int(sel[3, 0, 2]) == 2
    got = decode(s, sel)
    group = heads // kv_heads
    rows = torch.ones(len(lens), heads, dtype=torch.bool)
    rows[:3, :group] = False
    near(s, got, want, spread, rows, "the rest")
    assert torch.isnan(got[[0, 2], :group]).all()
    channels = torch.isnan(got[1, :group])
    assert channels[:, 5].all() and channels.sum() == group
    got[1, :group, 5] = want[1, :group, 5]
    rows[1] = True
    near(s, got, want, spread, rows, "the other channels")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("heads,D,dtype", [(4, 64, BF), (12, 128, FP)])
def test_visible_keys_that_are_infinite(heads, D, dtype, many):
    # scores of minus infinity weigh nothing; a row that has no other is NaN, as
    # is one with a score of plus infinity
    lens = [160, 160, 700] + ([16] * 170 if many else [])
    s = Scene(lens, heads, 1, D, 16, dtype)
    s.query.view(-1, heads, D)[:, :, 2] = 1.5
    sel = s.selection(10)
    flat = s.cache.view(2, s.blocks, 16, 1, D)
    flat[0, s.tables[0, 4].long(), :, 0, 2] = -INF
    flat[0, s.tables[1, 6].long(), 2, 0, 2] = INF
    flat[0, s.tables[2].long(), :, 0, 2] = -INF
    got = decode(s, sel)
    want, spread = expected(s, sel)            # its softmax of -infinities alone is NaN too
    assert torch.isnan(got[1:3]).all() and torch.isnan(want[1:3]).all()
    rows = torch.ones(len(lens), heads, dtype=torch.bool)
    rows[1:3] = False
    near(s, got, want, spread, rows, "the rest")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("heads,D,dtype", [(4, 64, BF), (8, 128, FP), (12, 128, FP), (17, 64, BF)])
def test_visible_values_that_are_infinite(heads, D, dtype, zero, many):
    # an infinite value makes its channel infinite, two of either sign NaN, for
    # weights of 1 (zero queries) as for any other; the other channels stay
    lens = [160, 90, 16, 33] + ([16] * 170 if many else [])
    s = Scene(lens, heads, 1, D, 16, dtype)
    if zero:
        s.query.zero_()
    sel = s.selection(10)
    want, spread = expected(s, sel)
    flat = s.cache.view(2, s.blocks, 16, D)
    flat[1, s.tables[0, 4].long(), 3, 1] = INF
    flat[1, s.tables[0, 9].long(), 15, 2] = -INF
    flat[1, s.tables[0, 0].long(), 0, 5] = INF
    flat[1, s.tables[0, 7].long(), 7, 5] = -INF
    flat[1, s.tables[2, 0].long(), 15, 9] = -INF
    flat[1, s.tables[1, 5].long(), 10:, 3] = INF     # past the end: not seen
    got = decode(s, sel)
    assert (got[0, :, 1] == INF).all() and (got[0, :, 2] == -INF).all() and (got[2, :, 9] == -INF).all()
    assert torch.isnan(got[0, :, 5]).all()
    for b, d in ((0, 1), (0, 2), (0, 5), (2, 9)):
        got[b, :, d] = want[b, :, d]
    near(s, got, want, spread, torch.ones(len(lens), heads, dtype=torch.bool), "the other channels")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("heads,D,dtype,fp8", [
    (1, 64, BF, False), (8, 128, BF, False), (16, 128, BF, False), (8, 64, FP, False), (12, 64, FP, False),
    (4, 128, BF, True), (8, 64, FP, True), (16, 128, FP, True), (3, 64, FP, True), (6, 64, BF, True)])
def test_every_bit_of_a_weight_counts(heads, D, dtype, fp8, many):
    # One block: eight keys of weight 1 and value v, eight of weight w = e^q and
    # value 1.  With v = -w rounded to 16 bits the output (v + w) / (1 + w) is what
    # w has beyond those bits.  Over an fp8 cache v = -0.8125, and q such that w is
    # close to it and about half way between two 16-bit values.
    lens = [16] * (174 if many else 1)
    s = Scene(lens, heads, 1, D, 16, dtype, fp8)
    if fp8:
        grid = (-torch.linspace(0.19, 0.23, 2000)).to(dtype).unique().double()
        part = torch.exp(grid) * 2 ** 11 % 1    # of fp16's step of 2^-11
        q0 = grid[(part - 0.5).abs() < 0.15][:heads]
    else:
        q0 = (-torch.linspace(0.3, 1.9, heads)).to(dtype).double()
    assert q0.numel() == heads
    w = torch.exp(q0)
    s.query.zero_()
    s.query.view(-1, heads, D)[0, :, 0] = q0.to(dtype)
    at = s.tables[0, 0].long()
    k, v = s.cache.view(2, s.blocks, 16, D)[:, at]
    k[:], v[:] = 0, 0
    if fp8:
        code = lambda x: torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        k[8:, 0], v[:8], v[8:] = code(1.0), code(-13.0), code(16.0)
        s.op = dataclasses.replace(s.op, scale=1 / SCALE8)
        v0, v1 = torch.full_like(w, -13.0 * SCALE8), 16.0 * SCALE8
    else:
        k[8:, 0], v[8:] = 1.0, 1.0
        v0, v1 = -w.to(dtype).double(), 1.0
        v[:8, :heads] = v0.to(dtype)           # channel h: head h's
        s.op = dataclasses.replace(s.op, scale=1.0)
    got = decode(s, s.selection(1))[0].diagonal()[:heads] if not fp8 else decode(s, s.selection(1))[0, :, 0]
    want, spread = (v0 + w * v1) / (1 + w), (v0.abs() + w * v1) / (1 + w)
    # half a step of the output; of the weights 2^-16 at most (bf16: the leading 8
    # bits, which leave less than 2^-7, and 8 bits of the rest to half a step) and
    # 2^-20 for the fp32 exponential, sums and quotient
    half = torch.finfo(dtype).eps / 2
    tol = 1.01 * half * want.abs() + (2.0 ** -16 + 2.0 ** -20) * spread + 2.0 ** -26
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()
    # (what rounded weights would give is told apart)
    rounded = w.to(FP if fp8 else dtype).double()
    assert (((v0 + rounded * v1) / (1 + w) - want).abs() > 2 * tol).any()


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("heads,kv_heads,D,fp8", [(4, 1, 128, True), (3, 1, 64, True), (2, 2, 64, True), (8, 4, 128, True),
                                                  (7, 1, 64, True), (12, 1, 64, True), (4, 1, 64, False), (12, 1, 128, False)])
def test_every_bit_of_a_weight_counts_under_alibi(heads, kv_heads, D, fp8, many):
    # Zero queries: the weights are those of the distances alone, another for
    # every head.  The last keys' values nearly cancel the others' sum, so that
    # the output is small beside what the weights carry.
    lens = [32] * (174 if many else 2)
    s = Scene(lens, heads, kv_heads, D, 16, FP, fp8)
    slopes = [0.3 * 0.7 ** (h % 5) for h in range(heads)]
    s.op = dataclasses.replace(s.op, alibi_slopes=torch.tensor(slopes).tolist())
    s.query.zero_()
    group = heads // kv_heads
    v = torch.randn(32, kv_heads, D, generator=s.gen, dtype=torch.float64)
    dist = torch.arange(32, dtype=torch.float64) - 31
    w = torch.softmax(torch.tensor(s.op.alibi_slopes, dtype=torch.float64)[:, None] * dist, 1)   # [heads, 32]
    typed = lambda x: ((x / SCALE8).to(torch.float8_e4m3fn) if fp8 else x.to(FP))  # noqa: E731
    plain = lambda x: typed(x).double() * (SCALE8 if fp8 else 1.0)  # noqa: E731
    lead = w.view(kv_heads, group, 32)[:, 0]                  # each group's first head cancels
    for k in (29, 30, 31):
        v = plain(v)
        v[k] = 0
        v[k] = (-torch.einsum("hk,khd->hd", lead, v) / lead[:, k, None]).clamp(-8, 8)   # E4M3 ends at 8.96
    v = plain(v)
    flat = s.cache.view(2, s.blocks, 16, kv_heads, D)
    for j in range(2):
        t = typed(v[16 * j:16 * j + 16] + 0.0)
        flat[1, s.tables[0, j].long()] = t.view(torch.uint8) if fp8 else t
    s.slopes = s.op.alibi_slopes
    dev = torch.tensor(s.slopes, device=DEV)
    p = B.make_params(heads, kv_heads, D, 16, FP, s.op.scale, dev, 0, **s._k)
    q = s.query.to(DEV)
    out = torch.full_like(q, 7.0)
    B.paged_attn_decode_sparse(out, q, s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV), s.selection(2).to(DEV), p)
    torch.cuda.synchronize()
    assert B.device_error()[0] == B.PKV_OK
    got = out.cpu().double().view(-1, kv_heads, group, D)[0]
    wg = w.view(kv_heads, group, 32)
    want = torch.einsum("hgk,khd->hgd", wg, v)
    spread = torch.einsum("hgk,khd->hgd", wg, v.abs())
    # half a step of fp16 (2^-25 below its normal range); the weights' two terms,
    # the exponential and distances of up to 31 slopes in fp32: 2^-17 in all
    tol = 1.01 * (2.0 ** -11 * want.abs() + 2.0 ** -17 * spread) + 2.0 ** -25
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).amax((0, 2))
    if heads == group:                                        # (rounded weights are told apart)
        rounded = (w / w.amax(1, keepdim=True)).to(FP).double() * w.amax(1, keepdim=True)
        off = (torch.einsum("hgk,khd->hgd", rounded.view(kv_heads, group, 32), v) - want).abs()
        assert (off[:, 0] > 2 * tol[:, 0]).any()

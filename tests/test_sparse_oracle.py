"""The oracle of the block-sparse decode, pinned by hand-made values and by
what the definitions imply (CPU)."""
import math

import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B


def _p(**kw):
    base = dict(num_heads=4, num_kv_heads=2, head_size=64, block_size=16, scale=0.125)
    base.update(kw)
    return O.AttnParams(**base)


def test_rotation_by_hand():
    # 90 degrees turns (1, 0) into (0, 1); channels past rot_dim stay
    x = torch.zeros(1, 64, dtype=torch.float64)
    x[0, 0], x[0, 40] = 1.0, 5.0
    row = torch.cat([torch.zeros(8), torch.ones(8)])
    half = O.rope_rotate(x, row, False)
    assert half[0, 0] == 0 and half[0, 8] == 1 and half[0, 40] == 5
    inter = O.rope_rotate(x, row, True)
    assert inter[0, 0] == 0 and inter[0, 1] == 1 and inter[0, 40] == 5


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_products_of_relative_positions(interleaved):
    # (R_m q).(R_n k) depends on m - n alone
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(1, 64, generator=g, dtype=torch.float64) for _ in range(2))
    table = B.rope_table(64, 64, device="cpu").double()
    dots = [float((O.rope_rotate(q, table[m], interleaved) *
                   O.rope_rotate(k, table[m - 7], interleaved)).sum()) for m in (7, 30, 63)]
    # the table is fp32: cos and sin off by 2^-25 each at most
    assert max(dots) - min(dots) <= 8 * 2.0 ** -24 * float(q.norm() * k.norm())


def test_table_angles_of_far_positions():
    t = B.rope_table(131072, 128, base=1e6, position_scale=0.5, device="cpu")
    for pos, i in ((131071, 0), (131071, 63), (99991, 1), (5, 2)):
        a = 0.5 * pos * 1e6 ** (-2 * i / 128)
        # one rounding to fp32 of values up to 1 (half a step is 2^-25), and
        # the 64-bit angle's own error, 2^-52 of 65536
        assert abs(float(t[pos, i]) - math.cos(a)) <= 2.0 ** -25 + 2.0 ** -34
        assert abs(float(t[pos, 64 + i]) - math.sin(a)) <= 2.0 ** -25 + 2.0 ** -34
    with pytest.raises(ValueError):
        B.rope_table(8, 7, device="cpu")


def _scene(p, lens, seed=0):
    g = torch.Generator().manual_seed(seed)
    wide = max((L + p.block_size - 1) // p.block_size for L in lens)
    nb = len(lens) * wide + 1
    tables = torch.randperm(nb, generator=g)[:len(lens) * wide].view(len(lens), wide).int()
    cache = torch.randn(2, nb, p.block_size * p.row_elems, generator=g).to(torch.bfloat16)
    q = torch.randn(len(lens), p.num_heads * p.head_size, generator=g).to(torch.bfloat16)
    return cache, tables, torch.tensor(lens, dtype=torch.int32), q


def test_bounds_bound_every_product():
    p = _p()
    cache, tables, lens, q = _scene(p, [37, 16, 1])
    bounds = torch.full((cache.shape[1], 2, 2, 64), float("nan"), dtype=torch.float64)
    O.kv_block_bounds(bounds, cache, tables, lens, p)
    for b, L in enumerate(lens.tolist()):
        K, _ = O.gather_kv(cache, tables[b], L, p)
        for h in range(2):
            qh = q[b].double().view(4, 64)[2 * h:2 * h + 2]
            for j in range((L + 15) // 16):
                top = float((K[16 * j:16 * j + 16, h] @ qh.T).max())
                pb = int(tables[b, j])
                assert O.block_score(qh, bounds[pb, h, 0], bounds[pb, h, 1]) >= top - 1e-12
    # only the block of the new position changes, and only by its keys
    again = bounds.clone()
    O.kv_block_bounds(again, cache, tables, lens, p, torch.tensor([36, 16, 1]))
    assert torch.equal(again.nan_to_num(), bounds.nan_to_num())


def test_selection_orders_by_score_and_breaks_ties_low():
    p = _p(num_heads=1, num_kv_heads=1)
    q = torch.zeros(1, 64, dtype=torch.bfloat16)
    q[0, 0] = 1.0
    bounds = torch.zeros(10, 1, 2, 64)
    for j, s in enumerate([0, 3, 1, 3, 2, 3, 5, 1, 1, 9]):
        bounds[j, 0, :, 0] = s
    tables = torch.arange(10, dtype=torch.int32).view(1, 10)
    pick = lambda k, sink=0, recent=1, L=150: O.paged_attn_select_blocks(   # noqa: E731
        q, bounds, tables, torch.tensor([L]), k, sink, recent, p)[0, 0].tolist()
    assert pick(4) == [1, 3, 6, 9]          # blocks 0..9; 6, then the first of the threes
    assert pick(4, sink=1) == [0, 1, 6, 9]
    assert pick(4, recent=3) == [6, 7, 8, 9]
    assert pick(12) == list(range(10)) + [-1, -1]
    assert pick(3, L=33) == [0, 1, 2]
    bounds[2] = float("nan")
    assert pick(4) == [1, 2, 6, 9]


def test_every_block_selected_is_the_plain_decode():
    p = _p(sliding_window=40, alibi_slopes=[0.5, 0.25, 0.125, 0.0625])
    cache, tables, lens, q = _scene(p, [90, 5, 64])
    sel = torch.full((3, 2, 8), -1, dtype=torch.int32)
    for b, L in enumerate(lens.tolist()):
        n = (L + 15) // 16
        sel[b, :, :n] = torch.arange(n)
    got, _ = O.paged_attn_decode_sparse(q, cache, tables, lens, sel, p)
    assert (got - O.paged_attn_decode(q, cache, tables, lens, p)).abs().max() <= 1e-12

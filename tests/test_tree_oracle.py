"""The oracle of the speculative step over trees, pinned by hand-made values
and by what the definitions imply (CPU)."""
import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from tree_helpers import FP, TreeScene


def test_a_chain_is_the_multi_token_decode():
    s = TreeScene([20, 0, 33], [4, 4, 4], heads=4, kv_heads=2, D=64, dtype=FP, shape="chain", window=9,
                  alibi=True)
    got, _ = s.expect()
    want = O.paged_attn_decode_multi(s.query, s.cache, s.tables, s.lens, 4, s.op)
    assert (got - want).abs().max() < 1e-12


def test_a_path_of_the_tree_is_a_chain():
    # nodes 0 - 1 - 3 and 0 - 2: node 3 attends as the third token of the run 0, 1, 3
    s = TreeScene([17], [4], heads=2, kv_heads=1, D=64, dtype=FP, alibi=True, window=7)
    s.trees = [[-1, 0, 0, 1]]
    s.parents = torch.tensor([-1, 0, 0, 1], dtype=torch.int32)
    got, _ = s.expect()
    run = TreeScene([17], [3], heads=2, kv_heads=1, D=64, dtype=FP, alibi=True, window=7, shape="chain")
    run.tables, run.cache = s.tables, s.cache.clone()
    run.query = s.query[[0, 1, 3]]
    rows = run.cache.view(2, -1, run.row)
    rows[:, run.slot(0, 19)] = rows[:, s.slot(0, 20)].clone()   # node 3's row where the run's third stands
    want, _ = run.expect()
    assert (got[[0, 1, 3]] - want).abs().max() < 1e-12


def test_a_sibling_does_not_matter():
    s = TreeScene([5], [5], heads=2, kv_heads=1, D=64, dtype=FP, shape="star")
    a, _ = s.expect()
    s.cache.view(2, -1, s.row)[:, s.slot(0, 5 + 3)] = float("nan")
    b, _ = s.expect()
    keep = [0, 1, 2, 4]
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[3]).all()


def test_acceptance_by_hand():
    parents = [-1, 0, 0, 1, 1, 2, 4]
    draft = [9, 5, 6, 7, 8, 7, 3]
    target = [5, 8, 7, 1, 3, 2, 44]
    assert O.paged_attn_tree_accept(draft, target, parents, [0, 7], 5) == ([[0, 1, 4, 6, -1]], [4], [44])
    assert O.paged_attn_tree_accept(draft, target, parents, [0, 7], 2) == ([[0, 1]], [2], [8])
    target[0] = 6
    assert O.paged_attn_tree_accept(draft, target, parents, [0, 7], 5) == ([[0, 2, 5, -1, -1]], [3], [2])
    assert O.paged_attn_tree_accept(draft, target, parents, [0, 0], 2) == ([[-1, -1]], [0], [-1])


def test_commit_by_hand():
    s = TreeScene([15], [6], heads=1, kv_heads=1, D=64, dtype=FP)
    was = s.cache.clone().view(2, -1, s.row)
    O.kv_commit_tree([s.cache], torch.tensor([[0, 2, 3, 5, -1]]), s.tables, s.lens, s.cu, s.op)
    rows = s.cache.view(2, -1, s.row)
    moved = {16: 17, 17: 18, 18: 20}
    for pos in range(21):
        assert torch.equal(rows[:, s.slot(0, pos)], was[:, s.slot(0, moved.get(pos, pos))]), pos


@pytest.mark.parametrize("interleaved", [False, True])
def test_axes_that_agree_are_one(interleaved):
    g = torch.Generator().manual_seed(3)
    p = O.AttnParams(2, 1, 64, 16, 0.125)
    q, k, v = (torch.randn(5, n, generator=g).half() for n in (128, 64, 64))
    pos, slots = torch.randint(0, 50, (5,), generator=g), torch.tensor([1, 2, -1, 4, 5])
    table = B.rope_table(50, 32, device="cpu")
    a = O.kv_cache_write_rope(q, k, v, slots, pos, table, p, interleaved)
    axes = B.rope_pair_axes([4, 6, 6], woven=True)
    b = O.kv_cache_write_rope_axes(q, k, v, slots, pos.expand(3, -1), table, axes, p, interleaved)
    for x, y in zip(a, b):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))


def test_axes_by_hand():
    # pair 0 turns by axis 0 (not at all), pair 1 by axis 1 (a quarter)
    p = O.AttnParams(1, 1, 64, 16, 0.125)
    x = torch.zeros(1, 64)
    x[0, 0] = x[0, 1] = 1.0
    table = torch.tensor([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])
    q, _, _ = O.kv_cache_write_rope_axes(x, x, x, torch.tensor([0]), torch.tensor([[0], [1]]), table,
                                         [0, 1], p, False)
    assert q[0, :4].tolist() == [1.0, 0.0, 0.0, 1.0]


def test_lists_of_axes():
    assert B.rope_pair_axes([2, 1, 3]) == (0, 0, 1, 2, 2, 2)
    assert B.rope_pair_axes([4, 2, 1], woven=True) == (0, 1, 2, 0, 1, 0, 0)
    assert B.rope_pair_axes([3]) == (0, 0, 0)
    with pytest.raises(ValueError):
        B.rope_pair_axes([1] * 5)

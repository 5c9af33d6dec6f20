"""The step over trees in a cache whose offsets pass 32 bits (in elements, within
a half): the blocks in use lie at its end."""
import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from test_gpu_tree import clean, within
from tree_helpers import BF, FP, TreeScene, tolerance

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (FP, True)])
def test_blocks_beyond_32_bits(dtype, fp8):
    s = TreeScene([900, 40], [20, 9], 8, 4, 128, 16, dtype, fp8, seed=3)
    total = (1 << 32) // (16 * s.row) + 2 * s.blocks
    assert (total - s.blocks) * 16 * s.row > 1 << 32
    far = torch.empty(2, total, 16 * s.row, dtype=s.cache.dtype, device=DEV)
    if not fp8:
        s.cache.view(2, -1, s.row)[1, s.slot(0, 300), 200] = float("inf")   # a value that is looked up again
    far[:, total - s.blocks:] = s.cache.to(DEV)
    tables = (s.tables + (total - s.blocks)).to(DEV)
    p, lens, cu, up = s.params(), s.lens.to(DEV), s.cu.to(DEV), s.parents.to(DEV)

    # the write of the nodes' rows, with positions of two axes
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s.rows, n, generator=g).to(dtype) for n in (s.H * s.D, s.row, s.row))
    slots = torch.tensor([s.slot(b, s.ctx[b] + t) for b in range(2) for t in range(s.nodes[b])])
    place = torch.tensor([s.ctx[b] + d for b in range(2) for d in s.depths(b)])
    pos = torch.stack([place, place // 2])
    table, axes = B.rope_table(1000, 128, device=DEV), B.rope_pair_axes([40, 24])
    rot = torch.zeros(s.rows, s.H * s.D, dtype=dtype, device=DEV)
    args = (q.to(DEV), k.to(DEV), v.to(DEV))
    B.kv_cache_write_rope_axes(rot, *args, far, slots.to(DEV) + (total - s.blocks) * 16, pos.to(DEV), table, axes, p)
    near, rot2 = s.cache.to(DEV), torch.zeros_like(rot)
    B.kv_cache_write_rope_axes(rot2, *args, near, slots.to(DEV), pos.to(DEV), table, axes, p)
    clean("write")
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert same(far[:, total - s.blocks:].contiguous(), near) and same(rot, rot2)

    # the attention
    s.query, s.cache = rot.cpu(), near.cpu()
    out = torch.zeros_like(rot)
    ws = torch.empty(max(16, B.paged_attn_decode_tree_workspace_size(2, 20, 920, p)), dtype=torch.uint8, device=DEV)
    B.paged_attn_decode_tree(out, rot, far, tables, lens, cu, up, 20, 920, p, ws)
    clean("attention")
    want, spread = s.expect()
    within(out.cpu().double(), want, tolerance(s, want, spread), "attention")

    # the commit
    path = torch.tensor([[0, 5, 9, 19], [0, 8, -1, -1]], dtype=torch.int32)
    B.kv_commit_tree([far], path.to(DEV), tables, lens, cu, p)
    clean("commit")
    moved = [s.cache.clone()]
    O.kv_commit_tree(moved, path, s.tables, s.lens, s.cu, s.op)
    assert same(far[:, total - s.blocks:].cpu().contiguous(), moved[0])

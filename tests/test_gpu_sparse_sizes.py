"""The block-sparse decode's calls at the sizes that no other test reaches: long
selections per warp, selections wider than their sequences, host bounds far
above the lengths."""
import pytest
import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import SCALE8, Scene, codes, values

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


def clean(where):
    torch.cuda.synchronize()
    st, d = B.device_error()
    assert st == B.PKV_OK, f"{where}: {B.status_string(st)} at {d}"


# ---- host bounds far above the lengths ----------------------------------------------


@pytest.mark.parametrize("BS,fp8", [(16, False), (32, True)])
@pytest.mark.parametrize("new", [0x7fffffff, 0x7fffffff - 13, 0x7fffffff - 29, 1 << 30])
def test_bounds_with_any_bound_on_the_new_tokens(BS, fp8, new):
    s = Scene([2 * BS - 3, BS, 0], 2, 2, 64, BS, fp8=fp8)
    got = torch.zeros(s.blocks, 2, 2, 64, dtype=s.cache.dtype, device=DEV)
    B.kv_block_bounds(got, s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV), new, s.params())
    clean("bounds")
    want = torch.zeros(got.shape, dtype=torch.float64)
    O.kv_block_bounds(want, s.cache, s.tables, s.lens, s.op)
    assert torch.equal(values(got.cpu(), fp8), want)

"""What kv_cache_write_rope_axes takes as the axes of the pairs (CPU only: every
call here is refused)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_246_gb300 import binding as B


def rope(pair_axes):
    p = B.AttnParams(32, 8, 128, 16, B.PKV_BF16, 0.088, None, 0, 0, B.PKV_CACHE_AUTO, 1.0, 1.0)
    cache = torch.zeros(2, 4, 16 * 1024, dtype=torch.bfloat16)
    q, kv = torch.zeros(3, 4096, dtype=torch.bfloat16), torch.zeros(3, 1024, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    B.kv_cache_write_rope_axes(q, q, kv, kv, cache, slots, torch.zeros(3, 3, dtype=torch.int64),
                               torch.zeros(8, 128), pair_axes, p)


def test_a_number_is_not_a_list_of_axes():
    # bytes(64) would be 64 pairs of axis 0
    for bad in (64, np.int64(64), torch.tensor(64)):
        with pytest.raises(TypeError):
            rope(bad)


def test_lists_of_other_kinds_are_read_by_their_elements():
    axes = B.rope_pair_axes([16, 24, 24])
    for same in (axes, list(axes), bytes(axes), np.array(axes), np.array(axes, dtype=np.int32), torch.tensor(axes)):
        with pytest.raises(ValueError, match="CUDA device"):    # as far as the tensors' device
            rope(same)
    for bad in (np.array(axes) + 4, [-1] * 64, [300] * 64):
        with pytest.raises(ValueError):
            rope(bad)
    with pytest.raises(TypeError):
        rope([0.5] * 64)

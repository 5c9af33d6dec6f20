"""Drawn selections against scores in 64 bits: the choice is that of the exact
scores, also where many blocks score almost alike."""
import random

import pytest
import torch

from paged_kv_cache_246_gb300 import binding as B
from sparse_helpers import codes

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def plain(query, bounds, tables, lens, K, sink, recent, window, BS, KVH, D):
    """By a stable sort of the scores in doubles.  Products of two 16-bit values
    are exact in them, and their sums too unless a score's terms differ by more
    than 2^20 or so."""
    n, wide = tables.shape
    b = bounds[tables.long()].double()                       # [n, wide, KVH, 2, D]
    q = query.double().view(n, KVH, -1, D)
    lo, hi = (b[:, :, :, x].permute(0, 2, 3, 1) for x in (0, 1))
    score = (q.clamp(min=0) @ hi + q.clamp(max=0) @ lo).amax(2)
    j = torch.arange(wide, device=query.device)
    count = ((lens.long() + BS - 1) // BS)[:, None, None]
    first = (lens.long() - window).clamp(min=0)[:, None, None] // BS if window else torch.zeros_like(count)
    seen = (j >= first) & (j < count)
    always = (j < sink) | (j >= count - recent)
    score = torch.where(seen, torch.where(always, float("inf"), score), float("-inf"))
    best, at = score.sort(dim=2, descending=True, stable=True)
    at = torch.where(best[:, :, :K] > float("-inf"), at[:, :, :K], wide).sort(dim=2).values
    out = torch.full((n, KVH, K), -1, dtype=torch.int32, device=query.device)
    out[:, :, :at.shape[2]] = torch.where(at < wide, at, -1).int()
    return out


@pytest.mark.parametrize("seed", range(16))
def test_drawn_selections(seed):
    rng, g = random.Random(seed), torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *sh: torch.randn(*sh, generator=g, device=DEV)  # noqa: E731
    for i in range(400):
        KVH, D, BS = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32])
        H, dtype = KVH * rng.choice([1, 2, 4, 5, 9]), rng.choice([torch.bfloat16, torch.float16])
        fp8, window = rng.random() < 0.4, rng.choice([0, 0, 0, 777])
        top = int(2 ** rng.uniform(5, 14.5))
        n = max(1, min(rng.choice([1, 2, 5, 40]), 40000 // top))
        K = rng.randrange(4, 200)
        lens = torch.randint(1, top + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        lens[0] = top
        wide = (top + BS - 1) // BS
        tables = torch.randperm(n * wide, generator=g, device=DEV).view(n, wide).int()
        mid, half = randn(n * wide, KVH, D), torch.rand(n * wide, KVH, D, generator=g, device=DEV)
        if i % 2:                              # blocks alike in all but a few channels
            few = rng.choice([1, 2, 6])
            mid[:, :, few:], half[:, :, few:] = mid[:1, :, few:].clone(), half[:1, :, few:].clone()
            mid[:, :, :few] *= 2.0 ** rng.randrange(-12, 1)
            half[:, :, :few] *= 2.0 ** -12
        b = torch.stack([mid - half, mid + half], 2)
        bounds = codes(b) if fp8 else b.to(dtype)
        vals = bounds.view(torch.float8_e4m3fn).float() if fp8 else bounds
        query = randn(n, H * D).to(dtype)
        k = dict(kv_cache_dtype="fp8_e4m3", k_scale=0.02, v_scale=0.02) if fp8 else {}
        p = B.make_params(H, KVH, D, BS, dtype, D ** -0.5, None, window, **k)
        sink, recent = rng.randrange(0, 3), rng.randrange(1, 3)
        got = torch.full((n, KVH, K), 99, dtype=torch.int32, device=DEV)
        B.paged_attn_select_blocks(got, query, bounds, tables, lens, top, p, num_sink=sink, num_recent=recent)
        want = plain(query, vals, tables, lens, K, sink, recent, window, BS, KVH, D)
        assert torch.equal(got, want), (seed, i)
    torch.cuda.synchronize()
    assert B.device_error()[0] == B.PKV_OK

"""Scenes for the tests of the block-sparse decode: caches, tables and lengths
on the CPU, with their params on both sides."""
from __future__ import annotations

import torch

import oracle as O
from paged_kv_cache_246_gb300 import binding as B

SCALE8 = 0.02


def codes(x: torch.Tensor) -> torch.Tensor:
    return (x / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def values(t: torch.Tensor, fp8: bool) -> torch.Tensor:
    return t.view(torch.float8_e4m3fn).double() if fp8 else t.double()


class Scene:
    def __init__(self, lens, heads=8, kv_heads=2, D=128, BS=16, dtype=torch.bfloat16, fp8=False,
                 window=0, alibi=False, seed=0, extra_blocks=1):
        self.gen = torch.Generator().manual_seed(seed)
        self.H, self.KVH, self.D, self.BS, self.dtype, self.fp8 = heads, kv_heads, D, BS, dtype, fp8
        self.row = kv_heads * D
        self.lens = torch.tensor(lens, dtype=torch.int32)
        n = len(lens)
        self.wide = max(1, max((L + BS - 1) // BS for L in lens))
        self.blocks = n * self.wide + extra_blocks
        self.tables = torch.randperm(self.blocks, generator=self.gen)[:n * self.wide].view(n, -1).int()
        x = torch.randn(2, self.blocks, BS * self.row, generator=self.gen)
        self.cache = codes(x) if fp8 else x.to(dtype)
        self.query = torch.randn(n, heads * D, generator=self.gen).to(dtype)
        self.slopes = [2.0 ** -(1 + h % 7) for h in range(heads)] if alibi else None
        self.window = window
        k = dict(kv_cache_dtype="fp8_e4m3" if fp8 else "auto", k_scale=SCALE8 if fp8 else 1.0,
                 v_scale=SCALE8 if fp8 else 1.0)
        self.op = O.AttnParams(heads, kv_heads, D, BS, D ** -0.5, self.slopes, window, True, **k)
        self._k = k

    def params(self, dev="cuda:0"):
        self.dev_slopes = None if self.slopes is None else torch.tensor(self.slopes, device=dev)
        return B.make_params(self.H, self.KVH, self.D, self.BS, self.dtype, self.D ** -0.5,
                             self.dev_slopes, self.window, **self._k)

    def selection(self, k, short=False):
        """Any k of each sequence's blocks per KV head (fewer where it has fewer)."""
        out = torch.full((self.lens.numel(), self.KVH, k), -1, dtype=torch.int32)
        for b, L in enumerate(self.lens.tolist()):
            n = (L + self.BS - 1) // self.BS
            for h in range(self.KVH):
                m = min(k, n)
                if short and m:
                    m = int(torch.randint(0, m + 1, (1,), generator=self.gen))
                out[b, h, :m] = torch.randperm(n, generator=self.gen)[:m].sort().values.int()
        return out

    def random_bounds(self):
        mid = torch.randn(self.blocks, self.KVH, self.D, generator=self.gen)
        half = torch.rand(self.blocks, self.KVH, self.D, generator=self.gen)
        b = torch.stack([mid - half, mid + half], 2)
        return codes(b) if self.fp8 else b.to(self.dtype)


def attention_tolerance(s: Scene, out: torch.Tensor, spread: torch.Tensor) -> torch.Tensor:
    """How far a decode may be from (out, spread), elementwise: the output is
    rounded once (half a step of its type) and the weights once on their way
    into the product with V (to the model's type; to fp16 over an fp8 cache;
    the sum they are divided by is not rounded, so the error is half a step of
    spread); a score may be off by d, which moves a weight by 2 d of itself at
    most (its own and the sum's)."""
    half = torch.finfo(s.dtype).eps / 2
    weights = torch.finfo(torch.float16).eps / 2 if s.fp8 else half
    q = s.query.double().abs().max().item()
    k = 448 * SCALE8 if s.fp8 else s.cache[0].double().nan_to_num(0.0).abs().max().item()
    # fp32 sums of D products, and over an fp8 cache the query's E4M3 terms:
    # off by 2^-17 of the largest component
    per = s.D * 2.0 ** -24 + (2.0 ** -17 if s.fp8 else 0.0)
    d = s.D ** -0.5 * s.D * q * k * per
    # ALiBi: slope * distance in fp32, and 2^x of the special-function unit
    far = float(s.lens.max()) if s.slopes is not None else 0.0
    d += (2 * far + 64.0) * 2.0 ** -22
    return (half * 1.01) * out.abs() + (weights + 2 * d) * 1.01 * spread + 1e-7

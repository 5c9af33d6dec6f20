"""How many bits of its softmax weights paged_attn_decode_tree brings into the
product with V.  The scores are exact (one channel, whole multiples of a power
of two), half of a tile's keys have weight 1 and value 1, the others a weight w
that rounds badly in 16 bits and a value that cancels them: what is left in the
output is the error of w.  A kernel with one term fewer is off by 2 to 50 times
the tolerance, which is shown on the CPU."""
import math

import pytest
import torch

from sparse_helpers import SCALE8
from test_gpu_tree import clean
from tree_helpers import BF, FP, TreeScene

CTX, SEQS = 256, 6
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}


def fitting(dtype, fp8):
    """(query component, value, exact output, spread, output of a weight with a
    term fewer, tolerance) of the SEQS scenes that would show it most."""
    scale8 = float(torch.tensor(SCALE8)) if fp8 else 1.0
    x = torch.arange(1, 400, dtype=torch.float64) * (5.0 if fp8 else 0.0625)
    x = x[x == x.to(dtype).double()]                 # query components that the type holds
    if fp8:
        c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        c = c[(c >= 0.5) & (c <= 128)]
    else:
        c = torch.arange(64, 128).double() / 64      # seven bits: in both types
        c = torch.cat([c * 2 ** e for e in range(-1, 7)])
    # one term fewer: 16-bit caches of the model's type, fp16 over 8 bits of one fp16 term; bf16 there (a single
    # fp16 term) of one bf16 term
    fewer, held = (BF, HALF[FP]) if fp8 and dtype == BF else (dtype, HALF[dtype] ** 2)
    w = torch.exp(-x * scale8 / 8)
    n = CTX // 2
    l = n + n * w + 1                                # and the node, whose value is 0
    w, l, x = w[:, None], l[:, None], x[:, None]
    want = (n - n * w * c) / l * scale8
    spread = (n + n * w * c) / l * scale8
    short = (n - n * w.to(fewer).double() * c) / l * scale8
    # the output's rounding; the weights' terms; the scale and the exponent's product in fp32 (three roundings
    # of an exponent below 16) and 2^x of the special-function unit; sums of 257 in fp32
    per = held + (3 * 16 + 4) * 2.0 ** -24 + 257 * 2.0 ** -24
    tol = 1.01 * HALF[dtype] * want.abs() + 1.01 * per * spread + (2.0 ** -25 if dtype == FP else 0.0)
    shown = ((short - want).abs() / tol)
    at = shown.flatten().argsort(descending=True)[:SEQS]
    i, j = at // c.numel(), at % c.numel()
    return x[i, 0], c[j], want[i, j], spread[i, j], short[i, j], tol[i, j]


KINDS = [(BF, False), (FP, False), (FP, True), (BF, True)]


@pytest.mark.parametrize("dtype,fp8", KINDS)
def test_a_term_fewer_would_show(dtype, fp8):
    _, _, want, _, short, tol = fitting(dtype, fp8)
    assert ((short - want).abs() > 2 * tol).all()


def scene(dtype, fp8, D):
    x, c, want, _, _, tol = fitting(dtype, fp8)
    s = TreeScene([CTX] * SEQS, [1] * SEQS, 2, 1, D, 16, dtype, fp8, seed=1)
    rows = s.cache.view(2, -1, s.row)
    rows[:] = 0
    s.query[:] = 0.0

    def held(v):
        return int(torch.tensor(v).to(torch.float8_e4m3fn).view(torch.uint8)) if fp8 else v

    p = s.params()
    p.scale = 0.125                                  # at heads of 128 too, whose own is no power of two
    for b in range(SEQS):
        s.query[b, 0] = s.query[b, D] = x[b]
        for pos in range(CTX):
            if pos % 2:
                rows[0, s.slot(b, pos), 0] = held(-1.0)
                rows[1, s.slot(b, pos)] = held(-float(c[b]))
            else:
                rows[1, s.slot(b, pos)] = held(1.0)
    return s, p, want, tol


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fp8", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_terms_of_the_weights(dtype, fp8, D):
    s, p, want, tol = scene(dtype, fp8, D)
    got = s.decode(params=p).cpu().double()
    clean("weights")
    off = (got - want[:, None]).abs() / tol[:, None]
    assert (off <= 1).all() and math.isfinite(float(off.max())), f"{float(off.max())} of the tolerance"

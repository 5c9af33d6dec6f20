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


# ---- every place of a long selection is read, and once ----------------------------


@pytest.mark.parametrize("seqs,kv_heads,K", [(160, 2, 300), (80, 2, 230), (100, 1, 600), (40, 1, 900), (3, 1, 1100)])
@pytest.mark.parametrize("heads,D,BS,dtype,fp8", [
    (1, 128, 16, BF, False), (2, 64, 32, FP, False), (8, 128, 16, FP, True), (12, 64, 16, BF, True)])
def test_each_place_counts_once(seqs, kv_heads, K, heads, D, BS, dtype, fp8):
    # Zero queries give every key of the n selected blocks the weight 1 / n.  The
    # values of place e are 1 in channel e mod D: a place that is lost or read
    # twice moves its channel by an eighteenth or more.  The sequences' selections end
    # at every place around a warp's 32nd and 64th unit (of 3, 4 or 8 warps, one or
    # two units per block) and where the parts of a cluster meet.
    L = K * BS - 3
    s = Scene([L], heads * kv_heads, kv_heads, D, BS, dtype, fp8)
    place = torch.zeros(K, D)
    place[torch.arange(K), torch.arange(K) % D] = 1.0
    v = place.view(K, 1, 1, D).expand(K, BS, kv_heads, D).reshape(K, -1)
    s.cache[1, s.tables[0].long()] = codes(v * SCALE8) if fp8 else v.to(dtype)
    s.cache[1, s.tables[0, -1].long()].view(BS, -1)[BS - 3:] = 0x7f if fp8 else float("nan")
    marks = sorted({n for m in (32, 64, 96) for w in (1, 3, 4, 8) for x in (-1, 0, 1)
                    if 0 < (n := m * w // (BS // 16) + x) <= K} | {1, K // 2, K - 1, K})
    ends = torch.tensor([marks[-1 - i % len(marks)] for i in range(seqs)])
    sel = torch.arange(K).view(1, 1, K).expand(seqs, kv_heads, K).clone().int()
    sel[sel >= ends.view(-1, 1, 1)] = -1
    p = B.make_params(s.H, kv_heads, D, BS, dtype, 1.0, **s._k)
    q = torch.zeros(seqs, s.H * D, dtype=dtype, device=DEV)
    out = torch.full_like(q, float("nan"))
    tables = s.tables.expand(seqs, -1).contiguous().to(DEV)
    lens = torch.full((seqs,), L, dtype=torch.int32, device=DEV)
    B.paged_attn_decode_sparse(out, q, s.cache.to(DEV), tables, lens, sel.to(DEV), p)
    clean("sparse")
    keys = torch.full((K,), float(BS))
    keys[-1] = BS - 3
    cum = torch.cumsum(keys.view(-1, 1) * place, 0).double()
    want = (cum / cum.sum(1, keepdim=True))[ends - 1] * (SCALE8 if fp8 else 1.0)
    got = out.cpu().double().view(seqs, s.H, D)
    # weights are exactly 1; fp32 sums, one rounding out (fp16 below its normal
    # range by half of 2^-24)
    tol = 1.01 * (torch.finfo(dtype).eps / 2 + 2.0 ** -20) * want.abs() + 2.0 ** -25
    assert ((got - want[:, None]).abs() <= tol[:, None]).all()


# ---- selections wider than the sequences -------------------------------------------


@pytest.mark.parametrize("heads,D,fp8", [(4, 128, False), (8, 64, True)])
def test_selection_wider_than_the_sequences(heads, D, fp8):
    # tables of 32 blocks under a selection of 4096 places: the same output, and
    # the same bits, as from one of 32 places
    s = Scene([500, 512, 17, 0], heads, 2, D, 16, fp8=fp8)
    narrow = s.selection(32, short=True)
    wide = torch.full((4, 2, 4096), -1, dtype=torch.int32)
    wide[:, :, :32] = narrow
    p, q = s.params(), s.query.to(DEV)
    args = [s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV)]
    out = []
    for sel in (narrow, wide):
        out.append(torch.full_like(q, float("nan")))
        B.paged_attn_decode_sparse(out[-1], q, *args, sel.to(DEV), p)
        clean("sparse")
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("places", [40, 4096])
@pytest.mark.parametrize("at", [33, 34, 39])
def test_numbers_behind_the_end_are_reported(places, at):
    # behind the first negative number only negative ones may stand, however far
    s = Scene([512, 512], 4, 2, 64, 16)
    sel = torch.full((2, 2, places), -1, dtype=torch.int32)
    sel[:, :, :32] = torch.arange(32)
    sel[1, 0, at if places == 40 else 100 * at] = 5
    p, q = s.params(), s.query.to(DEV)
    out = torch.zeros_like(q)
    B.paged_attn_decode_sparse(out, q, s.cache.to(DEV), s.tables.to(DEV), s.lens.to(DEV), sel.to(DEV), p)
    torch.cuda.synchronize()
    assert B.device_error() == (B.PKV_ERR_BOUNDS, 2 * places + (at if places == 40 else 100 * at))


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


@pytest.mark.parametrize("max_len", [0x7fffffff, 20_000_000, 16 * B.PKV_SELECT_MAX_BLOCKS + 1])
def test_select_under_a_window_takes_any_length(max_len):
    # only the blocks inside the window are scored: the bound on the lengths does
    # not limit them
    s = Scene([1777, 900, 16], 4, 2, 64, 16, window=700)
    b = s.random_bounds()
    got = torch.full((3, 2, 12), 99, dtype=torch.int32, device=DEV)
    B.paged_attn_select_blocks(got, s.query.to(DEV), b.to(DEV), s.tables.to(DEV), s.lens.to(DEV), max_len, s.params(),
                               num_sink=1, num_recent=2)
    clean("select")
    want = O.paged_attn_select_blocks(s.query, values(b, False), s.tables, s.lens, 12, 1, 2, s.op)
    assert torch.equal(got.cpu(), want)


def test_select_far_into_a_sequence_under_a_window():
    # 640,000 tokens, 40,000 blocks: more than are scored without a window
    s = Scene([640], 4, 2, 64, 16, window=600)
    L = 640_000
    tables = torch.full((1, L // 16), -1, dtype=torch.int32)
    tables[:, -40:] = s.tables
    b = s.random_bounds()
    got = torch.full((1, 2, 9), 99, dtype=torch.int32, device=DEV)
    B.paged_attn_select_blocks(got, s.query.to(DEV), b.to(DEV), tables.to(DEV), torch.tensor([L], dtype=torch.int32, device=DEV),
                               L, s.params(), num_recent=2)
    clean("select")
    want = O.paged_attn_select_blocks(s.query, values(b, False), s.tables, s.lens, 9, 0, 2, s.op)
    assert torch.equal(got.cpu(), torch.where(want >= 0, want + L // 16 - 40, -1))


@pytest.mark.parametrize("value", [1 << 31, 1 << 32, (1 << 32) + 40, -(1 << 31) - 1])
def test_numbers_beyond_32_bits_are_refused(value):
    # not cut to 32 bits on their way into the library
    s = Scene([40, 40], 4, 2, 64, 16)
    p, t, lens = s.params(), s.tables.to(DEV), s.lens.to(DEV)
    bounds, sel = s.random_bounds().to(DEV), s.selection(2).to(DEV)
    with pytest.raises(ValueError):
        B.kv_block_bounds(bounds, s.cache.to(DEV), t, lens, value, p)
    with pytest.raises(ValueError):
        B.paged_attn_select_blocks(sel, s.query.to(DEV), bounds, t, lens, value, p)
    with pytest.raises(ValueError):
        B.paged_attn_select_blocks(sel, s.query.to(DEV), bounds, t, lens, 40, p, num_sink=value)
    with pytest.raises(ValueError):
        B.paged_attn_select_blocks(sel, s.query.to(DEV), bounds, t, lens, 40, p, num_recent=value)
    clean("refusals")


# ---- errors ---------------------------------------------------------------------------


def test_one_poll_reports_and_clears_the_errors_of_all_calls():
    s = Scene([40, 40], 4, 2, 64, 16)
    p, q, t = s.params(), s.query.to(DEV), s.tables.to(DEV)
    bounds, sel = s.random_bounds().to(DEV), s.selection(2).to(DEV)
    bad = torch.tensor([40, 4000], dtype=torch.int32, device=DEV)
    cache = s.cache.to(DEV)
    kv = torch.zeros(1, 128, dtype=BF, device=DEV)
    B.paged_attn_decode_sparse(torch.zeros_like(q), q, cache, t, bad, sel, p)
    B.kv_cache_write(kv, kv, cache, torch.full((1,), s.blocks * 16, device=DEV), p)
    B.paged_attn_select_blocks(sel, q, bounds, t, bad, 40, p)
    torch.cuda.synchronize()
    assert B.device_error() == (B.PKV_ERR_BOUNDS, 0)      # the write's token
    assert B.device_error() == (B.PKV_OK, 0)

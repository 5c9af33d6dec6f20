"""Queries that are not finite, over an fp8 cache: the dense kernels scale a tile
of queries by its largest one, and the others keep their results."""
import pytest
import torch

from gpu_helpers import CudaRun, MAX_ABS, MEAN_ABS, assert_no_device_error
from test_gpu_parity import chunked, fp8, small

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def poison(w, call, bad):
    """call's rows [tokens, heads, D] with one component `bad` in every fifth
    (token, head), beside those of the clean queries."""
    clean, hurt = CudaRun(w), CudaRun(w)
    n, H = w.query.shape[0], w.num_heads
    q = hurt.query.view(n * H, -1)
    hit = torch.zeros(n * H, dtype=torch.bool)
    hit[2::5] = True
    q[hit.to(q.device), 7] = bad
    rows = []
    for r in (clean, hurt):
        r.write()
        rows.append(call(r).cpu().double().view(n * H, -1))
    assert_no_device_error("poison")
    err = (rows[1] - rows[0])[~hit].abs()
    assert err.max() <= MAX_ABS and err.mean() <= MEAN_ABS, (err.max(), err.mean())
    return rows[1][hit]


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("H,KVH,D,dtype,multi", [
    (8, 2, 128, torch.bfloat16, 0), (3, 1, 64, torch.float16, 0), (8, 1, 64, torch.bfloat16, 0),
    (16, 1, 128, torch.float16, 0), (4, 1, 128, torch.bfloat16, 6), (32, 2, 64, torch.bfloat16, 2)])
def test_decode_rows_beside_one_that_is_not_finite(H, KVH, D, dtype, multi, bad):
    w = fp8(small(201, dtype=dtype, H=H, KVH=KVH, D=D, multi=multi, seq_lens=[9, 40, 77, 200]))
    hurt = poison(w, lambda r: r.decode_multi() if multi else r.decode(), bad)
    assert (hurt == 0).all()                   # a sum that is NaN


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("H,KVH,D,dtype,alibi", [
    (4, 2, 128, torch.bfloat16, False), (2, 1, 64, torch.float16, False), (4, 1, 64, torch.bfloat16, True)])
def test_prefill_rows_beside_one_that_is_not_finite(H, KVH, D, dtype, alibi, bad):
    w = fp8(chunked(202, [0, 31], [100, 70], dtype=dtype, H=H, KVH=KVH, D=D, alibi=alibi))
    hurt = poison(w, lambda r: r.prefill(), bad)
    assert (torch.isnan(hurt) | (hurt == 0)).all()

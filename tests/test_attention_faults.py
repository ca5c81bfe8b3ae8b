"""The attention side where it once went wrong, or could: one test for each fault.

Definitions, bounds and inputs are those of test_attention_side.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from test_attention_side import (  # noqa: E402,F401
    attend_case, attend64_long, check_attended, check_long, freqs, generator, gpu, hrb, make_batch, make_pools, shared_pages,
)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_of_an_inner_edge_tile_are_cleaned(hrb, dtype):
    """Heads of 256: infinities in the last half of a tile that is not its item's last, among keys that
    some rows see and earlier ones do not, reach none of the earlier rows."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs, new, tiles = 2 * sms, 128, 5
    lens = [128 * tiles + 64] * seqs  # rows 0..127 stand at keys 64 of tile 4 to 63 of tile 5
    batch, offsets, kp, vp, q = attend_case(hrb, 256, 64, 1, 1, [new] * seqs, lens, dtype, 31)
    cache = hrb.PagedKV(kp, vp)
    clean = cache.attend(q, batch)
    for row in (8, 40, 62):  # the token whose value is not finite
        key = 128 * (tiles - 1) + 64 + row
        pages = batch.table[:, key // 64].long()
        keep = vp[pages, key % 64].clone()
        vp[pages, key % 64, 0, ::3] = math.inf
        vp[pages, key % 64, 0, 1::3] = math.nan
        got = cache.attend(q, batch).view(seqs, new, 256)
        vp[pages, key % 64] = keep
        assert torch.equal(got[:, :row], clean.view(seqs, new, 256)[:, :row])
        assert not bool(torch.isfinite(got[:, row:, ::3]).any()) and bool(torch.isnan(got[:, row:, 1::3]).all())
        assert torch.equal(got[:, row:, 2::3], clean.view(seqs, new, 256)[:, row:, 2::3])
    assert cache.get_error() == 0


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("low", [-100.0, -120.0, -300.0])
@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("gone,length", [(1100, 2600), (2200, 2600), (33000, 34000)])
def test_low_scores_after_drains_of_minus_infinity(hrb, dtype, low, cut, gone, length):
    """Keys of -inf scores past one drain and more of the output (8 tiles for an f32 one, 256 for a
    16-bit one), then scores near `low`, in parts of whole items and in cut ones."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs = sms // 2 + 7 if cut else sms
    lens = [length + (i % 5 if cut else 0) for i in range(seqs)]
    batch, offsets, kp, vp, q = shared_pages(hrb, generator(32), seqs, 1, lens, 64, 1, 2, 64, dtype)
    q[..., 0] = q[..., 1] = 1.0
    at = torch.arange(max(lens), device="cuda")
    where = batch.table[0, at // 64].long(), at % 64
    kp[where[0], where[1], 0, 0] = torch.where(at < gone, -math.inf, 0.0).to(dtype)
    kp[where[0], where[1], 0, 1] = 8.0 * low
    check_long(hrb, batch, offsets, kp, vp, q, lens, 0.125, dtype)

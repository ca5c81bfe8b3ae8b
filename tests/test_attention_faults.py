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

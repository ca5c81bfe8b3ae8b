"""Norms, gradients and the 4-bit cache where they once went wrong, or could: a test for each fault.

Definitions, bounds and inputs are those of test_quant_cache.py.
"""
import math
import os
import re

import pytest

torch = pytest.importorskip("torch")

from test_attention_side import attend64, freqs, rotate64  # noqa: E402
from test_quant_cache import (  # noqa: E402,F401
    Cache, attended, batch_of, check_attended, encode64, gpu, hrb, norm64, reference, unpacked,
)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hadamard_rotated_binary_gb300", "csrc")


def body(text, opening):
    """The braces that follow `opening`."""
    at = text.index("{", text.index(opening))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(opening)


# ------------------------------------------------------------------ attention

# The largest value that attended() stores: 7 times scale byte 114, 10 / 16.
LARGEST = 7 * 10 / 16


def lost(lens):
    """What weights near f16's smallest step, 2^-24, lose together: they are kept relative to 2^7 or more
    for a row's largest, and each is off by half a step at most, 2^-32 of that, times the largest value.
    Elements whose loud keys all hold zeros there are so small that it shows."""
    return max(lens) * 2.0**-32 * LARGEST


def test_an_items_state_is_not_read_behind_its_last_barrier():
    """Thread 0 puts the next item's state in place of this one's as soon as it is through itself: the
    other threads' reads have to stand before the item's last barrier."""
    with open(os.path.join(CSRC, "quant_attend.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    items = body(text[text.index("bitlin_quant_attend(const __grid_constant__"):], "for (;;)")
    tail = items[items.rindex("__syncthreads();"):]
    assert "write_four" in tail  # (the rows' way out stands there)
    assert [x for x in tail.splitlines() if re.search(r"\bwork\b", x) and "threadIdx.x == 0" not in x] == []


@gpu
@pytest.mark.parametrize("dim,group,out", [(256, 6, torch.bfloat16), (128, 4, torch.float32), (64, 8, torch.float32)])
def test_ragged_items_one_after_the_other_in_a_cta(hrb, dim, group, out):
    """Thousands of items of one step, with one to three tokens each: rows go to their own places."""
    seqs = 900
    lens, new = [3 + 7 * i % 41 for i in range(seqs)], [1 + (i * i) % 3 for i in range(seqs)]
    case = (lens, new, 16, 2, group, dim, torch.bfloat16, out, True, "heads")
    cache, batch, offsets, q, y, lse = attended(hrb, case, seed=21)
    check_attended(y, lse, reference(cache, offsets, lens, q, True), torch.float16, lost(lens))
    for _ in range(10):
        again, again_lse = torch.full_like(y, 7.0), torch.full_like(lse, 7.0)
        cache.kv.attend(q, batch, out=again, lse=again_lse)
        assert torch.equal(again, y) and torch.equal(again_lse, lse)
    assert cache.kv.get_error() == hrb.BITLIN_OK


@gpu
@pytest.mark.parametrize("bad", [-1, -2, -3, 8, -2**31])
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_every_page_outside_is_reported(hrb, bad, out):
    lens, page, kvh, dim = [40, 40], 16, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = Cache(hrb, gen, lens, page, kvh, dim, torch.float16).random(gen)
    q = torch.randn((2, 8, dim), generator=gen, device="cuda").half()
    batch, offsets = batch_of(hrb, [1, 1], cache)
    cache.kv.attend(q, batch, dtype=out)
    assert cache.kv.get_error() == hrb.BITLIN_OK
    cache.table[1, 1] = bad
    y = cache.kv.attend(q, batch, dtype=out)
    assert cache.kv.get_error() == hrb.BITLIN_EINDEX and cache.kv.get_error() == hrb.BITLIN_OK
    k, v = (torch.cat([x, torch.zeros_like(x[:1])]) for x in cache.values())
    table = cache.table.cpu().clone()
    table[1, 1] = k.shape[0] - 1
    check_attended(y, None, attend64(q, k, v, offsets, lens, table, dim**-0.5, True), torch.float16)


def scratch_of(hrb, cache):
    shape = cache.parts[0].shape[:3] + (2 * cache.parts[0].shape[3],)
    return hrb.PagedKV(*(torch.full(shape, math.nan, dtype=cache.kv.dtype, device="cuda") for _ in range(2)))


@gpu
def test_a_bad_page_through_16_bit_pages_is_reported_once(hrb):
    case = ([40, 40], [30, 30], 16, 2, 4, 64, torch.float16, torch.float16, True, "heads")
    cache, batch, offsets, q, y, _ = attended(hrb, case)
    through = scratch_of(hrb, cache)
    cache.table[1, 1] = 8
    cache.kv.attend(q, batch, through=through)
    assert cache.kv.get_error() == hrb.BITLIN_EINDEX and cache.kv.get_error() == hrb.BITLIN_OK
    assert through.get_error() == hrb.BITLIN_OK
    through.attend(q, batch)
    assert through.get_error() == hrb.BITLIN_EINDEX and cache.kv.get_error() == hrb.BITLIN_OK


@gpu
def test_a_wait_that_runs_out_in_16_bit_pages_is_the_4_bit_caches_error(hrb):
    case = ([300, 20], [40, 1], 16, 2, 4, 128, torch.bfloat16, torch.bfloat16, True, "heads")
    cache, batch, offsets, q, want, _ = attended(hrb, case)
    through = scratch_of(hrb, cache)
    want = cache.kv.attend(q, batch, through=through)
    assert cache.kv.get_error() == hrb.BITLIN_OK
    through.set_wait_budget(2_000_000)
    through.test_stall(True)
    cache.kv.attend(q, batch, through=through)
    through.test_stall(False)
    assert cache.kv.get_error() == hrb.BITLIN_ETIMEOUT
    with pytest.raises(hrb.BitlinError):
        cache.kv.attend(q, batch, through=through)
    assert cache.kv.get_error() == hrb.BITLIN_ETIMEOUT
    fresh = scratch_of(hrb, cache)
    assert torch.equal(cache.kv.attend(q, batch, through=fresh), want) and cache.kv.get_error() == hrb.BITLIN_OK
    assert through.get_error() == hrb.BITLIN_ETIMEOUT


# ------------------------------------------------------------------ norms and the append


@gpu
def test_an_eps_that_f32_does_not_hold_is_refused(hrb):
    rope, w = hrb.Rope(freqs(16)), torch.ones(64, device="cuda")
    x, pos = 1e18 * torch.randn((16, 1, 64), device="cuda"), torch.arange(16, dtype=torch.int32, device="cuda")
    cache = Cache(hrb, None, [16], 16, 1, 64, torch.bfloat16)
    batch, _ = batch_of(hrb, [16], cache)
    plain = hrb.PagedKV(*(torch.zeros((1, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    for eps in (1.1e38, 1e39, 1e300):
        for call in (lambda: rope.apply(x, pos, norm=w, eps=eps), lambda: rope.gradient(x, x, pos, w, eps=eps),
                     lambda: cache.kv.append(x, x, batch, k_norm=w, eps=eps), lambda: plain.append(x, x, batch, k_norm=w, eps=eps)):
            with pytest.raises(hrb.BitlinError):
                call()
    # up to there, codes are those of the exact rows
    cache.kv.append(x, x, batch, k_norm=w, eps=1e38)
    codes, scales = encode64(norm64(x, w, 1e38))
    page = int(cache.table[0, 0])
    assert bool((scales > 0).all()) and torch.equal(cache.parts[2].cpu()[page], scales)
    assert torch.equal(unpacked(cache.parts[0].cpu()[page]), codes)


@gpu
@pytest.mark.parametrize("adjacent", [None, False, True])
def test_codes_under_weights_whose_products_pass_f32(hrb, adjacent):
    """Root times weight overflows in 32 bits where the row's values do not."""
    dim, rotary = 64, 32
    gen = torch.Generator(device="cuda").manual_seed(13)
    x = 2e-15 * torch.randn((16, 1, dim), generator=gen, device="cuda").sign()
    x[..., 48:] = torch.randint(1, 90, (16, 1, 16), generator=gen, device="cuda") * 2.0**-149
    w = torch.ones(dim, device="cuda")
    w[48:] = 1e30
    n = norm64(x, w, 0.0)
    pos = torch.randint(0, 9000, (1, 16), generator=gen, device="cuda", dtype=torch.int32)
    want = n if adjacent is None else rotate64(n, pos, freqs(rotary // 2), [0] * (rotary // 2), adjacent)
    assert float(want[..., 48:].abs().max()) < 400
    rope = None if adjacent is None else hrb.Rope(freqs(rotary // 2), adjacent=adjacent)
    cache = Cache(hrb, None, [16], 16, 1, dim, torch.bfloat16)
    batch, _ = batch_of(hrb, [16], cache)
    cache.kv.append(x, x, batch, rope=rope, pos=None if rope is None else pos, k_norm=w, eps=0.0)
    codes, scales = encode64(want)
    page = int(cache.table[0, 0])
    assert torch.equal(cache.parts[2].cpu()[page], scales)
    assert torch.equal(unpacked(cache.parts[0].cpu()[page]), codes)

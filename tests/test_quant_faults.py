"""Norms, gradients and the 4-bit cache where they once went wrong, or could: a test for each fault.

Definitions, bounds and inputs are those of test_quant_cache.py.
"""
import math
import os
import re
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from test_attention_side import attend64, freqs, rotate64  # noqa: E402
import test_quant_cache as base  # noqa: E402
from test_quant_cache import (  # noqa: E402,F401
    ATTENDED, TINY, U, Cache, attended, batch_of, check_attended, encode64, gpu, gradient64, hrb, norm64, reference, rows, unpacked, weight,
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


PROMPTS = [
    # as base.STORED: prompts of which a team takes two to four key heads, whole rows four elements at a time
    ([1000], [1000], 16, 8, 2, 256, 64, False, torch.bfloat16, torch.bfloat16, "plain", "heads", True, False),
    ([900, 131], [900, 100], 64, 5, 3, 256, 256, True, torch.float32, torch.float16, "heads", "slots", True, True),
    ([2000], [2000], 64, 7, 1, 128, 128, False, torch.bfloat16, torch.float16, "plain", "heads", True, False),
    ([1500], [1500], 48, 5, 2, 128, 40, True, torch.float16, torch.bfloat16, "heads", "heads", True, True),
    ([3000], [3000], 64, 5, 1, 64, 32, False, torch.float32, torch.bfloat16, "plain", "heads", True, False),
    ([2900, 60], [2900, 60], 7, 6, 2, 64, 64, True, torch.bfloat16, torch.float16, "plain", "slots", False, True),
    ([1300], [1300], 64, 6, 1, 128, 0, False, torch.bfloat16, torch.bfloat16, "plain", "heads", True, False),
    ([1300], [1300], 64, 6, 1, 128, 0, False, torch.float32, torch.bfloat16, "plain", "heads", False, False),
]


@gpu
@pytest.mark.parametrize("case", PROMPTS, ids=range(len(PROMPTS)))
def test_prompts_stored_several_heads_to_a_team(hrb, case):
    base.test_stored_codes_are_those_of_the_exact_rows(hrb, case)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_normed_rows_under_weights_whose_products_pass_f32(hrb, dtype):
    """Root times weight overflows in 32 bits where the row's values do not."""
    gen = torch.Generator(device="cuda").manual_seed(14)
    rope, pos, w = hrb.Rope(freqs(16)), torch.zeros((1, 16), dtype=torch.int32, device="cuda"), torch.ones(64, device="cuda")
    x = 2e-15 * torch.randn((16, 3, 64), generator=gen, device="cuda").sign()
    x[..., 48:] *= 2.0**-30
    w[48:] = 1e30
    x = x.to(dtype)
    want = norm64(x, w, 0.0)
    assert 1e20 < float(want[..., 48:].abs().min()) and float(want.abs().max()) < 1e30
    got = rope.apply(x, pos, norm=w, eps=0.0)
    # the sum's root 4.5 u and rsqrt's 4, two products 2: 11 u, and the output's rounding
    assert bool(((got.double().cpu() - want).abs() <= (11 * 2.0**-24 + 1.01 * U[dtype]) * want.abs()).all())


# ------------------------------------------------------------------ the gradient

COUNTED = [
    # tokens, heads, dim, rotary, adjacent, type of x, of dy, layout: rows enough that a team takes several, the last round not full
    (4097, 5, 256, 64, False, torch.float32, torch.float32, "plain"),
    (4001, 9, 64, 64, True, torch.bfloat16, torch.bfloat16, "heads"),
    (2601, 7, 128, 32, False, torch.float16, torch.float32, "plain"),
    (1301, 5, 80, 20, False, torch.float32, torch.bfloat16, "odd"),
    (1301, 6, 30, 10, True, torch.bfloat16, torch.float32, "plain"),
]


@gpu
@pytest.mark.parametrize("case", COUNTED, ids=range(len(COUNTED)))
def test_every_row_counts_once_in_the_gradient(hrb, case):
    """Rows of +-1 without a rotation and whole numbers as dy: the weight's gradient is a sum of whole
    numbers up to 72,000 in magnitude together, so that roundings (5 u of a term and 90 u of the sum at
    most, u = 2^-24) leave it within 1/2 of its own, and a row that is lost or counted twice does not."""
    t, h, d, rotary, adjacent, x_type, dy_type, layout = case
    gen = torch.Generator(device="cuda").manual_seed(t)
    rope = hrb.Rope(freqs(rotary // 2), adjacent=adjacent)
    sign = lambda: torch.randint(0, 2, (t, h, d), generator=gen, device="cuda") * 2.0 - 1  # noqa: E731
    x, dy = sign(), sign() * torch.randint(1, 3, (t, h, d), generator=gen, device="cuda")
    assert 95 * 2.0**-24 * 2 * t * h < 0.5
    into = rows(gen, (t, h, d), x_type, layout), rows(gen, (t, h, d), dy_type, layout)
    for to, values in zip(into, (x, dy)):
        to.copy_(values)
    w = weight(gen, d)
    dx, dw = rope.gradient(into[1], into[0], torch.zeros(t, dtype=torch.int32, device="cuda"), w, eps=0.0)
    assert torch.equal(dw.double().round(), (x.double() * dy.double()).sum((0, 1)))
    hh = dy.double() * w.double()
    ref = hh - x.double() * (hh * x.double()).mean(-1, keepdim=True)
    size = hh.abs() + (hh * x.double()).abs().mean(-1, keepdim=True)
    bound = 40 * 2.0**-24 * size
    bound = bound + U[dx.dtype] * (ref.abs() + bound) + TINY[dx.dtype]
    assert bool(((dx.double() - ref).abs() <= bound).all())


@gpu
def test_the_weights_gradient_is_as_near_as_its_sums_allow(hrb):
    """A term is off by 30 u (rotated dy 6, the root 14, products 4); it passes four fused additions in
    each of 4 rounds, 8 teams, 10 blocks and 32 rows of the join, each 1 u of the sum so far: 2^-17 of the
    sum of magnitudes holds the 96 u.  And half as many additions, errors of both signs, stay below 2^-20
    of the norm."""
    t, h, d, r = 4097, 5, 256, 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    rope, pos = hrb.Rope(freqs(r // 2)), torch.arange(t, dtype=torch.int32, device="cuda")
    x, dy, w = rows(gen, (t, h, d), torch.float32), rows(gen, (t, h, d), torch.float32, loud=False), weight(gen, d)
    _, dw = rope.gradient(dy, x, pos, w)
    _, ref, _, size = gradient64(dy, x, w, pos[None], freqs(r // 2), [0] * (r // 2), False)
    off = dw.double().cpu() - ref
    assert bool((off.abs() <= 2.0**-17 * size).all()) and float(off.norm() / ref.norm()) <= 2.0**-20


@gpu
@pytest.mark.parametrize("d,r", [(256, 64), (80, 20)])
def test_gradient_of_broadcast_rows(hrb, d, r):
    """A head that several share and a dy that all tokens share, without copies of them."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rope, w, pos = hrb.Rope(freqs(r // 2)), weight(gen, d), torch.arange(300, dtype=torch.int32, device="cuda")
    x = torch.randn((300, 1, d), generator=gen, device="cuda").expand(300, 6, d)
    dy = torch.randn((1, 6, d), generator=gen, device="cuda").expand(300, 6, d)
    for a, b in zip(rope.gradient(dy, x, pos, w), rope.gradient(dy.contiguous(), x.contiguous(), pos, w)):
        assert torch.equal(a, b)
    assert torch.equal(rope.apply(x, pos, norm=w), rope.apply(x.contiguous(), pos, norm=w))


# ------------------------------------------------------------------ forms of calls

MIXED = [
    # lens, new, page, kv_heads, group, dim, dtype, out, causal, pools
    ([300, 40, 0, 700, 1], [300, 1, 0, 1, 1], 16, 2, 6, 256, torch.bfloat16, torch.bfloat16, True, "heads"),
    ([300, 40, 0, 700, 1], [300, 1, 0, 1, 1], 16, 2, 6, 256, torch.bfloat16, torch.float32, True, "heads"),
    ([1, 0, 130, 33, 500], [1, 0, 130, 1, 3], 8, 2, 4, 128, torch.float16, torch.float16, True, "slots"),
    ([90, 33, 600, 0], [40, 1, 1, 0], 16, 1, 6, 64, torch.float16, torch.float16, True, "heads"),  # too few rows on average
    ([90, 33, 600, 20], [40, 1, 1, 0], 16, 2, 4, 128, torch.bfloat16, torch.float32, False, "heads"),
]


@gpu
@pytest.mark.parametrize("case", MIXED, ids=range(len(MIXED)))
def test_prompts_beside_single_tokens(hrb, case):
    """One prompt, single tokens and empty sequences in one call, with 16-bit pages at hand and without."""
    lens, new, dtype = case[0], case[1], case[6]
    cache, batch, offsets, q, y, lse = attended(hrb, case)
    ref = reference(cache, offsets, lens, q, case[8])
    check_attended(y, lse, ref, torch.float16, lost(lens))
    through, again = scratch_of(hrb, cache), torch.full_like(lse, 9.0)
    z = cache.kv.attend(q, batch, causal=case[8], dtype=case[7], lse=again, through=through, f32_through=True)
    check_attended(z, again, ref, dtype, lost(lens))
    assert cache.kv.get_error() == hrb.BITLIN_OK and through.get_error() == hrb.BITLIN_OK


@gpu
@pytest.mark.parametrize("case", [MIXED[0], ATTENDED[5], ATTENDED[7]], ids=range(3))
def test_queries_and_outputs_that_are_parts_of_wider_rows(hrb, case):
    """Queries out of a fused projection, an output with heads outermost, two rows of padding."""
    lens, new, page, kvh, group, dim, dtype, out, causal, pools = case
    gen = torch.Generator(device="cuda").manual_seed(8)
    cache = Cache(hrb, gen, lens, page, kvh, dim, dtype, pools, fill=255).random(gen)
    batch, offsets = batch_of(hrb, new, cache)
    tokens, heads = offsets[-1], kvh * group
    q = torch.randn((tokens + 2, heads + 2 * kvh, dim), generator=gen, device="cuda").to(dtype)[:, kvh:kvh + heads]
    room = torch.full((heads + 1, tokens + 2, dim + 8), 7.0, dtype=out, device="cuda")
    y, lse = room[1:, :, :dim].transpose(0, 1), torch.full((tokens + 2, heads), 7.0, device="cuda")
    assert cache.kv.attend(q, batch, causal=causal, out=y, lse=lse) is y
    check_attended(y[:tokens], lse[:tokens], reference(cache, offsets, lens, q[:tokens], causal), torch.float16, lost(lens))
    assert bool((y[tokens:] == 7).all()) and bool((lse[tokens:] == 7).all())
    assert bool((room[0] == 7).all()) and bool((room[..., dim:] == 7).all())


@gpu
def test_two_caches_on_two_streams_at_once(hrb):
    case = ([3000, 700, 1, 90], [1] * 4, 16, 2, 6, 256, torch.bfloat16, torch.float32, True, "heads")
    cache, batch, offsets, q, y, _ = attended(hrb, case)
    both = [cache.kv, hrb.QuantKV(*cache.parts, dtype=torch.bfloat16)]  # each with a workspace of its own
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    outs = [kv.attend(q, batch, dtype=torch.float32, stream=s) for _ in range(50) for kv, s in zip(both, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)


FIRST = r'''
import sys
import torch
import hadamard_rotated_binary_gb300 as hrb
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
T, H, KVH, D = 40, 16, 2, 128
gen = torch.Generator(device="cuda").manual_seed(4)
q, k, v = (torch.randn((T, h, D), generator=gen, device="cuda") for h in (H, KVH, KVH))
dy = torch.randn((T, H, D), generator=gen, device="cuda")
rope, pos, w = hrb.Rope([1e4 ** (-i / 16) for i in range(16)]), torch.arange(T, dtype=torch.int32, device="cuda"), torch.ones(D, device="cuda")
cache = hrb.QuantKV(*hrb.QuantKV.pools(4, 16, KVH, D))
plain = hrb.PagedKV(*(torch.zeros((4, 16, KVH, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
through = hrb.PagedKV(*(torch.zeros((4, 16, KVH, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
batch = hrb.KVBatch(i32([0, T]), i32([T]), i32([[2, 0, 3]]))
qb = q.bfloat16()

def normed():
    return [rope.apply(q, pos, norm=w), rope.apply(qb[..., ::1], pos, dtype=torch.float16, norm=w)]
def gradient():
    return list(rope.gradient(dy, q, pos, w))
def append16():
    return [plain.append(k, v, batch, rope=rope, pos=pos, q=q, q_norm=w, k_norm=w), plain.k.clone()]
def append():
    return [cache.append(k, v, batch, rope=rope, pos=pos, q=q, q_norm=w, k_norm=w), *(p.clone() for p in (cache.k, cache.v, cache.k_scale, cache.v_scale))]
def read():
    return list(cache.read(batch, T))
def attend():
    return [cache.attend(qb, batch)]
def attend_through():
    return [cache.attend(qb, batch, through=through)]

torch.cuda.synchronize()
for name in sys.argv[1:]:
    call = globals()[name]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    want = call()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    print(name, "ok")
'''


@gpu
def test_first_calls_can_be_captured(hrb):
    """Each call for the first time in its process inside a capture, with modules loaded when first used."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    calls = ["append", "read", "attend", "attend_through", "append16", "normed", "gradient"]
    done = subprocess.run([sys.executable, "-c", FIRST, *calls], cwd=root, capture_output=True, text=True, timeout=300,
                          env={**os.environ, "CUDA_MODULE_LOADING": "LAZY"})
    assert done.returncode == 0 and done.stdout.split() == [w for c in calls for w in (c, "ok")], done.stderr[-2000:]


@gpu
def test_handles_of_another_kind_are_refused(hrb):
    parts = hrb.QuantKV.pools(4, 16, 2, 64)
    pools = [torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small, plain, rope = hrb.QuantKV(*parts), hrb.PagedKV(*pools), hrb.Rope(freqs(16))
    batch = hrb.KVBatch(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [3], [[1]])))
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    for call in (lambda: hrb.QuantKV(*parts, share=plain), lambda: hrb.PagedKV(*pools, share=small), lambda: hrb.QuantKV(*parts, share=rope),
                 lambda: small.attend(q, batch, through=small), lambda: small.attend(q, batch, through=rope),
                 lambda: small.append(q[:, :2], q[:, :2], batch, rope=small), lambda: plain.append(q[:, :2], q[:, :2], batch, rope=plain)):
        with pytest.raises(ValueError):
            call()
    assert small.get_error() == hrb.BITLIN_OK and plain.get_error() == hrb.BITLIN_OK

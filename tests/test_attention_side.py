"""Rotary positions, the paged append and attention over the paged cache.

Each call is compared with the definition in 64 bits on the CPU.  The bounds are worked out from
the arithmetic, element by element (u = 2^-8 for bf16, 2^-11 for f16, the relative error of one
rounding):

  rotation   the angle is exact to 2^-33 of a turn and rounded to 24 bits, sincospi is good to two
             units in the last place, and the sum of two products rounds three times: 2^-20 of
             |a| + |b| holds all of it; then one rounding to the output's type (f16's smallest
             step, 2^-25, added).
  attention  a score is a sum of products that are exact in f32; with at most 24 partial sums
             each off by 2^-23 of the sum of magnitudes A it is off by 24 * 2^-23 * A, and its
             product with the scale, the maximum's subtraction and exp add 2^-21 * (1 + |s|).
             That is the relative error of a weight (twice: numerator and sum).  A weight's own
             rounding adds u for a 16-bit output and u^2 for a 32-bit one (two digits).  All of it
             acts on sum_j w_j |v_j|; the 2^-20 covers the f32 accumulation.  Then one rounding.
"""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

U = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0**-25}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def hrb():
    from hadamard_rotated_binary_gb300 import build as hbuild

    hbuild.build()
    import hadamard_rotated_binary_gb300 as m

    return m


gpu = pytest.mark.gpu


# ------------------------------------------------------------------ definitions in 64 bits

def rotate64(x, pos, inv_freq, axis, adjacent, sign=1.0):
    """x [T][H][D], pos [axes][T] -> the rotated rows, one pair at a time."""
    y = x.double().cpu().clone()
    r = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        t = sign * pos[axis[i]].double().cpu()[:, None] * float(torch.tensor(f, dtype=torch.float32))
        ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + r // 2)
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia] = a * torch.cos(t) - b * torch.sin(t)
        y[..., ib] = b * torch.cos(t) + a * torch.sin(t)
    return y


def pair_size(x, r, adjacent):
    """|a| + |b| of each rotated element, 0 for the others."""
    a = x.double().abs().cpu()
    out = torch.zeros_like(a)
    if adjacent:
        s = a[..., 0:r:2] + a[..., 1:r:2]
        out[..., 0:r:2] = s
        out[..., 1:r:2] = s
    else:
        s = a[..., : r // 2] + a[..., r // 2: r]
        out[..., : r // 2] = s
        out[..., r // 2: r] = s
    return out


def check_rotated(y, x, pos, inv_freq, axis, adjacent, sign=1.0):
    ref = rotate64(x, pos, inv_freq, axis, adjacent, sign)
    bound = 2.0**-20 * pair_size(x, 2 * len(inv_freq), adjacent)
    bound = bound + U[y.dtype] * (ref.abs() + bound) + TINY[y.dtype]
    assert bool(((y.double().cpu() - ref).abs() <= bound).all())


def attend64(q, k_pool, v_pool, offsets, lens, table, scale, causal):
    """(out, lse, bound factor): the last is sum_j w_j |v_j| times the weights' relative error."""
    q, k_pool, v_pool = q.double().cpu(), k_pool.double().cpu(), v_pool.double().cpu()
    table = table.cpu()
    T, H, D = q.shape
    page, kvh = k_pool.shape[1], k_pool.shape[2]
    out, lse = torch.zeros_like(q), torch.full((T, H), -math.inf, dtype=torch.float64)
    err, size = torch.zeros_like(q), torch.zeros_like(q)
    for s in range(len(lens)):
        n = lens[s]
        if n == 0:
            continue
        at = torch.arange(n)
        rows = table[s, at // page].long()
        k, v = k_pool[rows, at % page], v_pool[rows, at % page]
        for i in range(offsets[s], offsets[s + 1]):
            place = n - (offsets[s + 1] - i)
            end = min(n, place + 1) if causal else n
            if end <= 0:
                continue
            for h in range(H):
                kk, vv = k[:end, h // (H // kvh)], v[:end, h // (H // kvh)]
                logits = scale * (kk @ q[i, h])
                w = torch.softmax(logits, 0)
                out[i, h] = w @ vv
                lse[i, h] = torch.logsumexp(logits, 0)
                size[i, h] = w @ vv.abs()
                mag = abs(scale) * (kk.abs() @ q[i, h].abs())
                e = 24 * 2.0**-23 * float(mag.max()) + 2.0**-21 * (1 + float(logits.abs().max()))
                err[i, h] = 2 * e + 2.0**-20
    return out, lse, err, size


def check_attended(y, lse, ref, pool_dtype):
    out, ref_lse, err, size = ref
    u = U[pool_dtype]
    bound = size * (err + (u if y.dtype != torch.float32 else u * u))
    bound = bound + U[y.dtype] * (out.abs() + bound) + TINY[y.dtype]
    got = y.double().cpu()
    assert bool(torch.isfinite(got).all())
    worst = float(((got - out).abs() / bound.clamp(min=1e-300)).max()) if got.numel() else 0.0
    assert worst <= 1.0, worst
    if lse is not None:
        got = lse.double().cpu()
        empty = torch.isinf(ref_lse)
        assert bool((got[empty] == -math.inf).all())
        d = (got - ref_lse).abs()[~empty]
        assert bool((d <= (err[..., 0] + 2.0**-21 * ref_lse.abs())[~empty]).all())


# ------------------------------------------------------------------ inputs

def freqs(pairs, base=10000.0):
    return [base ** (-i / pairs) for i in range(pairs)]


def make_pools(gen, pages, page, kvh, dim, dtype, layout="slots", fill=None):
    if layout == "slots":
        k, v = (torch.empty((pages, page, kvh, dim), dtype=dtype, device="cuda") for _ in range(2))
    elif layout == "heads":  # [pages][heads][slots][dim] seen through a permuted view
        k, v = (torch.empty((pages, kvh, page, dim), dtype=dtype, device="cuda").permute(0, 2, 1, 3) for _ in range(2))
    else:  # keys and values of a page together
        both = torch.empty((pages, 2, page, kvh, dim), dtype=dtype, device="cuda")
        k, v = both[:, 0], both[:, 1]
    if fill is None:
        k.copy_(torch.randn(k.shape, generator=gen, device="cuda"))
        v.copy_(torch.randn(v.shape, generator=gen, device="cuda"))
    else:
        k.fill_(fill)
        v.fill_(fill)
    return k, v


def make_batch(hrb, gen, new, lens, page, spare=2, junk=0):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + 1), junk, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    offsets = [sum(new[:i]) for i in range(len(new) + 1)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return hrb.KVBatch(i32(offsets), i32(lens), table), offsets, order.numel()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def fill_past(batch, k, v, lens, value):
    """Overwrite every slot that holds no place of a sequence."""
    page = k.shape[1]
    held = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        held[batch.table[s, at // page].long(), at % page] = True
    k[~held] = value
    v[~held] = value


# ------------------------------------------------------------------ rotation

@gpu
@pytest.mark.parametrize("tokens,heads,dim,rotary,axes,adjacent", [
    (1, 24, 256, 64, 3, False),
    (7, 3, 80, 80, 3, False),
    (33, 5, 72, 72, 2, True),
    (5, 1, 10, 6, 1, False),     # sizes that no chunk fits
    (9, 2, 7, 6, 1, True),       # an odd head
    (130, 9, 128, 32, 1, True),
    (3, 17, 64, 2, 1, False),
    (11, 3, 80, 20, 3, False),   # chunks of two
    (11, 3, 80, 20, 3, True),
    (6, 2, 48, 24, 8, False),    # more axes than registers hold
])
def test_rope_against_the_definition(hrb, tokens, heads, dim, rotary, axes, adjacent):
    gen = generator(tokens * 1000 + dim)
    inv_freq = freqs(rotary // 2)
    axis = [i % axes for i in range(rotary // 2)]
    rope = hrb.Rope(inv_freq, axis, adjacent=adjacent)
    pos = torch.randint(-5, 200000, (axes, tokens), generator=gen, device="cuda", dtype=torch.int32)
    for src in DTYPES:
        x = torch.randn((tokens, heads, dim), generator=gen, device="cuda").to(src)
        for dst in DTYPES:
            check_rotated(rope.apply(x, pos, dtype=dst), x, pos, inv_freq, axis, adjacent)
        check_rotated(rope.apply(x, pos, inverse=True), x, pos, inv_freq, axis, adjacent, -1.0)


@gpu
def test_rope_at_extreme_positions_and_frequencies(hrb):
    """The angle is a wrapping product: exact at every int32 position; frequencies past one turn and negative ones too."""
    inv_freq = [1.0, -0.25, 7.5, 1e-9, 6.25, 0.0]
    rope = hrb.Rope(inv_freq)
    pos = torch.tensor([[0, 1, -1, 131071, 2**24 + 1, 2**31 - 1, -2**31]], dtype=torch.int32, device="cuda")
    x = torch.randn((pos.shape[1], 2, 12), generator=generator(3), device="cuda")
    # 64-bit reference angles are off by 2^-53 of their size: 2^34 radians at most, 2^-19 at the largest position
    ref = rotate64(x, pos, inv_freq, [0] * 6, False)
    bound = (2.0**-18) * pair_size(x, 12, False)
    assert bool(((rope.apply(x, pos).double().cpu() - ref).abs() <= bound).all())


@gpu
def test_rope_strides_in_place_and_empty(hrb):
    gen = generator(5)
    inv_freq = freqs(16)
    rope = hrb.Rope(inv_freq)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    # every other half of a wider projection (a query beside its gate), then one that is off by one element
    wide = torch.randn((6, 4, 130), generator=gen, device="cuda")
    for x in (wide[..., :64], wide[..., 1:65]):
        before = wide.clone()
        check_rotated(rope.apply(x, pos, dtype=torch.bfloat16), x, pos[None], inv_freq, [0] * 16, False)
        assert torch.equal(wide, before)
    x = torch.randn((6, 4, 64), generator=gen, device="cuda")
    ref = rope.apply(x, pos)
    assert rope.apply(x, pos, out=x) is x and torch.equal(x, ref)
    out = torch.full((6, 9, 64), 5.0, device="cuda")
    rope.apply(ref, pos, out=out[:, 2:6])
    assert bool((out[:, :2] == 5).all()) and bool((out[:, 6:] == 5).all())
    assert torch.equal(out[:, 2:6], rope.apply(ref, pos))
    assert rope.apply(x[:0], pos[:0]).shape == (0, 4, 64)


@gpu
@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_gradient(hrb, adjacent):
    """The inverse is the gradient: against the formula's (the transposed map) and against differences."""
    gen = generator(11)
    inv_freq, axis = freqs(8), [i % 2 for i in range(8)]
    rope = hrb.Rope(inv_freq, axis, adjacent=adjacent)
    pos = torch.randint(0, 5000, (2, 3), generator=gen, device="cuda", dtype=torch.int32)
    x, g = (torch.randn((3, 2, 24), generator=gen, device="cuda") for _ in range(2))
    grad = rope.apply(g, pos, inverse=True)
    xd = x.double().cpu().requires_grad_()
    y = torch.zeros_like(xd)
    r = 16
    for i, f in enumerate(inv_freq):
        t = pos[axis[i]].double().cpu()[:, None] * float(torch.tensor(f, dtype=torch.float32))
        ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + r // 2)
        a, b = xd[..., ia], xd[..., ib]
        ea, eb = torch.zeros(24, dtype=torch.float64), torch.zeros(24, dtype=torch.float64)
        ea[ia] = 1
        eb[ib] = 1
        y = y + (a * torch.cos(t) - b * torch.sin(t))[..., None] * ea + (b * torch.cos(t) + a * torch.sin(t))[..., None] * eb
    y = y + torch.cat([torch.zeros_like(xd[..., :r]), xd[..., r:]], -1)
    (y * g.double().cpu()).sum().backward()
    bound = 2.0**-20 * pair_size(g, r, adjacent) + 2.0**-24 * xd.grad.abs()
    assert bool(((grad.double().cpu() - xd.grad).abs() <= bound).all())
    # differences: the map is linear, so a step of 1 is exact up to f32 rounding of values below 8
    for e in (0, 3, 9, 20):
        step = torch.zeros_like(x)
        step[..., e] = 1.0
        d = (rope.apply(x + step, pos).double() - rope.apply(x, pos).double())
        want = (d * g.double()).sum(-1)
        assert bool(((grad[..., e].double() - want).abs() <= 24 * 2.0**-18).all())


# ------------------------------------------------------------------ append

@gpu
@pytest.mark.parametrize("dim,page,kvh,heads,rotary,layout,new,lens", [
    (256, 16, 4, 24, 64, "slots", [1, 1, 1, 1], [1, 17, 16, 500]),
    (128, 64, 2, 8, 128, "heads", [70, 0, 3], [70, 0, 131]),
    (80, 24, 3, 6, 40, "both", [25, 1], [49, 1]),
    (64, 8, 1, 1, 64, "slots", [9], [9]),
    (72, 8, 2, 2, 36, "slots", [5, 4], [5, 40]),
    (64, 16, 5, 5, 32, "slots", [1] * 40, [3 + i for i in range(40)]),
])
def test_append_against_the_definition(hrb, dim, page, kvh, heads, rotary, layout, new, lens):
    gen = generator(dim + page)
    batch, offsets, pages = make_batch(hrb, gen, new, lens, page, junk=-1)
    T = offsets[-1]
    inv_freq, axis = freqs(rotary // 2), [i % 3 for i in range(rotary // 2)]
    for src in DTYPES:
        for dst in (torch.bfloat16, torch.float16):
            for adjacent in (False, True):
                rope = hrb.Rope(inv_freq, axis, adjacent=adjacent)
                pos = torch.randint(0, 9000, (3, T), generator=gen, device="cuda", dtype=torch.int32)
                kp, vp = make_pools(gen, pages, page, kvh, dim, dst, layout)
                before_k, before_v = kp.clone(), vp.clone()
                k, v = (torch.randn((T, kvh, dim), generator=gen, device="cuda").to(src) for _ in range(2))
                q = torch.randn((T, heads, dim), generator=gen, device="cuda").to(src)
                cache = hrb.PagedKV(kp, vp)
                q_out = cache.append(k, v, batch, rope=rope, pos=pos, q=q)
                check_rotated(q_out, q, pos, inv_freq, axis, adjacent)
                assert q_out.dtype == dst
                got_k, got_v = [], []
                for s in range(len(lens)):
                    at = torch.arange(lens[s] - new[s], lens[s], device="cuda")
                    where = batch.table[s, at // page].long(), at % page
                    got_k.append(kp[where])
                    got_v.append(vp[where])
                    before_k[where], before_v[where] = got_k[-1], got_v[-1]
                check_rotated(torch.cat(got_k), k, pos, inv_freq, axis, adjacent)
                assert torch.equal(torch.cat(got_v), v.to(dst))
                assert torch.equal(before_k, kp) and torch.equal(before_v, vp)  # nothing else was touched
                assert cache.get_error() == 0


@gpu
def test_append_without_rotation_and_with_places(hrb):
    gen = generator(2)
    batch, offsets, pages = make_batch(hrb, gen, [3, 2], [20, 2], 8)
    kp, vp = make_pools(gen, pages, 8, 2, 32, torch.bfloat16)
    cache = hrb.PagedKV(kp, vp)
    k, v = (torch.randn((5, 2, 32), generator=gen, device="cuda") for _ in range(2))
    assert cache.append(k, v, batch) is None
    at = torch.tensor([17, 18, 19, 0, 1], device="cuda")
    seq = torch.tensor([0, 0, 0, 1, 1], device="cuda")
    where = batch.table[seq, at // 8].long(), at % 8
    assert torch.equal(kp[where], k.bfloat16()) and torch.equal(vp[where], v.bfloat16())
    # positions left out: the place itself
    rope = hrb.Rope(freqs(16))
    q = torch.randn((5, 4, 32), generator=gen, device="cuda")
    q_out = cache.append(k, v, batch, rope=rope, q=q)
    check_rotated(kp[where], k, at[None], freqs(16), [0] * 16, False)
    check_rotated(q_out, q, at[None], freqs(16), [0] * 16, False)


@gpu
def test_append_padding_and_bad_places(hrb):
    gen = generator(4)
    kp, vp = make_pools(gen, 4, 8, 1, 64, torch.float16)
    cache = hrb.PagedKV(kp, vp)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = (torch.randn((6, 1, 64), generator=gen, device="cuda") for _ in range(2))
    before = kp.clone(), vp.clone()
    # rows 2.. are padding; q_out of padding is left alone
    batch = hrb.KVBatch(i32([0, 2]), i32([2]), i32([[3]]))
    q_out = torch.full((6, 1, 64), 9.0, dtype=torch.float16, device="cuda")
    cache.append(k, v, batch, q=k, q_out=q_out)
    assert cache.get_error() == 0
    assert torch.equal(kp[3, :2], k[:2].half()) and torch.equal(kp[:3], before[0][:3]) and torch.equal(kp[3, 2:], before[0][3, 2:])
    assert bool((q_out[2:] == 9).all()) and torch.equal(q_out[:2], k[:2].half())
    # a page outside the pool, a negative page, a place past the table, more new rows than the sequence holds
    for lens, table in (([2], [[4]]), ([2], [[-1]]), ([9], [[0]]), ([1], [[0]])):
        kp.copy_(before[0])
        cache.append(k[:2], v[:2], hrb.KVBatch(i32([0, 2]), i32(lens), i32(table)))
        assert cache.get_error() == hrb.BITLIN_EINDEX
        assert cache.get_error() == 0
        if lens == [9]:  # the row at place 7 is in range
            assert torch.equal(kp[0, 7], k[0].half())
        if lens == [1]:  # row 0 would stand at place -1, row 1 stands at place 0
            assert torch.equal(kp[0, 0], k[1].half())
        assert torch.equal(kp[1:], before[0][1:])


# ------------------------------------------------------------------ attention

ATTEND = [
    # dim, page, kv_heads, heads, new, lens
    (256, 64, 4, 24, [1], [777]),
    (256, 16, 2, 12, [1, 1, 1, 1, 1], [1, 15, 16, 17, 300]),
    (128, 32, 2, 8, [5, 5, 5], [128, 129, 5]),
    (64, 8, 1, 1, [130], [130]),
    (64, 48, 3, 9, [3, 0, 40], [127, 0, 290]),
    (80, 24, 2, 8, [2, 33], [257, 33]),
    (8, 16, 1, 4, [6], [30]),
    (136, 128, 1, 2, [1, 7], [640, 129]),
    (128, 256, 1, 128, [1, 2], [300, 2]),   # one key head under 128 query heads
    (256, 8, 1, 7, [20], [150]),
    (192, 16, 2, 2, [150], [400]),
    (64, 16, 8, 8, [1] * 33, [7 * i for i in range(33)]),
]


def attend_case(hrb, dim, page, kvh, heads, new, lens, dtype, seed, layout="slots", q_scale=1.0, junk=-1):
    gen = generator(seed)
    batch, offsets, pages = make_batch(hrb, gen, new, lens, page, junk=junk)
    kp, vp = make_pools(gen, pages, page, kvh, dim, dtype, layout)
    q = (torch.randn((offsets[-1], heads, dim), generator=gen, device="cuda") * q_scale).to(dtype)
    return batch, offsets, kp, vp, q


@gpu
@pytest.mark.parametrize("dim,page,kvh,heads,new,lens", ATTEND)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_against_the_definition(hrb, dim, page, kvh, heads, new, lens, dtype, causal):
    batch, offsets, kp, vp, q = attend_case(hrb, dim, page, kvh, heads, new, lens, dtype, dim + heads, q_scale=2.0)
    # what no place holds must not count, whatever it is
    fill_past(batch, kp, vp, lens, math.nan)
    cache = hrb.PagedKV(kp, vp)
    scale = 1.0 / math.sqrt(dim)
    ref = attend64(q, kp, vp, offsets, lens, batch.table, scale, causal)
    for out_dtype in (dtype, torch.float32):
        lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
        out = cache.attend(q, batch, causal=causal, dtype=out_dtype, lse=lse)
        assert out.dtype == out_dtype and cache.get_error() == 0
        check_attended(out, lse, ref, dtype)
        again = cache.attend(q, batch, causal=causal, dtype=out_dtype)
        assert torch.equal(out, again)  # no order that changes


@gpu
@pytest.mark.parametrize("layout", ["heads", "both"])
def test_attend_page_layouts(hrb, layout):
    batch, offsets, kp, vp, q = attend_case(hrb, 128, 16, 2, 6, [3, 1], [200, 33], torch.bfloat16, 8, layout=layout)
    ref = attend64(q, kp, vp, offsets, [200, 33], batch.table, 0.1, True)
    check_attended(hrb.PagedKV(kp, vp).attend(q, batch, scale=0.1), None, ref, torch.bfloat16)


@gpu
def test_attend_rows_without_keys(hrb):
    """More new rows than the sequence holds: the first ones stand before its start and see nothing."""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 1, 2, [150, 4, 2], [20, 0, 2], torch.bfloat16, 9)
    cache = hrb.PagedKV(kp, vp)
    for causal in (True, False):
        ref = attend64(q, kp, vp, offsets, [20, 0, 2], batch.table, 0.125, causal)
        lse = torch.zeros((q.shape[0], 2), device="cuda")
        out = cache.attend(q, batch, causal=causal, lse=lse)
        check_attended(out, lse, ref, torch.bfloat16)
        empty = torch.arange(156, device="cuda") < 130 if causal else torch.zeros(156, dtype=torch.bool, device="cuda")
        empty[150:154] = True
        assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())


@gpu
def test_attend_padding_rows_are_left_alone(hrb):
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 2, 4, [3, 2], [50, 9], torch.float16, 10)
    more = torch.cat([q, torch.full((4, 4, 64), math.nan, dtype=q.dtype, device="cuda")])
    out = torch.full(more.shape, 3.0, dtype=q.dtype, device="cuda")
    lse = torch.full(more.shape[:2], 3.0, device="cuda")
    cache = hrb.PagedKV(kp, vp)
    cache.attend(more, batch, out=out, lse=lse)
    assert bool((out[5:] == 3).all()) and bool((lse[5:] == 3).all())
    assert torch.equal(out[:5], cache.attend(q, batch))


@gpu
def test_attend_strided_rows(hrb):
    """A query inside a wider projection, and an output inside a wider buffer."""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 2, 6, [9], [70], torch.bfloat16, 12)
    cache = hrb.PagedKV(kp, vp)
    wide = torch.zeros((9, 6, 2, 64), dtype=q.dtype, device="cuda")
    wide[:, :, 0] = q
    buf = torch.full((9, 8, 72), 2.0, device="cuda")
    got = cache.attend(wide[:, :, 0], batch, out=buf[:, 1:7, :64])
    assert torch.equal(got, cache.attend(q, batch, dtype=torch.float32))
    assert bool((buf[:, 0] == 2).all()) and bool((buf[:, 7] == 2).all()) and bool((buf[..., 64:] == 2).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_scores_of_every_size(hrb, dtype):
    """Scores from flat to one key taking all, rising and falling along the keys."""
    gen = generator(14)
    lens = [700, 700, 700]
    batch, offsets, kp, vp, q = attend_case(hrb, 128, 64, 1, 2, [2, 2, 2], lens, dtype, 14)
    ramp = torch.linspace(0, 1, 700, device="cuda")
    for s in range(3):
        at = torch.arange(700, device="cuda")
        where = batch.table[s, at // 64].long(), at % 64
        r = ramp if s == 0 else ramp.flip(0) if s == 1 else torch.zeros_like(ramp)
        base = torch.ones(128, device="cuda")
        kp[where] = (r[:, None, None] * 40 * base).to(dtype)
    q[:] = (torch.rand(q.shape, generator=gen, device="cuda") * 0.2 + 0.9).to(dtype)
    cache = hrb.PagedKV(kp, vp)
    for scale in (0.0, 0.02, 0.3, -0.3):
        ref = attend64(q, kp, vp, offsets, lens, batch.table, scale, True)
        lse = torch.empty(q.shape[:2], device="cuda")
        for out_dtype in (dtype, torch.float32):
            check_attended(cache.attend(q, batch, scale=scale, dtype=out_dtype, lse=lse), lse, ref, dtype)


@gpu
def test_attend_infinite_scores_and_values(hrb):
    """A key of -inf scores weighs nothing; a NaN or an infinite value reaches the rows that see it."""
    lens = [200]
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 1, 1, [1], lens, torch.bfloat16, 15)
    q.fill_(1.0)
    at = torch.arange(200, device="cuda")
    where = batch.table[0, at // 16].long(), at % 16
    k, v = kp[where].clone(), vp[where].clone()
    k[150] = -math.inf
    k[3] = -math.inf
    kp[where] = k
    cache = hrb.PagedKV(kp, vp)
    keep = [i for i in range(200) if i not in (3, 150)]
    got = cache.attend(q, batch, dtype=torch.float32)
    w = torch.softmax((k[keep, 0].double() @ q[0, 0].double()) / 8, 0)
    want = w @ v[keep, 0].double()
    assert bool(((got[0, 0].double() - want).abs() <= 1e-4 * (w @ v[keep, 0].double().abs())).all())
    k[150] = math.nan
    kp[where] = k
    assert bool(torch.isnan(cache.attend(q, batch, dtype=torch.float32)).all())
    k[150] = 0.0
    v[150, 0, 5] = math.inf
    v[150, 0, 6] = math.nan
    kp[where], vp[where] = k, v
    got = cache.attend(q, batch, dtype=torch.float32)[0, 0]
    assert bool(torch.isnan(got[6])) and not bool(torch.isfinite(got[5])) and bool(torch.isfinite(got[:5]).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_later_tokens_do_not_reach_earlier_rows(hrb, dtype):
    """An infinity or a NaN in a token's key or value reaches that token's rows and the later ones alone."""
    lens, new = [300], [90]
    batch, offsets, kp, vp, q = attend_case(hrb, 128, 16, 1, 2, new, lens, dtype, 21)
    cache = hrb.PagedKV(kp, vp)
    place = 240  # token row 30
    where = int(batch.table[0, place // 16]), place % 16
    value, key = vp[where[0], where[1], 0].clone(), kp[where[0], where[1], 0].clone()
    for out_dtype in (dtype, torch.float32):
        vp[where[0], where[1], 0], kp[where[0], where[1], 0] = value, key
        clean = cache.attend(q, batch, dtype=out_dtype)
        vp[where[0], where[1], 0, 3] = math.inf
        vp[where[0], where[1], 0, 77] = math.nan
        got = cache.attend(q, batch, dtype=out_dtype)
        assert torch.equal(got[:30], clean[:30])
        assert bool(torch.isnan(got[30:, :, 77]).all())
        # two digits of a weight may multiply an infinity with opposite signs: not a number then
        assert not bool(torch.isfinite(got[30:, :, 3]).any())
        assert out_dtype == torch.float32 or bool((got[30:, :, 3] == math.inf).all())
        rest = [d for d in range(128) if d not in (3, 77)]
        assert torch.equal(got[30:][..., rest], clean[30:][..., rest])
        kp[where[0], where[1], 0, 9] = math.nan
        got = cache.attend(q, batch, dtype=out_dtype)
        assert torch.equal(got[:30], clean[:30]) and bool(torch.isnan(got[30:]).all())


@gpu
def test_attend_wait_that_runs_out(hrb):
    """A barrier that nothing arrives at: the kernel gives up, the status is sticky, the context stays usable."""
    batch, offsets, kp, vp, q = attend_case(hrb, 128, 16, 2, 4, [40, 1], [300, 20], torch.bfloat16, 22)
    cache = hrb.PagedKV(kp, vp)
    want = cache.attend(q, batch)
    assert cache.get_error() == 0
    cache.set_wait_budget(2_000_000)
    cache.test_stall(True)
    cache.attend(q, batch)
    assert cache.get_error() == hrb.BITLIN_ETIMEOUT
    with pytest.raises(hrb.BitlinError):
        cache.attend(q, batch)
    assert torch.equal(hrb.PagedKV(kp, vp).attend(q, batch), want)


@gpu
def test_attend_long_ragged_batch_matches_its_parts(hrb):
    """Work split over the keys and joined: a long sequence beside short ones, against each alone."""
    lens, new = [9000, 3, 2500, 129, 1], [1, 3, 130, 2, 1]
    batch, offsets, kp, vp, q = attend_case(hrb, 128, 16, 2, 8, new, lens, torch.bfloat16, 16, q_scale=1.5)
    cache = hrb.PagedKV(kp, vp)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = cache.attend(q, batch, dtype=torch.float32, lse=lse)
    for s in range(5):
        rows = slice(offsets[s], offsets[s + 1])
        at = torch.arange(lens[s], device="cuda")
        where = batch.table[s, at // 16].long(), at % 16
        k, v = kp[where].double(), vp[where].double()
        i = torch.arange(new[s], device="cuda")
        seen = at[None, :] <= (lens[s] - new[s] + i)[:, None]
        qs = q[rows].double().view(new[s], 2, 4, 128)
        logits = torch.einsum("nhgd,khd->nhgk", qs, k) / math.sqrt(128)
        logits = logits.masked_fill(~seen[:, None, None], -math.inf)
        w = torch.softmax(logits, -1)
        want = torch.einsum("nhgk,khd->nhgd", w, v).reshape(new[s], 8, 128)
        size = torch.einsum("nhgk,khd->nhgd", w, v.abs()).reshape(new[s], 8, 128)
        mag = torch.einsum("nhgd,khd->nhgk", qs.abs(), k.abs()).amax() / math.sqrt(128)
        err = 2 * (24 * 2.0**-23 * float(mag) + 2.0**-21 * (1 + float(mag))) + 2.0**-20 + 2.0**-16
        assert bool(((out[rows].double() - want).abs() <= err * size).all())
        d = (lse[rows].double() - torch.logsumexp(logits, -1).reshape(new[s], 8)).abs()
        assert float(d.max()) <= err


def attend64_long(q, kp, vp, offsets, lens, table, scale):
    """attend64 for many keys, causal, a sequence at a time on the device.

    The relative error has three terms more.  A weight sum of n f32 additions, rounded to nearest: a
    random walk, 4 sqrt(n) 2^-24.  The tensor cores' additions, which lose 2.1e-8 of the sum each: 16 of
    them for each of 8 tiles (f32 output; 2.7e-6 < 2^-18), or 8 for each of 256 (16-bit; 4.3e-5 <
    2^-14).  One f32 addition for each drain and each part: at most 256 of 2^-24 together.
    Returns the reference of a 16-bit output and that of an f32 one."""
    T, H, D = q.shape
    page, kvh = kp.shape[1], kp.shape[2]
    out, size = (torch.zeros((T, H, D), dtype=torch.float64, device="cuda") for _ in range(2))
    lse, rel = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
    for s, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        where = table[s, at // page].long(), at % page
        k, v = kp[where].double(), vp[where].double()
        k_size = torch.where(torch.isfinite(k), k, 0.0).abs()
        new = offsets[s + 1] - offsets[s]
        for i0 in range(0, new, 64):
            i1 = min(new, i0 + 64)
            rows = slice(offsets[s] + i0, offsets[s] + i1)
            qs = q[rows].double().view(i1 - i0, kvh, H // kvh, D)
            seen = at[None, :] <= (n - new + torch.arange(i0, i1, device="cuda"))[:, None]
            logits = scale * torch.einsum("nhgd,khd->nhgk", qs, k)
            logits = logits.masked_fill(~seen[:, None, None], -math.inf)
            w = torch.softmax(logits, -1)
            out[rows] = torch.einsum("nhgk,khd->nhgd", w, v).reshape(i1 - i0, H, D)
            size[rows] = torch.einsum("nhgk,khd->nhgd", w, v.abs()).reshape(i1 - i0, H, D)
            lse[rows] = torch.logsumexp(logits, -1).reshape(i1 - i0, H)
            mag = abs(scale) * torch.einsum("nhgd,khd->nhgk", qs.abs(), k_size).amax(-1).reshape(i1 - i0, H)
            rel[rows] = 2 * (24 * 2.0**-23 * mag + 2.0**-21 * (1 + mag)) + 2.0**-20
    walk = 4 * math.sqrt(max(lens)) * 2.0**-24 + 256 * 2.0**-24
    out, lse, rel, size = out.cpu(), lse.cpu(), rel.cpu()[..., None].expand(T, H, D), size.cpu()
    return (out, lse, rel + walk + 2.0**-14, size), (out, lse, rel + walk + 2.0**-18, size)


def shared_pages(hrb, gen, seqs, new, lens, page, kvh, heads, dim, dtype):
    """A batch whose sequences all read the same pages, each a length of its own."""
    batch, _, pages = make_batch(hrb, gen, [1], [max(lens)], page)
    kp, vp = make_pools(gen, pages, page, kvh, dim, dtype)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets = [i * new for i in range(seqs + 1)]
    table = batch.table.expand(seqs, -1).contiguous()
    q = torch.randn((seqs * new, heads, dim), generator=gen, device="cuda").to(dtype)
    return hrb.KVBatch(i32(offsets), i32(lens), table), offsets, kp, vp, q


def check_long(hrb, batch, offsets, kp, vp, q, lens, scale, dtype):
    cache = hrb.PagedKV(kp, vp)
    refs = attend64_long(q, kp, vp, offsets, lens, batch.table, scale)
    for out_dtype, ref in zip((dtype, torch.float32), refs):
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = cache.attend(q, batch, scale=scale, dtype=out_dtype, lse=lse)
        assert cache.get_error() == 0
        check_attended(out, lse, ref, dtype)


@gpu
@pytest.mark.parametrize("per_sm,extra,kvh,heads,dim,new,length", [
    (1, 0, 1, 2, 64, 1, 200),     # as many items as SMs
    (1, 8, 4, 8, 128, 1, 260),    # a round, and a rest that is cut
    (2, 26, 3, 3, 64, 2, 130),    # two rounds
    (1, 1, 1, 6, 256, 3, 400),    # a rest of one item
    (70, 40, 8, 8, 64, 1, 5),     # more than the rounds that are listed
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_rounds_of_like_items(hrb, per_sm, extra, kvh, heads, dim, new, length, dtype):
    """Items of about the same cost, at least one per SM: taken whole, and the rest cut."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs = -(-(sms * per_sm + extra) // kvh)
    lens = [length - i % 2 for i in range(seqs)]
    case = shared_pages(hrb, generator(21), seqs, new, lens, 16, kvh, heads, dim, dtype)
    check_long(hrb, *case, lens, 1 / math.sqrt(dim), dtype)


@gpu
def test_attend_rounds_of_row_tiles(hrb):
    """One long sequence whose row tiles (8 tokens of 16 heads) cost about the same."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    new, lens = 8 * (sms + 23) - 3, [16000]
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 64, 1, 16, [new], lens, torch.bfloat16, 22)
    check_long(hrb, batch, offsets, kp, vp, q, lens, 0.125, torch.bfloat16)


@gpu
@pytest.mark.parametrize("rise", [0.0, 60.0, -60.0])
@pytest.mark.parametrize("lens_of", ["alike", "ragged"])
@pytest.mark.parametrize("dtype,length,dim", [(torch.bfloat16, 3000, 128), (torch.float16, 3000, 256),
                                              (torch.bfloat16, 36000, 64)])
def test_attend_drains(hrb, dtype, length, dim, lens_of, rise):
    """Parts long enough that their output goes to the workspace in between (past 8 tiles for an f32
    output, past 256 for a 16-bit one), with scores that are flat or rise or fall by 60 along the keys,
    so that the reference differs from one drain to the next."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs = sms + 48 if length < 10000 else sms + 4
    lens = [length - i % 3 if lens_of == "alike" else length + (i % 5) * (length // 16) for i in range(seqs)]
    batch, offsets, kp, vp, q = shared_pages(hrb, generator(23), seqs, 1, lens, 64, 1, 2, dim, dtype)
    q[..., 0] = 1.0
    most = max(lens)
    at = torch.arange(most, device="cuda")
    kp[batch.table[0, at // 64].long(), at % 64, 0, 0] = (rise * math.sqrt(dim) * at / most).to(dtype)
    check_long(hrb, batch, offsets, kp, vp, q, lens, 1 / math.sqrt(dim), dtype)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gone", [[(0, 128)], [(0, 256)], [(0, 300), (384, 512)], [(0, 639)]])
def test_attend_first_tiles_of_minus_infinity(hrb, dtype, gone):
    """Keys that score -inf through the whole first tile or more weigh nothing."""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 32, 1, 4, [1, 1], [640, 640], dtype, 24)
    q[..., 0] = 1.0
    for s in range(2):
        at = torch.cat([torch.arange(a, b, device="cuda") for a, b in gone])
        kp[batch.table[s, at // 32].long(), at % 32, 0, 0] = -math.inf
    check_long(hrb, batch, offsets, kp, vp, q, [640, 640], 0.125, dtype)


@gpu
def test_attend_and_append_past_32_bits(hrb):
    """Pools whose element offsets pass 2^32."""
    stride = 1 << 31
    buf = torch.empty(3 * stride + (1 << 20), dtype=torch.bfloat16, device="cuda")
    k, v = (buf[at:].as_strided((3, 16, 1, 64), (stride, 64, 64, 1)) for at in (0, 1 << 16))
    gen = generator(17)
    k.copy_(torch.randn(k.shape, generator=gen, device="cuda"))
    v.copy_(torch.randn(v.shape, generator=gen, device="cuda"))
    cache = hrb.PagedKV(k, v)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = hrb.KVBatch(i32([0, 2]), i32([45]), i32([[1, 0, 2]]))
    nk, nv = (torch.randn((2, 1, 64), generator=gen, device="cuda") for _ in range(2))
    q = cache.append(nk, nv, batch, q=torch.randn((2, 3, 64), generator=gen, device="cuda"))
    assert torch.equal(k[2, 11:13], nk.bfloat16()) and torch.equal(v[2, 11:13], nv.bfloat16())
    ref = attend64(q, k, v, [0, 2], [45], batch.table, 0.125, True)
    check_attended(cache.attend(q, batch, dtype=torch.float32), None, ref, torch.bfloat16)
    assert cache.get_error() == 0


@gpu
def test_attend_bad_tables(hrb):
    """A page outside the pool reads as zeros, a length past the table is cut; both are reported once."""
    gen = generator(18)
    kp, vp = make_pools(gen, 2, 16, 1, 64, torch.bfloat16)
    cache = hrb.PagedKV(kp, vp)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn((1, 1, 64), generator=gen, device="cuda").bfloat16()
    zk, zv = (torch.cat([p, torch.zeros_like(p[:1])]) for p in (kp, vp))
    for page in (2, 99, -1):
        got = cache.attend(q, hrb.KVBatch(i32([0, 1]), i32([40]), i32([[1, page, 0]])), dtype=torch.float32)
        assert cache.get_error() == hrb.BITLIN_EINDEX and cache.get_error() == 0
        ref = attend64(q, zk, zv, [0, 1], [40], torch.tensor([[1, 2, 0]]), 0.125, True)
        check_attended(got, None, ref, torch.bfloat16)
    got = cache.attend(q, hrb.KVBatch(i32([0, 1]), i32([33]), i32([[1, 0]])), dtype=torch.float32)
    assert cache.get_error() == hrb.BITLIN_EINDEX
    ref = attend64(q, kp, vp, [0, 1], [32], torch.tensor([[1, 0]]), 0.125, False)
    check_attended(got, None, ref, torch.bfloat16)


@gpu
def test_step_in_a_graph_and_on_another_stream(hrb):
    """Append and attention captured once, replayed as the sequence grows."""
    gen = generator(19)
    kp, vp = make_pools(gen, 8, 16, 2, 64, torch.bfloat16)
    cache = hrb.PagedKV(kp, vp)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = i32([60])
    batch = hrb.KVBatch(i32([0, 1]), lens, i32([[5, 1, 7, 0, 2, 6]]))
    rope = hrb.Rope(freqs(32))
    k, v = (torch.randn((1, 2, 64), generator=gen, device="cuda") for _ in range(2))
    q = torch.randn((1, 6, 64), generator=gen, device="cuda")
    q_out = torch.empty((1, 6, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((1, 6, 64), device="cuda")

    def step():
        cache.append(k, v, batch, rope=rope, q=q, q_out=q_out)
        cache.attend(q_out, batch, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (61, 64, 65, 90):
        lens.fill_(n)
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ref = attend64(q_out, kp, vp, [0, 1], [n], batch.table, 0.125, True)
        check_attended(out, None, ref, torch.bfloat16)
        at = n - 1
        assert torch.equal(vp[batch.table[0, at // 16], at % 16], v[0].bfloat16())
        check_rotated(q_out, q, torch.tensor([[at]]), freqs(32), [0] * 32, False)
    assert cache.get_error() == 0


@gpu
def test_layer_example(hrb):
    """Prompts and captured single-token steps of a layer, part by part against the definition.

    The projections' results are taken as given (their tests are elsewhere): projecting the same rows
    again gives the same bits.  The cache and the attention are compared with the definition, and the
    layer's output with the output projection of that attention, bit by bit.
    """
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
    import attention_layer as example

    lens, steps = [70, 1, 133], 5
    layer, table, inputs, outputs = example.serve(lens, steps)
    pairs = example.ROTARY // 2
    freq, axis = [1e7 ** (-i / pairs) for i in range(pairs)], [i % 3 for i in range(pairs)]
    past = [0] * len(lens)
    for part, x in enumerate(inputs):
        new = lens if part == 0 else [1] * len(lens)
        past = [a + b for a, b in zip(past, new)]
        batch, pos = example.make_batch(new, past, table)
        q, gate, k, v = layer.project(x)
        at = [(s, past[s] - new[s] + i) for s in range(len(lens)) for i in range(new[s])]
        where = (torch.stack([table[s, i // example.PAGE] for s, i in at]).long(),
                 torch.tensor([i % example.PAGE for _, i in at], device="cuda"))
        check_rotated(layer.cache.k[where], k, pos, freq, axis, False)
        assert torch.equal(layer.cache.v[where], v.bfloat16())
        # the attention over the cache as it was then
        q = layer.rope.apply(q, pos, dtype=torch.bfloat16)
        a = layer.cache.attend(q, batch, dtype=torch.float32)
        offsets = [sum(new[:i]) for i in range(len(new) + 1)]
        ref = attend64(q, layer.cache.k, layer.cache.v, offsets, past, table, 1 / math.sqrt(example.DIM), True)
        check_attended(a, None, ref, torch.bfloat16)
        again = layer.out((a * torch.sigmoid(gate)).view(-1, example.HEADS * example.DIM))
        assert torch.equal(again, outputs[part])


# ------------------------------------------------------------------ refusals

def test_refusals_without_device(hrb):
    """Arguments are checked before any device work."""
    L = hrb.lib()
    from hadamard_rotated_binary_gb300._binding import Batch, Rows

    E = hrb.BITLIN_EINVAL
    h = ctypes.c_void_p()
    f = (ctypes.c_float * 4)(1.0, 0.5, 0.25, 0.1)
    a = (ctypes.c_int32 * 4)(0, 1, 2, 0)
    new = lambda rotary=8, axes=3, freq=f, axis=a, pairing=0: L.bitlin_rope_create(ctypes.byref(h), rotary, axes, freq, axis, pairing)  # noqa: E731
    assert L.bitlin_rope_create(None, 8, 3, f, a, 0) == E
    for bad in (dict(rotary=0), dict(rotary=7), dict(axes=0), dict(axes=9), dict(freq=None), dict(pairing=2),
                dict(axes=2), dict(axis=(ctypes.c_int32 * 4)(0, -1, 0, 0)),
                dict(freq=(ctypes.c_float * 4)(1.0, math.inf, 0.0, 0.0)),
                dict(freq=(ctypes.c_float * 4)(1.0, math.nan, 0.0, 0.0))):
        assert new(**bad) == E and h.value is None
    p = 4096
    good = dict(k=p, v=p, pages=4, page_size=16, kv_heads=2, head_dim=64, dtype=1, page_stride=2048, slot_stride=128,
                head_stride=64)

    def kv(**change):
        return L.bitlin_kv_create(ctypes.byref(h), *{**good, **change}.values())

    assert L.bitlin_kv_create(None, *good.values()) == E
    for bad in (dict(k=None), dict(v=None), dict(k=p + 8), dict(v=p + 2), dict(pages=0), dict(page_size=4),
                dict(page_size=20), dict(page_size=65544), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=60),
                dict(head_dim=264), dict(dtype=0), dict(dtype=3), dict(page_stride=0), dict(slot_stride=100),
                dict(head_stride=-64), dict(page_stride=1 << 39)):
        assert kv(**bad) == E and h.value is None, bad
    r, b = Rows(p, 1, 64, 64), Batch(1, p, p, p, 1, 1)
    assert L.bitlin_rope_apply(None, r, 1, 1, 64, p, r, 0, None) == E
    assert L.bitlin_kv_append(None, b, 1, None, None, r, r, None, 0, None, None) == E
    assert L.bitlin_kv_attend(None, b, 1, r, 1, 1.0, 1, r, None, None) == E
    assert L.bitlin_kv_get_error(None) == E
    assert L.bitlin_kv_set_wait_budget(None, 1) == E and L.bitlin_kv_test_stall(None, 1) == E
    assert L.bitlin_kv_cuda_error(None) == 0
    assert L.bitlin_kv_destroy(None) == 0 and L.bitlin_rope_destroy(None) == 0


@gpu
def test_refusals(hrb):
    gen = generator(20)
    kp, vp = make_pools(gen, 4, 16, 2, 64, torch.bfloat16)
    cache = hrb.PagedKV(kp, vp)
    rope = hrb.Rope(freqs(32))
    wide = hrb.Rope(freqs(40))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = hrb.KVBatch(i32([0, 2]), i32([2]), i32([[0]]))
    k = torch.randn((2, 2, 64), device="cuda")
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    pos = i32([0, 1])
    before = kp.clone()
    refused = (ValueError, hrb.BitlinError)
    for call in (
        lambda: rope.apply(k[..., :32], pos),                                # narrower than the rotation
        lambda: rope.apply(k.double(), pos),
        lambda: rope.apply(k.transpose(1, 2), pos),                          # heads not contiguous
        lambda: rope.apply(k, pos.long()),
        lambda: rope.apply(k, pos[:1]),
        lambda: rope.apply(k.cpu(), pos),
        lambda: rope.apply(k, pos, out=k[:1]),
        lambda: cache.append(k, k[:1], batch),
        lambda: cache.append(k, k.bfloat16(), batch),                        # two types
        lambda: cache.append(k, k, batch, rope=wide, pos=pos),               # rotation wider than the head
        lambda: cache.append(k, k, batch, q=k[:1]),
        lambda: cache.append(k, k, batch, q=k, q_out=torch.empty_like(k)),   # q_out not of the cache's type
        lambda: cache.append(k[:, :1], k[:, :1], batch),
        lambda: cache.attend(q.half(), batch),
        lambda: cache.attend(q.float(), batch),
        lambda: cache.attend(q[:, :3], batch),                               # 3 heads over 2
        lambda: cache.attend(q[..., :32], batch),
        lambda: cache.attend(q, batch, dtype=torch.float16),
        lambda: cache.attend(q, batch, scale=math.inf),
        lambda: cache.attend(q, batch, lse=torch.empty((2, 3), device="cuda")),
        lambda: cache.attend(q, batch, out=torch.empty((2, 4, 65), device="cuda", dtype=q.dtype)[..., 1:]),
        lambda: cache.attend(torch.empty((2, 4, 68), device="cuda", dtype=q.dtype)[..., :64], batch),
        lambda: hrb.KVBatch(i32([0, 2]).long(), i32([2]), i32([[0]])),
        lambda: hrb.KVBatch(i32([0, 2]), i32([2, 3]), i32([[0]])),
        lambda: hrb.KVBatch(i32([0, 2]), i32([2]), i32([0])),
        lambda: hrb.PagedKV(kp, vp[:3]),
        lambda: hrb.PagedKV(kp.float(), vp.float()),
        lambda: hrb.PagedKV(kp[:, :4], vp[:, :4]),                           # pages of 4
    ):
        with pytest.raises(refused):
            call()
    assert cache.get_error() == 0 and torch.equal(kp, before)
    assert cache.attend(q[:0], hrb.KVBatch(i32([0, 0]), i32([2]), i32([[0]]))).shape == (0, 4, 64)

"""Norms of heads with their rotation, and the paged cache in 4 bits.

Calls are compared with the definition in 64 bits on the CPU, with bounds worked out from the
arithmetic (u = 2^-24):

  normed rotation   the sum of 256 squares in a tree of 9 roundings and one product each is off by
                    9 u, its root by half of that, rsqrt by 4 u, two products by 2 u; angle, sine
                    and cosine add 4 u and the rotation 2 u: 24 u of |a| + |b| holds all of it.  A
                    16-bit output takes the hardware's sine and cosine, 2^-21 each: 16 u more.
  gradient          g as a rotation (6 u of |a| + |b|), r and the row's sum of products as above:
                    40 u of the sum of magnitudes in r (|h| + |n| mean |h n|); the weight's
                    gradient adds N of them, in f32 partial sums of at most 2^-14 of the sum of
                    magnitudes.
  codes             equal to those of the 64-bit row, element by element.
  attention         as in test_attention_side, with weights in f16 (2^-11, two digits for an f32
                    output), whatever the cache's type.  f16 ends at 2^-24, half a step of which a
                    weight loses however small it is; weights are kept relative to 2^7 or more for
                    the largest, so that is 2^-32 of the largest a key, times the largest value.
"""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from test_attention_side import TINY, U, attend64, freqs, pair_size, rotate64  # noqa: E402

EPS = 1e-6
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def hrb():
    from hadamard_rotated_binary_gb300 import build as hbuild

    hbuild.build()
    import hadamard_rotated_binary_gb300 as m

    return m


# ------------------------------------------------------------------ definitions in 64 bits

def norm64(x, weight, eps=EPS):
    x = x.double().cpu()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()


def all_scales():
    return torch.tensor([math.ldexp((b & 7) + (8 if b >> 3 else 0), max(b >> 3, 1) - 18) for b in range(168)], dtype=torch.float64)


def encode64(x):
    """(codes 1..15 [..., D], scale bytes [..., 4]) of x in 64 bits, by search."""
    every = all_scales()
    x = torch.nan_to_num(x.double().cpu(), nan=0.0, posinf=1e300, neginf=-1e300)
    g = x.unflatten(-1, (4, -1))
    want = (g.abs().amax(-1) / 7).clamp(max=60.0)
    up = torch.searchsorted(every, want).clamp(max=167)  # the first scale >= want
    down = (up - 1).clamp(min=0)
    to_up, to_down = every[up] - want, want - every[down]
    byte = torch.where((to_up < to_down) | ((to_up == to_down) & (up % 2 == 0)), up, down)
    s = every[byte][..., None]
    code = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, 1.0)), 0.0).clamp(-7, 7) + 8
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def decode64(codes, scales):
    """Values of packed codes [..., D / 2] and scale bytes [..., 4]."""
    nibbles = torch.stack((codes.cpu() & 15, codes.cpu() >> 4), -1).flatten(-2).double() - 8
    return (nibbles.unflatten(-1, (4, -1)) * all_scales()[scales.cpu().long()][..., None]).flatten(-2)


def unpacked(codes):
    return torch.stack((codes.cpu() & 15, codes.cpu() >> 4), -1).flatten(-2)


# ------------------------------------------------------------------ inputs

def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(gen, shape, dtype, layout="plain", loud=True):
    """[T][H][D] in one of several memory layouts."""
    t, h, d = shape
    x = torch.randn(shape, generator=gen, device="cuda")
    if loud:
        x = x * torch.exp(torch.randn((h, d), generator=gen, device="cuda"))
    x = x.to(dtype)
    if layout == "plain":
        return x
    if layout == "heads":  # [H][T][D] in memory
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "odd":    # rows that no vector access fits
        wide = torch.zeros((t, h, d + 3), dtype=dtype, device="cuda")
        wide[..., 1:d + 1] = x
        return wide[..., 1:d + 1]
    raise ValueError(layout)


def weight(gen, dim):
    return torch.exp(0.5 * torch.randn((dim,), generator=gen, device="cuda"))


class Cache:
    """A 4-bit cache of sequences of the given lengths, with a shuffled table."""

    def __init__(self, hrb, gen, lens, page, kvh, dim, dtype, layout="heads", fill=None, spare=2, width=0):
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        if layout == "heads":
            parts = hrb.QuantKV.pools(pages, page, kvh, dim)
        else:
            parts = tuple(torch.zeros((pages, page, kvh, n), dtype=torch.uint8, device="cuda") for n in (dim // 2, dim // 2, 4, 4))
        self.parts = parts
        if fill is not None:
            for p in parts:
                p.fill_(fill)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(page)).to(torch.int32)
        width = max(max(need), width, 1)
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        self.table, self.page, self.lens = table.cuda(), page, list(lens)
        self.kv = hrb.QuantKV(*parts, dtype=dtype)

    def random(self, gen):
        """Codes and scales of ordinary values in every slot that a sequence holds."""
        for s, n in enumerate(self.lens):
            place = torch.arange(n, device="cuda")
            at = (self.table[s, (place // self.page)].long(), place % self.page)
            kvh, half = self.parts[0].shape[2:]
            for p in self.parts[:2]:
                # nibbles 1..15
                p[at] = (torch.randint(1, 16, (n, kvh, half), generator=gen, device="cuda")
                         + 16 * torch.randint(1, 16, (n, kvh, half), generator=gen, device="cuda")).to(torch.uint8)
            for p in self.parts[2:]:
                p[at] = torch.randint(90, 115, (n, kvh, 4), generator=gen, device="cuda").to(torch.uint8)
        return self

    def values(self):
        parts = [p.cpu() for p in self.parts]
        keep = [p.clone() for p in parts[2:]]
        for p in keep:
            p[p > 167] = 0  # bytes that no append writes
        return decode64(parts[0], keep[0]), decode64(parts[1], keep[1])


def batch_of(hrb, new, cache, lens=None):
    offsets = [sum(new[:i]) for i in range(len(new) + 1)]
    return hrb.KVBatch(i32(offsets), i32(lens or cache.lens), cache.table), offsets


# ------------------------------------------------------------------ norm and rotation

NORMED = [
    # tokens, heads, dim, rotary, axes, adjacent, src, dst, layout
    (1, 24, 256, 64, 3, False, torch.float32, torch.bfloat16, "plain"),
    (5, 3, 80, 80, 2, False, torch.bfloat16, torch.bfloat16, "heads"),
    (33, 1, 128, 128, 1, True, torch.float16, torch.float32, "plain"),
    (7, 5, 64, 32, 3, True, torch.bfloat16, torch.float16, "odd"),
    (130, 6, 256, 256, 5, False, torch.float32, torch.float32, "plain"),
    (3, 2, 30, 10, 1, False, torch.float32, torch.float32, "plain"),
    (2, 9, 8, 8, 1, True, torch.float32, torch.float32, "plain"),
    (4, 2, 7, 2, 1, True, torch.float32, torch.float32, "odd"),
    (3, 4, 248, 120, 2, False, torch.float16, torch.float16, "plain"),
    (2, 3, 256, 250, 2, False, torch.bfloat16, torch.float32, "heads"),
]


def normed_inputs(hrb, case, seed=0):
    t, h, d, r, axes, adjacent, src, dst, layout = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    inv, axis = freqs(r // 2), [i % axes for i in range(r // 2)]
    rope = hrb.Rope(inv, axis, adjacent=adjacent)
    pos = torch.randint(-5000, 100000, (rope.axes, t), generator=gen, device="cuda", dtype=torch.int32)
    return gen, inv, axis, rope, pos, rows(gen, (t, h, d), src, layout), weight(gen, d)


def check_normed(y, n, pos, inv, axis, adjacent):
    ref = rotate64(n, pos, inv, axis, adjacent)
    units = 24 if y.dtype == torch.float32 else 40
    size = pair_size(n, 2 * len(inv), adjacent)
    size[..., 2 * len(inv):] = n[..., 2 * len(inv):].abs()
    bound = units * 2.0**-24 * size
    bound = bound + U[y.dtype] * (ref.abs() + bound) + TINY[y.dtype]
    assert bool(((y.double().cpu() - ref).abs() <= bound).all())


@gpu
@pytest.mark.parametrize("case", NORMED, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_normed_rotation(hrb, case):
    _, inv, axis, rope, pos, x, w = normed_inputs(hrb, case)
    y = rope.apply(x, pos, dtype=case[7], norm=w)
    check_normed(y, norm64(x, w), pos, inv, axis, case[5])
    if case[7] == case[6]:  # in place
        z = x.clone() if case[8] == "plain" else x
        assert rope.apply(z, pos, out=z, norm=w) is z
        assert torch.equal(z, y)


@gpu
def test_normed_rotation_of_rows_that_are_zero_huge_or_not_finite(hrb):
    rope, w = hrb.Rope(freqs(16)), torch.full((64,), 2.0, device="cuda")
    x = torch.randn((6, 1, 64), device="cuda")
    x[0] = 0
    x[1] *= 1e18
    x[2] *= 1e-18
    x[3, 0, 5] = math.nan
    x[4, 0, 63] = math.inf
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    y = rope.apply(x, pos, norm=w, eps=1e-6)
    keep = [0, 1, 2, 5]
    assert bool(torch.isfinite(y[keep]).all()) and bool((y[0] == 0).all())
    check_normed(y[keep], norm64(x, w)[keep], pos[keep][None], freqs(16), [0] * 16, False)
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4, 0, 63]))
    z = rope.apply(x[:1], pos[:1], norm=w, eps=0.0)
    assert bool(torch.isnan(z).all())
    # a sum of squares past what f32 holds
    assert bool((rope.apply(x[5:] * 1e25, pos[5:], norm=w) == 0).all())


def gradient64(dy, x, w, pos, inv, axis, adjacent):
    """(dx, dw, sizes of their terms)."""
    g = rotate64(dy, pos, inv, axis, adjacent, -1.0)
    x, w = x.double().cpu(), w.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, h = x * r, g * w
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    gs = pair_size(dy, 2 * len(inv), adjacent)
    gs[..., 2 * len(inv):] = dy.double().cpu()[..., 2 * len(inv):].abs()
    size = r * (gs * w.abs() + n.abs() * (gs * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1)), size, (gs * n.abs()).sum((0, 1))


@gpu
@pytest.mark.parametrize("case", NORMED, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_gradient(hrb, case):
    gen, inv, axis, rope, pos, x, w = normed_inputs(hrb, case, 1)
    dy = rows(gen, x.shape, case[7], case[8], loud=False)
    dx, dw = rope.gradient(dy, x, pos, w)
    assert dx.dtype == x.dtype and dw.dtype == torch.float32
    ref, ref_w, size, size_w = gradient64(dy, x, w, pos, inv, axis, case[5])
    bound = 40 * 2.0**-24 * size
    bound = bound + U[dx.dtype] * (ref.abs() + bound) + TINY[dx.dtype]
    assert bool(((dx.double().cpu() - ref).abs() <= bound).all())
    assert bool(((dw.double().cpu() - ref_w).abs() <= 2.0**-14 * size_w).all())
    again = rope.gradient(dy, x, pos, w)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@gpu
def test_gradient_of_many_rows_and_against_differences(hrb):
    t, h, d, r = 1531, 7, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    rope, pos = hrb.Rope(freqs(r // 2)), torch.arange(t, dtype=torch.int32, device="cuda")
    x, dy, w = rows(gen, (t, h, d), torch.float32), rows(gen, (t, h, d), torch.float32, loud=False), weight(gen, d)
    dx, dw = rope.gradient(dy, x, pos, w)
    ref, ref_w, size, size_w = gradient64(dy, x, w, pos[None], freqs(r // 2), [0] * (r // 2), False)
    assert bool(((dx.double().cpu() - ref).abs() <= 41 * 2.0**-24 * size).all())
    assert bool(((dw.double().cpu() - ref_w).abs() <= 2.0**-14 * size_w).all())
    # along a direction, by central differences of the f32 forward pass: each of its 2^20 products is off
    # by 2^-21 at random, 2^-11 together, over a step of 2^-6; the third derivative adds the step's square
    for which in ("x", "w"):
        step = 2.0**-6
        along = torch.randn((t, h, d) if which == "x" else (d,), generator=gen, device="cuda")
        f = lambda a: (rope.apply(x + a * along, pos, norm=w) if which == "x" else  # noqa: E731
                       rope.apply(x, pos, norm=w + a * along)).double().mul(dy.double()).sum()
        slope = float(f(step) - f(-step)) / (2 * step)
        want = float(((dx if which == "x" else dw).double() * along.double()).sum())
        scale = float(((dx if which == "x" else dw).double() * along.double()).norm())
        assert abs(slope - want) <= 2.0**-6 * scale + 2.0**-4, (which, slope, want, scale)


@gpu
def test_gradient_in_place_and_of_nothing(hrb):
    rope, w = hrb.Rope(freqs(32)), torch.ones(64, device="cuda")
    x, dy = torch.randn((9, 3, 64), device="cuda"), torch.randn((9, 3, 64), device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    dx, dw = rope.gradient(dy, x, pos, w)
    for name in ("x", "dy"):
        a, b = x.clone(), dy.clone()
        got, got_w = rope.gradient(b, a, pos, w, dx=a if name == "x" else b)
        assert got is (a if name == "x" else b) and torch.equal(got, dx) and torch.equal(got_w, dw)
    empty, zero = rope.gradient(dy[:0], x[:0], pos[:0], w)
    assert empty.shape == (0, 3, 64) and bool((zero == 0).all())


# ------------------------------------------------------------------ append

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,rotary", [(256, 64), (80, 40)])
def test_normed_append_to_the_16_bit_cache(hrb, dtype, dim, rotary):
    gen = torch.Generator(device="cuda").manual_seed(2)
    lens, new, page, kvh, heads = [40, 7, 100], [3, 7, 1], 16, 2, 6
    pools = [torch.zeros((16, page, kvh, dim), dtype=dtype, device="cuda") for _ in range(2)]
    table = torch.randperm(16, generator=torch.Generator().manual_seed(1)).to(torch.int32)[:21 - 6].view(3, 5).repeat(1, 2).cuda()
    cache, rope = hrb.PagedKV(*pools), hrb.Rope(freqs(rotary // 2))
    k, v, q = (rows(gen, (12, n, dim), torch.float32) for n in (kvh, kvh, heads))
    qw, kw = weight(gen, dim), weight(gen, dim)
    pos = torch.arange(100, 112, dtype=torch.int32, device="cuda")
    batch = hrb.KVBatch(i32([0, 3, 10, 11]), i32(lens), table)  # the 12th row is padding
    q_out = torch.full((12, heads, dim), 7.0, dtype=dtype, device="cuda")
    assert cache.append(k, v, batch, rope=rope, pos=pos, q=q, q_out=q_out, q_norm=qw, k_norm=kw) is q_out
    want = rope.apply(k, pos, dtype=dtype, norm=kw)
    assert torch.equal(q_out[:11], rope.apply(q, pos, dtype=dtype, norm=qw)[:11]) and bool((q_out[11] == 7).all())
    row = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        for place in range(n - m, n):
            at = (int(table[s, place // page]), place % page)
            assert torch.equal(cache.k[at], want[row]) and torch.equal(cache.v[at], v[row].to(dtype))
            row += 1
    # a norm of one of the two alone, and without a rotation
    got = cache.append(k, v, batch, q=q, q_norm=qw)
    assert torch.allclose(got[:11].double().cpu(), norm64(q, qw)[:11], rtol=2 * U[dtype], atol=1e-4)
    at = (int(table[0, 37 // page]), 37 % page)
    assert torch.equal(cache.k[at], k[0].to(dtype))


STORED = [
    # lens, new, page, kv_heads, heads, dim, rotary, adjacent, src, dtype, layout, pools, norms, positions
    ([40, 7, 100], [3, 7, 1], 16, 2, 6, 256, 64, False, torch.float32, torch.bfloat16, "plain", "heads", True, True),
    ([300, 1], [300, 1], 48, 4, 4, 128, 128, True, torch.bfloat16, torch.float16, "heads", "slots", True, False),
    ([64, 65, 66], [5, 60, 0], 7, 1, 3, 64, 32, False, torch.float16, torch.bfloat16, "plain", "heads", True, True),
    ([1000], [1000], 1, 8, 8, 64, 64, True, torch.float32, torch.float16, "odd", "heads", True, False),
    ([90, 30], [90, 30], 16, 3, 3, 128, 20, False, torch.float32, torch.bfloat16, "plain", "slots", True, True),
    ([200], [77], 64, 5, 5, 256, 0, False, torch.bfloat16, torch.bfloat16, "plain", "heads", False, False),
    ([200], [77], 64, 5, 5, 256, 128, False, torch.float32, torch.bfloat16, "plain", "heads", False, True),
    ([700], [700], 32, 8, 8, 256, 0, False, torch.float32, torch.float16, "odd", "heads", True, False),
]


@gpu
@pytest.mark.parametrize("case", STORED, ids=range(len(STORED)))
def test_stored_codes_are_those_of_the_exact_rows(hrb, case):
    lens, new, page, kvh, heads, dim, rotary, adjacent, src, dtype, layout, pools, norms, positions = case
    gen = torch.Generator(device="cuda").manual_seed(len(lens) + dim)
    cache = Cache(hrb, gen, lens, page, kvh, dim, dtype, pools)
    batch, offsets = batch_of(hrb, new, cache)
    tokens = offsets[-1]
    k, v, q = (rows(gen, (tokens + 2, n, dim), src, layout) for n in (kvh, kvh, heads))
    qw, kw = (weight(gen, dim), weight(gen, dim)) if norms else (None, None)
    inv, axis = freqs(rotary // 2, 1e6), [0] * (rotary // 2)
    rope = hrb.Rope(inv, adjacent=adjacent) if rotary else None
    places = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)] + [torch.zeros(2, dtype=torch.long)])
    pos = (places * 3 + 1 if positions else places).to(torch.int32)[None]
    q_out = torch.full((tokens + 2, heads, dim), 7.0, dtype=dtype, device="cuda")
    cache.kv.append(k, v, batch, rope=rope, pos=pos.cuda() if positions else None, q=q, q_out=q_out, q_norm=qw, k_norm=kw)
    assert cache.kv.get_error() == hrb.BITLIN_OK and bool((q_out[tokens:] == 7).all())
    turned = lambda x: rotate64(x, pos, inv, axis, adjacent) if rotary else x  # noqa: E731
    n = norm64(q, qw) if norms else q.double().cpu()
    if rotary:
        check_normed(q_out[:tokens], n[:tokens], pos[:, :tokens], inv, axis, adjacent)
    else:
        bound = (24 * 2.0**-24 + U[dtype]) * 1.01 * n.abs() + TINY[dtype]
        assert bool(((q_out.double().cpu() - n).abs() <= bound)[:tokens].all())
    want = {"k": encode64(turned(norm64(k, kw) if norms else k.double().cpu())), "v": encode64(v)}
    row, held = 0, torch.zeros(cache.parts[0].shape[:2], dtype=torch.bool)
    for s, (length, m) in enumerate(zip(lens, new)):
        place = torch.arange(length - m, length)
        at = (cache.table[s].cpu()[place // page].long(), place % page)
        held[at] = True
        for name, codes, scales in (("k", cache.parts[0], cache.parts[2]), ("v", cache.parts[1], cache.parts[3])):
            assert torch.equal(scales.cpu()[at], want[name][1][row:row + m]), name
            assert torch.equal(unpacked(codes.cpu()[at]), want[name][0][row:row + m]), name
        row += m
    for p in cache.parts:  # nothing else was written
        assert bool((p.cpu()[~held] == 0).all())
    # reading the rows back gives their values, exactly, in every type
    for out in (torch.float32, torch.bfloat16, torch.float16):
        got = cache.kv.read(batch, tokens, dtype=out)
        for y, name in zip(got, ("k", "v")):
            code, byte = (w[:tokens] for w in want[name])
            value = ((code.double() - 8).unflatten(-1, (4, -1)) * all_scales()[byte.long()][..., None]).flatten(-2)
            assert y.dtype == out and torch.equal(y.double().cpu(), value)


@gpu
def test_borders_ties_and_values_that_are_not_finite(hrb):
    """Elements at, just below and just above the middle of two codes; scales likewise; extremes."""
    dim = 64
    special = []
    every = all_scales().tolist()
    for b in (1, 7, 8, 100, 119, 120, 166):  # a scale's own magnitude, and the middle to the next one
        for at in (every[b] * 7, (every[b] + every[b + 1]) / 2 * 7):
            x = float(torch.tensor(at, dtype=torch.float32))
            for y in (x, x * (1 - 2.0**-23), x * (1 + 2.0**-23)):
                special.append([y] + [0.0] * 15)
    for b in (3, 90, 117):
        s = every[b]
        tie = [(c + 0.5) * s for c in range(-7, 7)]
        for f in (1.0, 1 - 2.0**-23, 1 + 2.0**-23):
            special.append([7 * s] + [t * f for t in tie] + [-7 * s])
    special += [[math.nan] * 16, [math.nan] + [1.0] * 15, [math.inf] + [-1.0] * 15, [-math.inf, math.nan] + [300.0] * 14,
                [1e30] * 16, [1e-30] * 16, [2.6e-5] * 16, [2.8e-5] * 16, [-0.0] * 16, [419.0, 420.0, 421.0, -450.0] * 4,
                [1e-45] * 16, [3.4e38] * 16]
    special += [[0.0] * 16] * (-len(special) % 4)
    x = torch.tensor(special, dtype=torch.float32).view(-1, 1, dim).cuda()
    n = x.shape[0]
    cache = Cache(hrb, None, [n], 16, 1, dim, torch.float16)
    batch, _ = batch_of(hrb, [n], cache)
    cache.kv.append(x, x, batch)
    codes, scales = encode64(x)
    place = torch.arange(n)
    at = (cache.table[0].cpu()[place // 16].long(), place % 16)
    for c, s in ((cache.parts[0], cache.parts[2]), (cache.parts[1], cache.parts[3])):
        assert torch.equal(s.cpu()[at], scales)
        assert torch.equal(unpacked(c.cpu()[at]), codes)
    k, v = cache.kv.read(batch, n, dtype=torch.float32)
    assert bool(torch.isfinite(k).all()) and torch.equal(k, v)


@gpu
def test_normed_rows_at_borders_go_by_their_64_bit_values(hrb):
    """Rows whose normed values lie within 32 bits' error of borders, by construction of the weight."""
    dim, n = 128, 512
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((n, 1, dim), generator=gen, device="cuda").sign() * (1 + torch.randint(0, 3, (n, 1, dim), generator=gen, device="cuda"))
    w = torch.ones(dim, device="cuda")
    # in the first row, put elements at borders of the first group's codes: x r w = (c + 1/2) s
    code, byte = encode64(norm64(x[:1], w))
    s = all_scales()[byte.long()][0, 0].repeat_interleave(dim // 4)
    n0 = norm64(x[:1], w)[0, 0]
    target = (torch.round(n0 / s) + 0.5 * torch.sign(n0)).clamp(-6.5, 6.5) * s
    w[1::2] = (target / n0)[1::2].float().cuda()
    cache = Cache(hrb, None, [n], 16, 1, dim, torch.bfloat16)
    batch, _ = batch_of(hrb, [n], cache)
    cache.kv.append(x, x, batch, k_norm=w)
    codes, scales = encode64(norm64(x, w))
    place = torch.arange(n)
    at = (cache.table[0].cpu()[place // 16].long(), place % 16)
    assert torch.equal(cache.parts[2].cpu()[at], scales)
    assert torch.equal(unpacked(cache.parts[0].cpu()[at]), codes)


@gpu
@pytest.mark.parametrize("adjacent", [None, False, True])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
def test_normed_rows_whose_squares_leave_the_range_of_f32(hrb, src, adjacent):
    """Codes of rows whose squares overflow or underflow in 32 bits are those of the exact rows."""
    dim, rotary = 64, 32
    gen = torch.Generator(device="cuda").manual_seed(12)
    for eps, sizes in ((EPS, (1e18, 1e19, 1e25, 1e37, 1.0)), (0.0, (1e-18, 1e-22, 1e-30, 1e-37, 0.0)), (1e-40, (1e-18, 1e-20, 1e-22, 0.0, 1.0))):
        x = torch.cat([torch.randn((4, 2, dim), generator=gen, device="cuda") * s for s in sizes]).to(src)
        n, w = x.shape[0], weight(gen, dim)
        rope = None if adjacent is None else hrb.Rope(freqs(rotary // 2), adjacent=adjacent)
        pos = torch.randint(0, 9000, (1, n), generator=gen, device="cuda", dtype=torch.int32)
        want = norm64(x, w, eps)
        if rope is not None:
            want = rotate64(want, pos, freqs(rotary // 2), [0] * (rotary // 2), adjacent)
        cache = Cache(hrb, None, [n], 16, 2, dim, torch.bfloat16)
        batch, _ = batch_of(hrb, [n], cache)
        cache.kv.append(x, x, batch, rope=rope, pos=None if rope is None else pos, k_norm=w, eps=eps)
        codes, scales = encode64(want)
        place = torch.arange(n)
        at = (cache.table[0].cpu()[place // 16].long(), place % 16)
        assert torch.equal(cache.parts[2].cpu()[at], scales)
        assert torch.equal(unpacked(cache.parts[0].cpu()[at]), codes)


@gpu
def test_places_outside_are_reported_and_not_written(hrb):
    cache = Cache(hrb, None, [20, 20], 16, 1, 64, torch.bfloat16, spare=0)
    cache.table[1, 1] = 99
    k = torch.ones((4, 1, 64), device="cuda")
    batch, _ = batch_of(hrb, [2, 2], cache, [20, 20])
    cache.kv.append(k, k, batch)  # the second sequence's rows fall into page 99
    assert cache.kv.get_error() == hrb.BITLIN_EINDEX and cache.kv.get_error() == hrb.BITLIN_OK
    before = [p.clone() for p in cache.parts]
    got = cache.kv.read(batch, 4)
    assert cache.kv.get_error() == hrb.BITLIN_EINDEX
    one = 7 * 9 / 64  # the scale nearest to 1 / 7 is 9 / 64
    assert bool((got[0][:2] == one).all()) and bool((got[0][2:] == 0).all())
    for lens in ([33, 20], [20, 1]):  # past the table's row; a negative place
        batch, _ = batch_of(hrb, [0, 4] if lens[0] == 20 else [1, 0], cache, lens)
        cache.kv.append(k[:1] if lens[0] == 33 else k[:3], k[:1] if lens[0] == 33 else k[:3], batch)
        assert cache.kv.get_error() == hrb.BITLIN_EINDEX
    out = torch.full((6, 1, 64), 3.0, device="cuda"), torch.full((6, 1, 64), 3.0, device="cuda")
    batch, _ = batch_of(hrb, [2, 0], cache, [20, 0])
    assert cache.kv.read(batch, 6, *out) == out
    assert bool((out[0][:2] == one).all()) and bool((out[0][2:] == 3).all()) and bool((out[1][2:] == 3).all())
    assert all(torch.equal(a, b) for a, b in zip(before, cache.parts))
    assert cache.kv.get_error() == hrb.BITLIN_OK


@gpu
def test_read_into_strided_rows_and_whole_sequences(hrb):
    gen = torch.Generator(device="cuda").manual_seed(4)
    cache = Cache(hrb, gen, [50, 0, 3], 16, 3, 128, torch.float16).random(gen)
    batch, offsets = batch_of(hrb, [50, 0, 3], cache)
    want = [torch.cat([p[cache.table[s].cpu()[torch.arange(n) // 16].long(), torch.arange(n) % 16] for s, n in enumerate(cache.lens)])
            for p in cache.values()]
    for layout in ("heads", "odd"):
        out = [rows(gen, (53, 3, 128), torch.bfloat16, layout) for _ in range(2)]
        cache.kv.read(batch, 53, *out)
        assert all(torch.equal(o.double().cpu(), w) for o, w in zip(out, want))


# ------------------------------------------------------------------ attention

ATTENDED = [
    # lens, new, page, kv_heads, group, dim, dtype, out, causal, pools
    ([1], [1], 16, 1, 1, 64, torch.float16, torch.float32, True, "heads"),
    ([777], [1], 64, 4, 6, 256, torch.bfloat16, torch.float32, True, "heads"),
    ([5000], [1], 64, 2, 6, 256, torch.bfloat16, torch.bfloat16, True, "heads"),
    ([31, 32, 33, 1, 500, 129], [1] * 6, 16, 2, 8, 128, torch.float16, torch.float16, True, "slots"),
    ([31, 0, 33, 1, 260], [1] * 5, 5, 3, 3, 64, torch.bfloat16, torch.float32, True, "heads"),
    ([300, 80], [5, 5], 32, 2, 4, 128, torch.float16, torch.float16, True, "heads"),
    ([300, 80, 4], [5, 0, 4], 48, 2, 3, 256, torch.bfloat16, torch.float32, True, "slots"),
    ([90, 64], [90, 3], 16, 1, 8, 64, torch.bfloat16, torch.bfloat16, False, "heads"),
    ([3, 10], [5, 10], 16, 2, 2, 128, torch.float16, torch.float32, True, "heads"),  # more rows than keys: some see none
    ([70], [2], 1, 1, 128, 64, torch.float16, torch.float16, True, "heads"),
    ([1000], [17], 256, 1, 9, 128, torch.bfloat16, torch.bfloat16, True, "slots"),
    ([2100, 900], [1, 1], 16, 1, 16, 128, torch.bfloat16, torch.float32, False, "heads"),
]


def attended(hrb, case, seed=0, **more):
    lens, new, page, kvh, group, dim, dtype, out, causal, pools = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    # free slots hold scales that are infinities and NaNs
    cache = Cache(hrb, gen, lens, page, kvh, dim, dtype, pools, fill=255).random(gen)
    batch, offsets = batch_of(hrb, new, cache)
    q = (2 * torch.randn((offsets[-1], kvh * group, dim), generator=gen, device="cuda")).to(dtype)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    y = cache.kv.attend(q, batch, causal=causal, dtype=out, lse=lse, **more)
    return cache, batch, offsets, q, y, lse


def check_attended(y, lse, ref, pool_dtype, lost=0.0):
    """lost: what weights below f16's smallest step may be off by together, times the largest value."""
    out, ref_lse, err, size = ref
    u = U[pool_dtype]
    bound = size * (err + (u if y.dtype != torch.float32 else u * u)) + lost
    bound = bound + U[y.dtype] * (out.abs() + bound) + TINY[y.dtype]
    got = y.double().cpu()
    assert bool(torch.isfinite(got).all())
    assert bool(((got - out).abs() <= bound).all()), float(((got - out).abs() / bound.clamp(min=1e-300)).max())
    if lse is not None:
        got = lse.double().cpu()
        empty = torch.isinf(ref_lse)
        assert bool((got[empty] == -math.inf).all())
        assert bool(((got - ref_lse).abs() <= err[..., 0] + 2.0**-21 * ref_lse.abs())[~empty].all())


def reference(cache, offsets, lens, q, causal, scale=None):
    k, v = cache.values()
    return attend64(q, k, v, offsets, lens, cache.table, scale or q.shape[-1] ** -0.5, causal)


@gpu
@pytest.mark.parametrize("case", ATTENDED, ids=range(len(ATTENDED)))
def test_attention(hrb, case):
    cache, _, offsets, q, y, lse = attended(hrb, case)
    check_attended(y, lse, reference(cache, offsets, case[0], q, case[8]), torch.float16)
    assert cache.kv.get_error() == hrb.BITLIN_OK


THROUGH = [c for c in ATTENDED if c[2] % 8 == 0] + [
    ([300, 80], [25, 25], 32, 2, 4, 128, torch.float16, torch.float16, True, "heads"),
    ([300, 80, 4], [60, 0, 9], 48, 2, 6, 256, torch.bfloat16, torch.float32, True, "slots"),
    ([300, 80, 4], [60, 0, 9], 48, 2, 6, 256, torch.bfloat16, torch.bfloat16, True, "slots"),
    ([130, 0, 64], [130, 5, 0], 8, 3, 4, 64, torch.bfloat16, torch.bfloat16, False, "heads"),
]


@gpu
@pytest.mark.parametrize("case", THROUGH, ids=str)
def test_attention_through_16_bit_pages(hrb, case):
    lens, new, page, kvh, group, dim, dtype, out, causal, pools = case
    need = sum(-(-n // page) for n in lens) + 2
    scratch = [torch.full((need, page, kvh, dim), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
    through = hrb.PagedKV(*scratch)
    cache, _, offsets, q, y, lse = attended(hrb, case, through=through, f32_through=True)
    many = offsets[-1] * group > 80 * len(lens)
    check_attended(y, lse, reference(cache, offsets, lens, q, causal), dtype if many else torch.float16)
    assert cache.kv.get_error() == hrb.BITLIN_OK and through.get_error() == hrb.BITLIN_OK


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,new,group,dim", [([900, 3000], [60, 60], 4, 128), ([700], [300], 6, 256)])
def test_f32_outputs_of_many_rows_are_as_exact_as_f32_arithmetic(hrb, dtype, lens, new, group, dim):
    """With 16-bit pages at hand and without, the same bits, and 2^-20 off at most."""
    case = (lens, new, 64, 2, group, dim, dtype, torch.float32, True, "heads")
    need = sum(-(-n // 64) for n in lens) + 2
    through = hrb.PagedKV(*(torch.zeros((need, 64, 2, dim), dtype=dtype, device="cuda") for _ in range(2)))
    cache, batch, offsets, q, y, _ = attended(hrb, case, through=through)
    assert torch.equal(y, cache.kv.attend(q, batch, dtype=torch.float32))
    out = reference(cache, offsets, lens, q, True)[0]
    ours = float((y.double().cpu() - out).norm() / out.norm())
    # a weight is two f16 digits (2^-23 of it), its exponential and the sum's some 2^-21 at scores of 10, the
    # additions, rounded, 2^-24 times the root of some 100 tiles: 2^-20 together
    assert ours <= 2.0**-20, ours


@gpu
@pytest.mark.parametrize("many", [False, True])
def test_attention_over_pages_outside_and_lengths_past_the_table(hrb, many):
    lens, page, kvh, dim = [40, 40], 16, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = Cache(hrb, gen, lens, page, kvh, dim, torch.float16).random(gen)
    through = hrb.PagedKV(*(torch.zeros((8, page, kvh, dim), dtype=torch.float16, device="cuda") for _ in range(2))) if many else None
    out = torch.float16 if many else torch.float32
    new = [30, 30] if many else [1, 1]  # 60 rows, or 2, of 8 query heads: the first through 16-bit pages
    q = torch.randn((sum(new), 8, dim), generator=gen, device="cuda").half()
    batch, offsets = batch_of(hrb, new, cache)
    k, v = cache.values()
    old = int(cache.table[1, 1])
    for bad in (8, -1, 2**31 - 1):
        cache.table[1, 1] = bad
        y = cache.kv.attend(q, batch, dtype=out, through=through)
        assert cache.kv.get_error() == hrb.BITLIN_EINDEX
        kk, vv = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (k, v))
        table = cache.table.cpu().clone()
        table[1, 1] = kk.shape[0] - 1
        check_attended(y, None, attend64(q, kk, vv, offsets, lens, table, dim**-0.5, True), torch.float16)
    cache.table[1, 1] = old
    # (causal rows past the end of the table's row see all of it)
    batch, _ = batch_of(hrb, new, cache, [40, 1000])
    y = cache.kv.attend(q, batch, dtype=out, causal=False, through=through)
    assert cache.kv.get_error() == hrb.BITLIN_EINDEX
    ref = attend64(q, k, v, offsets, [40, 48], cache.table, dim**-0.5, False)
    if int(cache.table[1, 2]) >= 0:
        check_attended(y, None, ref, torch.float16)


@gpu
def test_attention_of_large_and_small_scores(hrb):
    lens, dim = [400], 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = Cache(hrb, gen, lens, 16, 1, dim, torch.bfloat16).random(gen)
    batch, offsets = batch_of(hrb, [1], cache)
    for size in (2.0**-120, 2.0**-20, 1.0, 64.0, 2.0**20, 2.0**60):
        q = (torch.randn((1, 4, dim), generator=gen, device="cuda") * size).bfloat16()
        y = cache.kv.attend(q, batch, scale=dim**-0.5 * min(1.0, 8 / size), dtype=torch.float32)
        check_attended(y, None, reference(cache, offsets, lens, q, True, dim**-0.5 * min(1.0, 8 / size)), torch.float16)
    # a negative scale, and one of zero: the mean of the values
    q = torch.randn((1, 4, dim), generator=gen, device="cuda").bfloat16()
    for scale in (-0.3, 1e-30):
        y = cache.kv.attend(q, batch, scale=scale, dtype=torch.float32)
        check_attended(y, None, reference(cache, offsets, lens, q, True, scale), torch.float16)
    # rows that are not finite stay in their rows
    q[0, 1, 3] = math.nan
    q[0, 2, 4] = math.inf
    y = cache.kv.attend(q, batch, dtype=torch.float32)
    assert bool(torch.isnan(y[0, 1]).all()) and bool(torch.isnan(y[0, 2]).any())
    z = cache.kv.attend(q[:, [0, 0, 0, 3]].contiguous(), batch, dtype=torch.float32)
    assert bool(torch.isfinite(y[0, [0, 3]]).all()) and torch.equal(y[0, 3], z[0, 3])


@gpu
def test_values_of_every_size(hrb):
    """Scales from the smallest to the largest, in one head and along a sequence."""
    dim, n = 128, 336
    cache = Cache(hrb, None, [n], 16, 1, dim, torch.float16)
    gen = torch.Generator(device="cuda").manual_seed(8)
    cache.random(gen)
    place = torch.arange(n, device="cuda")
    at = (cache.table[0, place // 16].long(), place % 16)
    cache.parts[3][at] = torch.stack([(place * a) % 168 for a in (1, 5, 11, 13)], -1).to(torch.uint8)[:, None]
    batch, offsets = batch_of(hrb, [1], cache)
    q = torch.randn((1, 8, dim), generator=gen, device="cuda").half()
    for out in (torch.float32, torch.float16):
        y = cache.kv.attend(q, batch, dtype=out)
        check_attended(y, None, reference(cache, offsets, [n], q, True), torch.float16, n * 2.0**-32 * 420)
    cache.parts[2][at] = cache.parts[3][at]
    for small in (167, 40, 0):  # keys of every size too, then small ones alone
        cache.parts[2][at] = cache.parts[2][at].clamp(max=small)
        y = cache.kv.attend(q, batch, dtype=torch.float32)
        check_attended(y, None, reference(cache, offsets, [n], q, True), torch.float16, n * 2.0**-32 * 420)


@gpu
def test_rows_behind_the_last_sequence_and_calls_of_nothing(hrb):
    gen = torch.Generator(device="cuda").manual_seed(6)
    cache = Cache(hrb, gen, [30, 40], 16, 2, 64, torch.bfloat16).random(gen)
    batch, offsets = batch_of(hrb, [1, 1], cache)
    q = torch.randn((5, 4, 64), generator=gen, device="cuda").bfloat16()
    out, lse = torch.full((5, 4, 64), 7.0, device="cuda"), torch.full((5, 4), 7.0, device="cuda")
    cache.kv.attend(q, batch, out=out, lse=lse)
    assert bool((out[2:] == 7).all()) and bool((lse[2:] == 7).all())
    check_attended(out[:2], lse[:2], reference(cache, offsets, [30, 40], q[:2], True), torch.float16)
    assert cache.kv.attend(q[:0], batch).shape == (0, 4, 64)
    k = q[:0, :2].contiguous()
    assert cache.kv.append(k, k, batch, q=q[:0]).shape == (0, 4, 64)
    assert cache.kv.read(batch, 0)[0].shape == (0, 2, 64)


@gpu
def test_a_sequence_longer_than_32_bits_of_bytes(hrb):
    """Page offsets past 2^32 bytes: one page far up in a pool of 5 GB (the rest is never read)."""
    page, kvh, dim, pages = 64, 8, 256, 80000
    codes = [torch.empty((pages, kvh, page, dim // 2), dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
    scales = [torch.empty((pages, kvh, page, 4), dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
    kv = hrb.QuantKV(*codes, *scales)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn((70, n, dim), generator=gen, device="cuda").bfloat16() for n in (kvh, kvh, kvh))
    table = i32([[pages - 1, 3]])
    batch = hrb.KVBatch(i32([0, 70]), i32([70]), table)
    kv.append(k, v, batch)
    back = kv.read(batch, 70, dtype=torch.float32)
    for x, y in zip((k, v), back):
        code, byte = encode64(x)
        value = ((code.double() - 8).unflatten(-1, (4, -1)) * all_scales()[byte.long()][..., None]).flatten(-2)
        assert torch.equal(y.double().cpu(), value)
    one = hrb.KVBatch(i32([0, 1]), i32([70]), table)
    y = kv.attend(q[-1:], one, dtype=torch.float32)
    pools = [torch.zeros((2, page, kvh, dim), dtype=torch.float64) for _ in range(2)]
    for p, x in zip(pools, back):
        p.view(-1, kvh, dim)[:70] = x.double().cpu()
    check_attended(y, None, attend64(q[-1:], *pools, [0, 1], [70], i32([[0, 1]]), dim**-0.5, True), torch.float16)


# ------------------------------------------------------------------ as they are used

@gpu
def test_prompts_then_captured_single_tokens(hrb):
    """Norm, rotation, append and attention of prompts, then steps from a graph, against 64 bits."""
    kvh, heads, dim, rotary, page, lens, steps = 2, 8, 128, 64, 16, [37, 5, 64], 6
    gen = torch.Generator(device="cuda").manual_seed(11)
    final = [n + steps for n in lens]
    cache = Cache(hrb, gen, final, page, kvh, dim, torch.bfloat16)
    scratch = hrb.PagedKV(*(torch.zeros(cache.parts[0].shape[:3] + (dim,), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    rope, qw, kw = hrb.Rope(freqs(rotary // 2)), weight(gen, dim), weight(gen, dim)
    inv, axis = freqs(rotary // 2), [0] * (rotary // 2)
    every = {name: rows(gen, (sum(final), n, dim), torch.float32) for name, n in (("q", heads), ("k", kvh), ("v", kvh))}
    starts = [sum(final[:i]) for i in range(3)]
    place = torch.cat([torch.arange(n) for n in final])[None]
    turned = {n: rotate64(norm64(every[n], w), place, inv, axis, False) for n, w in (("q", qw), ("k", kw))}

    def stored(x):
        code, byte = encode64(x)
        return ((code.double() - 8).unflatten(-1, (4, -1)) * all_scales()[byte.long()][..., None]).flatten(-2)

    kk, vv = stored(turned["k"]), stored(every["v"])

    def want(s, at):
        q = turned["q"][starts[s] + at].view(kvh, heads // kvh, dim)
        k, v = (x[starts[s]:starts[s] + at + 1].transpose(0, 1) for x in (kk, vv))
        return torch.softmax(q @ k.transpose(1, 2) / dim**0.5, -1).matmul(v).reshape(heads, dim)

    def call(x, batch, pos, dtype=None):
        q = cache.kv.append(x["k"], x["v"], batch, rope=rope, pos=pos, q=x["q"], q_norm=qw, k_norm=kw)
        return cache.kv.attend(q, batch, dtype=dtype, through=scratch)

    pick = torch.cat([torch.arange(n) + st for n, st in zip(lens, starts)]).cuda()
    batch, offsets = batch_of(hrb, lens, cache, lens)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)[None].cuda()
    y = call({n: x[pick] for n, x in every.items()}, batch, pos)
    # queries and weights in bf16: 2^-9 of scores up to 40 and of the values, rounded once each
    near = lambda a, b: float((a.double().cpu() - b).norm() / b.norm()) <= 2.0**-5  # noqa: E731
    for s, n in enumerate(lens):
        assert near(y[offsets[s]:offsets[s + 1]], torch.stack([want(s, at) for at in range(n)]))

    x = {n: torch.zeros((3,) + t.shape[1:], device="cuda") for n, t in every.items()}
    one, _ = batch_of(hrb, [1, 1, 1], cache, [n + 1 for n in lens])
    pos = i32([lens])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(x, one, pos)  # (its rows are overwritten by the first step)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x, one, pos, torch.float32)
        one.kv_lens += 1
        pos += 1
    for i in range(steps):
        at = torch.tensor([st + n + i for st, n in zip(starts, lens)], device="cuda")
        for n in x:
            x[n].copy_(every[n][at])
        graph.replay()
        for s, n in enumerate(lens):
            assert near(out[s], want(s, n + i)), (i, s)
    assert cache.kv.get_error() == hrb.BITLIN_OK


@gpu
def test_other_streams_and_a_shared_workspace(hrb):
    case = ([3000, 700, 1], [1, 1, 1], 16, 2, 6, 256, torch.bfloat16, torch.float32, True, "heads")
    cache, batch, offsets, q, y, _ = attended(hrb, case)
    other = hrb.QuantKV(*cache.parts, dtype=torch.bfloat16, share=cache.kv)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    z = other.attend(q, batch, dtype=torch.float32, stream=stream)
    w = torch.empty_like(z)
    other.attend(q, batch, out=w, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(y, w)
    k = torch.randn((3, 2, 256), device="cuda").bfloat16()
    stream.wait_stream(torch.cuda.current_stream())
    other.append(k, k, batch, stream=stream)
    a, b = other.read(batch, 3, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and bool((a != 0).any())
    cache.kv.close()
    assert torch.equal(other.attend(q, batch, dtype=torch.float32), other.attend(q, batch, dtype=torch.float32))
    with pytest.raises(ValueError):
        cache.kv.attend(q, batch)


@gpu
def test_layer_example_with_norms_over_4_bits(hrb):
    """Prompts and captured single-token steps of the example's layer, its projections taken as given."""
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
    import attention_layer as example

    lens, steps = [70, 1, 133], 3
    layer, table, inputs, outputs = example.serve(lens, steps, bits=4, norms=True)
    pairs = example.ROTARY // 2
    freq, axis = torch.tensor([1e7 ** (-i / pairs) for i in range(pairs)]).tolist(), [i % 3 for i in range(pairs)]  # (as f32)
    past = [0] * len(lens)
    for part, x in enumerate(inputs):
        new = lens if part == 0 else [1] * len(lens)
        past = [a + b for a, b in zip(past, new)]
        batch, pos = example.make_batch(new, past, table)
        q, gate, k, v = layer.project(x)
        # what the cache holds of the new rows is what their 64-bit values come to
        turned = rotate64(norm64(k, layer.norms["k_norm"]), pos, freq, axis, False)
        for got, want in zip(layer.cache.read(batch, sum(new), dtype=torch.float32), (turned, v)):
            code, byte = encode64(want)
            assert torch.equal(got.double().cpu(), ((code.double() - 8).unflatten(-1, (4, -1)) * all_scales()[byte.long()][..., None]).flatten(-2))
        q = layer.rope.apply(q, pos, dtype=torch.bfloat16, norm=layer.norms["q_norm"])
        a = layer.cache.attend(q, batch, dtype=torch.float32, **layer.through)
        offsets = [sum(new[:i]) for i in range(len(new) + 1)]
        starts = [sum(past[:i]) for i in range(len(past) + 1)]
        kk, vv = layer.cache.read(hrb.KVBatch(i32(starts), i32(past), table), starts[-1], dtype=torch.float32)
        # pages of one slot, in the order that the rows were read in
        places = torch.full((len(past), max(past)), -1)
        for s, n in enumerate(past):
            places[s, :n] = torch.arange(starts[s], starts[s + 1])
        ref = attend64(q, kk[:, None], vv[:, None], offsets, past, places, example.DIM**-0.5, True)
        check_attended(a, None, ref, torch.bfloat16 if part == 0 else torch.float16)
        again = layer.out((a * torch.sigmoid(gate)).view(-1, example.HEADS * example.DIM))
        assert torch.equal(again, outputs[part])


# ------------------------------------------------------------------ refusals

def test_the_c_abi_refuses_without_a_device(hrb):
    lib = hrb.lib()
    h, p = ctypes.c_void_p(), 4096
    from hadamard_rotated_binary_gb300._binding import HeadNorms, QuantPools

    good = dict(k=p, v=p, k_scale=p, v_scale=p, pages=4, page_size=16, kv_heads=2, head_dim=128, page_stride=2048, slot_stride=64,
                head_stride=1024, scale_page_stride=128, scale_slot_stride=4, scale_head_stride=64)
    assert lib.bitlin_kvq_create(None, ctypes.byref(QuantPools(**good)), 1) == hrb.BITLIN_EINVAL
    assert lib.bitlin_kvq_create(ctypes.byref(h), None, 1) == hrb.BITLIN_EINVAL
    for bad in (dict(k=0), dict(v=p + 8), dict(k_scale=p + 2), dict(v_scale=0), dict(pages=0), dict(page_size=0), dict(page_size=65537),
                dict(kv_heads=0), dict(kv_heads=4097), dict(head_dim=80), dict(head_dim=512), dict(page_stride=0), dict(slot_stride=24),
                dict(head_stride=-16), dict(scale_page_stride=2), dict(scale_slot_stride=0), dict(scale_head_stride=1 << 39)):
        assert lib.bitlin_kvq_create(ctypes.byref(h), ctypes.byref(QuantPools(**{**good, **bad})), 1) == hrb.BITLIN_EINVAL, bad
    assert lib.bitlin_kvq_create(ctypes.byref(h), ctypes.byref(QuantPools(**good)), 0) == hrb.BITLIN_EINVAL
    assert h.value is None
    norms = HeadNorms(p, p, 1e-6)
    assert lib.bitlin_kvq_append(None, None, 1, None, None, None, None, None, 1, None, ctypes.byref(norms), None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_kv_append_normed(None, None, 1, None, None, None, None, None, 1, None, ctypes.byref(norms), None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_kvq_read(None, None, 1, None, None, None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_kvq_attend(None, None, 1, None, 1, 1.0, 1, None, None, None, 0, None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_rope_apply_normed(None, None, 1, 1, 64, None, p, 1e-6, None, None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_rope_gradient(None, None, None, 1, 1, 64, None, p, 1e-6, None, p, p, 1 << 20, None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_kvq_share(None, None) == hrb.BITLIN_EINVAL and lib.bitlin_kvq_get_error(None) == hrb.BITLIN_EINVAL
    assert lib.bitlin_kvq_destroy(None) == hrb.BITLIN_OK and lib.bitlin_kvq_cuda_error(None) == 0
    assert lib.bitlin_rope_gradient_scratch(1, 1, 257) == 0 and lib.bitlin_rope_gradient_scratch(-1, 1, 64) == 0
    assert lib.bitlin_rope_gradient_scratch(10, 4, 64) >= 64 * 4


@gpu
def test_refusals(hrb):
    rope, w = hrb.Rope(freqs(16)), torch.ones(64, device="cuda")
    x, pos = torch.randn((3, 2, 64), device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    for norm in (w.half(), w[:32], w.cpu(), torch.ones((1, 64), device="cuda"), torch.ones(128, device="cuda")[::2]):
        with pytest.raises(ValueError):
            rope.apply(x, pos, norm=norm)
        with pytest.raises(ValueError):
            rope.gradient(x, x, pos, norm)
    with pytest.raises(ValueError):
        rope.apply(x, pos, norm=w, inverse=True)
    for eps in (-1.0, math.nan, math.inf):
        with pytest.raises(hrb.BitlinError):
            rope.apply(x, pos, norm=w, eps=eps)
    wide = torch.randn((3, 2, 264), device="cuda")
    with pytest.raises(hrb.BitlinError):
        rope.apply(wide, pos, norm=torch.ones(264, device="cuda"))
    with pytest.raises(ValueError):
        rope.gradient(x[:2], x, pos, w)
    with pytest.raises(ValueError):
        rope.gradient(x, x, pos, None)
    with pytest.raises(hrb.BitlinError):
        rope.gradient(x, x, pos, w, dx=torch.empty_like(x, dtype=torch.float16))
    pools = hrb.QuantKV.pools(4, 16, 2, 64)
    for bad in ((pools[0].int(), *pools[1:]), (pools[0], pools[1][:3], *pools[2:]), (*pools[:3], pools[3].contiguous()),
                (pools[0].cpu(), *pools[1:]), (*pools[:2], pools[0], pools[1])):
        with pytest.raises(ValueError):
            hrb.QuantKV(*bad)
    with pytest.raises(ValueError):
        hrb.QuantKV(*pools, dtype=torch.float32)
    with pytest.raises(hrb.BitlinError):
        hrb.QuantKV(*hrb.QuantKV.pools(4, 16, 2, 80))
    kv = hrb.QuantKV(*pools)
    with pytest.raises(AttributeError):
        kv.k = pools[0].clone()
    batch = hrb.KVBatch(i32([0, 3]), i32([3]), i32([[1]]))
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    with pytest.raises(hrb.BitlinError):
        kv.attend(q.half(), batch)
    with pytest.raises(hrb.BitlinError):
        kv.attend(q[:, :3], batch)
    with pytest.raises(hrb.BitlinError):
        kv.attend(q, batch, dtype=torch.float16)
    with pytest.raises(hrb.BitlinError):
        kv.attend(q, batch, scale=math.nan)
    with pytest.raises(ValueError):
        kv.attend(torch.randn((3, 4, 128), device="cuda").bfloat16(), batch)
    for shape, dtype in (((5, 16, 2, 64), torch.bfloat16), ((4, 32, 2, 64), torch.bfloat16), ((4, 16, 2, 64), torch.float16)):
        other = hrb.PagedKV(*(torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2)))
        with pytest.raises(hrb.BitlinError):
            kv.attend(q, batch, through=other)
    with pytest.raises(ValueError):
        kv.append(q[:, :1], q[:, :1], batch)
    with pytest.raises(ValueError):
        kv.append(q[:, :2], q[:, :2], batch, k_norm=torch.ones(65, device="cuda"))
    with pytest.raises(ValueError):
        kv.read(batch, 3, k=torch.empty((3, 2, 32), device="cuda"))
    with pytest.raises(hrb.BitlinError):
        kv.read(batch, 3, k=torch.empty((3, 2, 64), device="cuda"), v=torch.empty((3, 2, 64), device="cuda").half())
    with pytest.raises(ValueError):
        kv.read(batch, -1)
    closed = hrb.Rope(freqs(16))
    closed.close()
    with pytest.raises(ValueError):
        kv.append(q[:, :2], q[:, :2], batch, rope=closed)
    assert kv.get_error() == hrb.BITLIN_OK


@gpu
def test_more_sequences_than_a_grid_has_rows(hrb):
    """70,000 sequences of 1 to 8 keys, through 16-bit pages and directly; a few of them compared."""
    seqs, page, dim, heads = 70000, 8, 64, 96
    gen = torch.Generator(device="cuda").manual_seed(12)
    parts = hrb.QuantKV.pools(seqs, page, 1, dim)
    kv = hrb.QuantKV(*parts, dtype=torch.float16)
    lens = torch.arange(seqs, dtype=torch.int32, device="cuda") % 8 + 1
    table = torch.randperm(seqs, generator=gen, device="cuda").to(torch.int32)[:, None].contiguous()
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0).to(torch.int32)])
    k, v = (torch.randn((int(offsets[-1]), 1, dim), generator=gen, device="cuda").half() for _ in range(2))
    every = hrb.KVBatch(offsets, lens, table)
    kv.append(k, v, every)
    back = kv.read(every, k.shape[0], dtype=torch.float32)
    one = hrb.KVBatch(torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), lens, table)
    q = torch.randn((seqs, heads, dim), generator=gen, device="cuda").half()
    through = hrb.PagedKV(*(torch.empty((seqs, page, 1, dim), dtype=torch.float16, device="cuda") for _ in range(2)))
    outs = [kv.attend(q, one, through=t) for t in (None, through)]
    for s in (0, 7, 65534, 65535, 65536, 69999):
        at = slice(int(offsets[s]), int(offsets[s + 1]))
        kk, vv = (x[at, 0].double().cpu() for x in back)
        want = torch.softmax(q[s].double().cpu() @ kk.t() / dim**0.5, -1) @ vv
        for y in outs:  # weights and output in f16, values up to 4
            assert bool(((y[s].double().cpu() - want).abs() <= 2 * 2.0**-11 * 4).all())
    assert kv.get_error() == hrb.BITLIN_OK


@gpu
@pytest.mark.parametrize("dim", [64, 256])
def test_long_sums_of_f32_outputs_are_rounded_not_truncated(hrb, dim):
    """The mean of 65,536 positive values, by more items than CTAs, so that each is summed in one
    place: 700 to 1,400 additions of 16 keys each, rounded at random by 2^-25 of the sum at most,
    are off by 2^-20 together; truncated ones would be by 2^-14."""
    n, seqs, page = 65536, 400, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    parts = hrb.QuantKV.pools(n // page, page, 1, dim)  # all sequences read the same pages
    for p in parts[:2]:
        p.copy_(17 * torch.randint(9, 16, p.shape, generator=gen, device="cuda"))
    for p in parts[2:]:
        p.copy_(torch.randint(96, 104, p.shape, generator=gen, device="cuda"))
    kv = hrb.QuantKV(*parts)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].repeat(seqs, 1).contiguous()
    batch = hrb.KVBatch(torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), i32([n] * seqs), table)
    y = kv.attend(torch.zeros((seqs, 2, dim), dtype=torch.bfloat16, device="cuda"), batch, dtype=torch.float32)
    want = decode64(parts[1], parts[3]).mean((0, 1, 2))
    assert float((y.double().cpu() - want).norm() / (want.norm() * (2 * seqs) ** 0.5)) <= 2.0**-20


@gpu
def test_as_many_heads_as_a_row_tile_and_more(hrb):
    """Groups of up to 128 query heads, tokens that straddle row tiles, ragged new tokens."""
    for group, new, dim in ((128, [1, 1], 256), (127, [2, 1], 128), (5, [7, 1], 256), (24, [1, 1], 128), (25, [1, 3], 64)):
        case = ([200, 77], new, 16, 2, group, dim, torch.bfloat16, torch.float32, True, "heads")
        cache, _, offsets, q, y, lse = attended(hrb, case)
        check_attended(y, lse, reference(cache, offsets, case[0], q, True), torch.float16)

"""A cache in 4 bits as measured cases: norms of queries and keys with the position rotation in the
same pass (and its gradient), writing keys and values to a paged cache in 4 bits and reading them
back, and attention over that cache.

Each case names one call (for "store" the two that belong together) with its sizes and types.
``run`` makes it: in the plain form (elementary torch operations, rounded once at the end) where
``own`` is false, through the library's entry points where it is true.

  turn    x [T][H][D] -> rotated by its positions, after each head's norm: n = x / sqrt(mean(x^2) +
          eps) * weight.  For pair i of a head: (a, b) -> (a cos t - b sin t, b cos t + a sin t),
          t = pos[axis[i]][token] * inv_freq[i]; the pair is (i, i + R/2) within the first R =
          rotary elements, or (2i, 2i + 1) where "adjacent"; elements past R are not rotated.
  slope   the gradient of turn: from that of its output to those of x and of the weight.
  store   k, v [T][Hkv][D] of the new tokens go to their sequences' pages in 4 bits, k after its
          norm and rotation; q [T][H][D] is normed and rotated to the cache's type.  The new rows
          are then read back: they come as the values that the codes stand for.
  attend  q [T][H][D] of the new tokens against every key of their sequence in the 4-bit cache
          (causal: up to their own position); query head h reads key head h // (H / Hkv).

The 4-bit form: a head's D elements are four groups with a scale each.  Scales have 5 bits of
exponent and 3 of significand (a float16 without sign and last 7 bits), at most 60: a group's is
its largest magnitude / 7, rounded to the nearest one (ties to even).  A value is stored as
clamp(round(x / scale), -7, 7) + 8, element 2i in the low and 2i + 1 in the high half of byte i.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
GROUPS = 4
SCALE_MAX = 60.0


# ------------------------------------------------------------------ cases

def _turn(name, tokens, heads, dim, rotary, axes, src, dst, adjacent=False):
    return {"op": "turn", "name": name, "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary, "axes": axes,
            "src": src, "dst": dst, "adjacent": adjacent}


def _slope(name, tokens, heads, dim, rotary, axes, src, dst, adjacent=False):
    return {**_turn(name, tokens, heads, dim, rotary, axes, src, dst, adjacent), "op": "slope"}


def _store(name, seqs, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, rotary, axes, page, src, cache,
           adjacent=False):
    return {"op": "store", "name": name, "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rotary": rotary, "axes": axes,
            "page": page, "src": src, "cache": cache, "adjacent": adjacent}


def _attend(name, seqs, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, page, cache, dst, causal=True,
            lse=False):
    return {"op": "attend", "name": name, "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache,
            "dst": dst, "causal": causal, "lse": lse}


def listed():
    return [
        # one decoded token's queries, 24 heads of 256 with 64 rotated, as the projection leaves them (f32)
        _turn("turn_step", 1, 24, 256, 64, 3, "f32", "bf16"),
        # the queries of several prompts, whole heads rotated
        _turn("turn_prompts", 8191, 32, 128, 128, 1, "bf16", "bf16", adjacent=True),
        # the gradient of a training sequence, one token past 4096
        _slope("slope_sequence", 4097, 24, 256, 64, 3, "f32", "f32"),
        # the gradient of a short sequence's keys in 16 bits
        _slope("slope_keys", 777, 8, 80, 80, 2, "bf16", "bf16"),
        # one decoded token: its query, key and value
        _store("store_step", 1, 1, 1, 4100, 4100, 24, 4, 256, 64, 3, 64, "f32", "bf16"),
        # a serving batch of single tokens at ragged positions, small pages
        _store("store_batch", 64, 1, 1, 17, 4000, 24, 4, 256, 64, 3, 16, "f32", "bf16"),
        # prompts of several users in one call
        _store("store_prompts", 3, 1300, 4096, 0, 0, 32, 8, 128, 128, 1, 128, "bf16", "f16", adjacent=True),
        # one decoded token early in a conversation: latency counts
        _attend("attend_step_short", 1, 1, 1, 776, 776, 24, 4, 256, 64, "bf16", "f32"),
        # one decoded token at 128K tokens: the cache is read once
        _attend("attend_step_long", 1, 1, 1, 131071, 131071, 24, 4, 256, 64, "bf16", "f32"),
        # a serving batch of single tokens over ragged contexts
        _attend("attend_batch", 64, 1, 1, 100, 8000, 24, 4, 256, 16, "bf16", "bf16"),
        # drafted tokens of 16 sequences checked together
        _attend("attend_draft", 16, 5, 5, 1000, 6000, 32, 8, 128, 32, "f16", "f16", lse=True),
        # a chunk of a long prompt: 2048 new tokens, 32768 in the cache with them
        _attend("attend_chunk", 1, 2048, 2048, 30720, 30720, 24, 4, 256, 64, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("turn", "slope", "store", "store", "attend", "attend", "attend"))
    dim = rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 8))
    page = rng.choice((16, 32, 48, 64, 128))
    cache = rng.choice(("bf16", "f16"))
    axes = rng.choice((1, 2, 3))
    if op in ("turn", "slope"):
        dim = rng.choice((dim, 80))
        rotary = rng.choice((dim, dim // 2, dim // 4)) // 4 * 4
        src = rng.choice(("f32", "bf16", "f16"))
        tokens = min(_log(rng, 1, 16000), (1 << 25) // (heads * dim))
        case = (_turn if op == "turn" else _slope)("", tokens, heads, dim, rotary, axes, src,
                                                   rng.choice((src, "f32", "bf16")), rng.random() < 0.3)
        return {k: v for k, v in case.items() if k != "name"}
    rotary = rng.choice((dim, dim // 2, dim // 4))
    seqs = _log(rng, 1, 64)
    if op == "store":
        new = _log(rng, 1, max(1, 8000 // seqs))
        past = _log(rng, 1, 4000)
        case = _store("", seqs, max(1, new // 3), new, past // 5, past, heads, kv_heads, dim, rotary, axes, page,
                      rng.choice(("f32", "bf16", "f16")), cache, rng.random() < 0.3)
    else:
        new = 1 if rng.random() < 0.6 else _log(rng, 2, max(2, 4000 // seqs))
        # the padded score matrix of the plain form stays under 2^30 values
        most = max(1, min(120000 // seqs, (1 << 30) // (seqs * new * heads)) - new)
        past = _log(rng, 1, most)
        case = _attend("", seqs, max(1, new // 3), new, past // 5, past, heads, kv_heads, dim, page, cache,
                       rng.choice((cache, cache, "f32")), rng.random() < 0.8, rng.random() < 0.3)
    return {k: v for k, v in case.items() if k != "name"}


def _spread(lo, hi, n, by):
    """n whole numbers from lo to hi, spread without a pattern that sizes would share; hi is among them."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((i * by) % 1.0)) for i in range(n)]


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence."""
    new = _spread(case["new_lo"], case["new_hi"], case["seqs"], 0.6180339887)
    past = _spread(case["past_lo"], case["past_hi"], case["seqs"], 0.7548776662)
    return new, [n + p for n, p in zip(new, past)]


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(TYPES[dtype])


def _projected(gen, shape, dtype):
    """What a projection leaves: some of a head's channels stand out in every token."""
    loud = torch.exp(0.5 * torch.randn(shape[1:], generator=gen, device="cuda"))
    return (torch.randn(shape, generator=gen, device="cuda") * loud).to(TYPES[dtype])


def _weight(gen, dim):
    return torch.exp(0.3 * torch.randn((dim,), generator=gen, device="cuda"))


def _positions(case, gen, tokens, first=None):
    """int32 [axes][tokens]: running positions on the first axis, a grid's rows and columns on the others."""
    t = torch.arange(tokens, device="cuda") if first is None else first
    start = int(torch.randint(0, 1000, (1,), generator=gen, device="cuda"))
    rows = [t + start, t // 42 % 24 + start, t % 42 + start]
    return torch.stack(rows[: case["axes"]]).to(torch.int32).contiguous()


def _frequencies(case):
    """(inv_freq, axis) of each rotated pair: base 10^7, the axes taken in turn."""
    pairs = case["rotary"] // 2
    inv_freq = [float(torch.tensor(1e7 ** (-i / pairs), dtype=torch.float32)) for i in range(pairs)]
    return inv_freq, [i % case["axes"] for i in range(pairs)]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"] != "attend":
        inv_freq, axis = _frequencies(case)
        s["inv_freq"] = torch.tensor(inv_freq, dtype=torch.float32, device="cuda")
        s["axis"] = torch.tensor(axis, dtype=torch.int64, device="cuda")
        s["weight"] = _weight(gen, case["dim"])
    if case["op"] in ("turn", "slope"):
        s["x"] = _projected(gen, (case["tokens"], case["heads"], case["dim"]), case["src"])
        s["pos"] = _positions(case, gen, case["tokens"])
        if case["op"] == "slope":
            s["dy"] = _normal(gen, (case["tokens"], case["heads"], case["dim"]), case["dst"])
        return s
    new, total = _lengths(case)
    tokens, page = sum(new), case["page"]
    pages = [-(-n // page) for n in total]
    spare = 3
    order = torch.randperm(sum(pages) + spare, generator=gen, device="cuda").to(torch.int32)
    width = max(pages)
    at = torch.tensor([sum(pages[:b]) for b in range(len(pages))], device="cuda")
    index = at[:, None] + torch.arange(width, device="cuda")[None, :]
    held = torch.arange(width, device="cuda")[None, :] < torch.tensor(pages, device="cuda")[:, None]
    s["table"] = torch.where(held, order[index.clamp(max=order.numel() - 1)], torch.zeros_like(order[:1])).contiguous()
    offsets = [sum(new[:b]) for b in range(len(new) + 1)]
    s["q_offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    s["kv_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    # [pages][page_size][kv_heads][...], the slots of a head side by side in memory
    shape = (order.numel(), case["kv_heads"], page, case["dim"])
    for name in ("k", "v"):
        if case["op"] == "attend":
            codes, scales = _encode(_normal(gen, shape, "f32"), torch.float32)
        else:
            codes = torch.zeros(shape[:3] + (case["dim"] // 2,), dtype=torch.uint8, device="cuda")
            scales = torch.zeros(shape[:3] + (GROUPS,), dtype=torch.uint8, device="cuda")
        s[name + "_pool"], s[name + "_scale"] = codes.transpose(1, 2), scales.transpose(1, 2)
    if case["op"] == "store":
        s["k"] = _projected(gen, (tokens, case["kv_heads"], case["dim"]), case["src"])
        s["v"] = _normal(gen, (tokens, case["kv_heads"], case["dim"]), case["src"])
        s["q"] = _projected(gen, (tokens, case["heads"], case["dim"]), case["src"])
        s["q_weight"] = _weight(gen, case["dim"])
        place = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)])
        s["pos"] = _positions(case, gen, tokens, place)
    else:
        # scores with a spread of about 2: some keys stand out, none takes all
        s["q"] = _normal(gen, (tokens, case["heads"], case["dim"]), case["cache"], 2.0)
        s["lse"] = torch.empty((tokens, case["heads"]), dtype=torch.float32, device="cuda") if case["lse"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import hadamard_rotated_binary_gb300 as hrb

        if case["op"] != "attend":
            inv_freq, axis = _frequencies(case)
            s["rope"] = hrb.Rope(inv_freq, axis, adjacent=case["adjacent"])
        if case["op"] in ("store", "attend"):
            s["cache"] = hrb.QuantKV(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], dtype=TYPES[case["cache"]])
            s["batch"] = hrb.KVBatch(s["q_offsets"], s["kv_lens"], s["table"])
        if case["op"] == "attend" and case["new_hi"] > 1:
            # a 16-bit cache of the same pages, which the layers of a model share: prompts go through it
            shape = s["k_pool"].shape[:3] + (case["dim"],)
            s["through"] = hrb.PagedKV(*(torch.empty(shape, dtype=TYPES[case["cache"]], device="cuda") for _ in range(2)))
    return s


# ------------------------------------------------------------------ one pass

def _encode(x, compute=torch.float64):
    """(codes, scales) of x [..., D].  64 bits: a value next to a border between two codes goes to the right one."""
    g = x.to(compute).unflatten(-1, (GROUPS, -1))
    want = (g.abs().amax(-1, keepdim=True) / 7).clamp_(max=SCALE_MAX)
    step = torch.exp2((torch.frexp(want)[1] - 4).clamp_(min=-17).to(compute))
    scale = torch.round(want / step) * step
    code = torch.where(scale > 0, torch.round(g / scale), 0.0).clamp_(-7, 7).add_(8).to(torch.uint8).flatten(-2)
    bits = scale.squeeze(-1).to(torch.float16).view(torch.int16) >> 7
    return code[..., 0::2] | code[..., 1::2] << 4, bits.to(torch.uint8)


def _decode(codes, scales):
    """float32 [..., D]: the values that the codes stand for (exact)."""
    value = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    scale = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (value.unflatten(-1, (GROUPS, -1)) * scale[..., None]).flatten(-2)


def _plain_rotate(x, pos, inv_freq, axis, adjacent, inverse=False):
    """[T][H][D] in x's type.  The angles are formed in 64 bits: at position 10^5 a 32-bit product is off by 2^-8."""
    r = 2 * inv_freq.numel()
    angle = pos.to(torch.float64)[axis].t() * inv_freq.to(torch.float64)
    cos, sin = torch.cos(angle).to(x.dtype)[:, None, :], torch.sin(angle).to(x.dtype)[:, None, :]
    sin = -sin if inverse else sin
    y = x.clone()
    first = slice(0, r, 2) if adjacent else slice(0, r // 2)
    second = slice(1, r, 2) if adjacent else slice(r // 2, r)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _plain_norm(x):
    """(x / rms, 1 / rms) of each head."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_turn(s, x, weight, compute=torch.float32):
    n, _ = _plain_norm(x.to(compute))
    return _plain_rotate(n * weight.to(compute), s["pos"], s["inv_freq"], s["axis"], s["case"]["adjacent"])


def _plain_slope(s, case):
    n, r = _plain_norm(s["x"].float())
    g = _plain_rotate(s["dy"].float(), s["pos"], s["inv_freq"], s["axis"], case["adjacent"], inverse=True)
    h = g * s["weight"]
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (g * n).double().sum((0, 1)).float()}


def _sequence_of(q_offsets, tokens):
    return torch.bucketize(torch.arange(tokens, device=q_offsets.device, dtype=q_offsets.dtype), q_offsets, right=True) - 1


def _plain_store(s, case):
    dtype, page, tokens = TYPES[case["cache"]], case["page"], s["k"].shape[0]
    seq = _sequence_of(s["q_offsets"], tokens)
    place = s["kv_lens"][seq] - s["q_offsets"][seq + 1] + torch.arange(tokens, device="cuda")
    pages, slots = s["table"][seq, place // page].long(), place % page
    rows = {"k": _plain_turn(s, s["k"], s["weight"], torch.float64), "v": s["v"]}
    out = {"q": _plain_turn(s, s["q"], s["q_weight"]).to(dtype)}
    for name, x in rows.items():
        codes, scales = _encode(x)
        s[name + "_pool"][pages, slots], s[name + "_scale"][pages, slots] = codes, scales
        out[name] = _decode(s[name + "_pool"][pages, slots], s[name + "_scale"][pages, slots]).to(dtype)
    return out


def _plain_attend(s, case):
    q, offsets, lens = s["q"].float(), s["q_offsets"].long(), s["kv_lens"].long()
    tokens, heads, dim = q.shape
    seqs, kv_heads = lens.numel(), case["kv_heads"]
    group, most_new = heads // kv_heads, case["new_hi"]
    at = s["table"].long()
    k, v = (_decode(s[n + "_pool"][at].flatten(1, 2), s[n + "_scale"][at].flatten(1, 2)) for n in ("k", "v"))
    key = torch.arange(k.shape[1], device="cuda")
    held = key[None, :] < lens[:, None]
    v = torch.where(held[:, :, None, None], v, 0.0)
    new = offsets[1:] - offsets[:-1]
    row = torch.arange(most_new, device="cuda")
    qp = q[(offsets[:-1, None] + row).clamp(max=tokens - 1)].view(seqs, most_new, kv_heads, group, dim)
    qp = qp.permute(0, 2, 3, 1, 4).reshape(seqs, kv_heads, group * most_new, dim)
    score = torch.matmul(qp, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(dim)).view(seqs, kv_heads, group, most_new, -1)
    seen = held[:, None, :]
    if case["causal"]:
        seen = seen & (key <= (lens - new)[:, None, None] + row[:, None])
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).view(seqs, kv_heads, group, most_new, dim)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(seqs, most_new, heads, dim)
    lse = (top + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(seqs, most_new, heads)
    seq = _sequence_of(s["q_offsets"], tokens)
    at = torch.arange(tokens, device="cuda") - offsets[seq]
    return out[seq, at].to(TYPES[case["dst"]]), lse[seq, at]


def run(s):
    case = s["case"]
    if case["op"] == "turn":
        if own:
            return s["rope"].apply(s["x"], s["pos"], dtype=TYPES[case["dst"]], norm=s["weight"], eps=EPS)
        return _plain_turn(s, s["x"], s["weight"]).to(TYPES[case["dst"]])
    if case["op"] == "slope":
        if own:
            dx, dweight = s["rope"].gradient(s["dy"], s["x"], s["pos"], s["weight"], eps=EPS)
            return {"dx": dx, "dweight": dweight}
        return _plain_slope(s, case)
    if case["op"] == "store":
        if own:
            q = s["cache"].append(s["k"], s["v"], s["batch"], rope=s["rope"], pos=s["pos"], q=s["q"],
                                  q_norm=s["q_weight"], k_norm=s["weight"], eps=EPS)
            k, v = s["cache"].read(s["batch"], s["k"].shape[0])
            return {"q": q, "k": k, "v": v}
        return _plain_store(s, case)
    if own:
        out, lse = s["cache"].attend(s["q"], s["batch"], causal=case["causal"], dtype=TYPES[case["dst"]], lse=s["lse"],
                                     through=s.get("through")), s["lse"]
    else:
        out, lse = _plain_attend(s, case)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def work(case):
    """Bytes of each input read once and each output written once; attention's flops over the visible pairs."""
    if case["op"] in ("turn", "slope"):
        n = case["tokens"] * case["heads"] * case["dim"]
        rest = 4 * case["axes"] * case["tokens"] + 4 * case["dim"]
        if case["op"] == "turn":
            return {"bytes": n * (SIZE[case["src"]] + SIZE[case["dst"]]) + rest, "flops": 8 * n}
        return {"bytes": n * (2 * SIZE[case["src"]] + SIZE[case["dst"]]) + rest + 4 * case["dim"], "flops": 14 * n}
    new, total = _lengths(case)
    tokens, rows = sum(new), 4 * (2 * case["seqs"] + 1)
    held = case["dim"] / 2 + GROUPS  # bytes of a head in the cache
    if case["op"] == "store":
        heads, kv = tokens * case["heads"] * case["dim"], tokens * 2 * case["kv_heads"]
        bytes_ = (heads + kv * case["dim"]) * (SIZE[case["src"]] + 2) + kv * held
        return {"bytes": bytes_ + 4 * (case["axes"] + 1) * tokens + rows + 8 * case["dim"],
                "flops": 8 * (heads + kv * case["dim"])}
    pairs = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in zip(new, total))
    bytes_ = sum(total) * case["kv_heads"] * held * 2 + sum(-(-t // case["page"]) for t in total) * 4 + rows
    bytes_ += tokens * case["heads"] * (case["dim"] * (2 + SIZE[case["dst"]]) + (4 if case["lse"] else 0))
    return {"bytes": bytes_, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ in 64 bits

def _complex_turn(x, pos, inv_freq, axis, adjacent, sign):
    """Rotation as a product of complex numbers, 64 bits."""
    r = 2 * len(inv_freq)
    head, rest = x[..., :r], x[..., r:]
    pairs = head.unflatten(-1, (-1, 2)) if adjacent else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turn = torch.stack([pos[a].double() * f for f, a in zip(inv_freq, axis)], -1) * sign
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(turn), turn)[:, None, :]
    z = torch.view_as_real(z)
    z = z.flatten(-2) if adjacent else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, rest], -1)


def _all_scales():
    """The 168 scales from 0 to 60, by their code."""
    return torch.tensor([math.ldexp((b & 7) + (8 if b >> 3 else 0), max(b >> 3, 1) - 18) for b in range(168)],
                        dtype=torch.float64, device="cuda")


def _stored(x):
    """What x [..., D] is once stored: nearest scale by search, nearest code by halves."""
    every = _all_scales()
    middles = (every[1:] + every[:-1]) / 2
    g = x.double().reshape(x.shape[:-1] + (GROUPS, -1))
    want = g.abs().max(-1, keepdim=True).values / 7.0
    b = torch.bucketize(want, middles)
    b = b + ((want == middles[b.clamp(max=middles.numel() - 1)]) & (b < middles.numel()) & (b % 2 == 1)).long()
    scale = every[b]
    t = torch.where(scale > 0, g / torch.where(scale > 0, scale, 1.0), 0.0)
    low = torch.floor(t)
    up = (t - low > 0.5) | ((t - low == 0.5) & (low.remainder(2) == 1))
    return (torch.clip(low + up.double(), -7, 7) * scale).reshape(x.shape)


def _exact_norm(x, weight):
    x = x.double()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "attend":
        inv_freq, axis = _frequencies(case)
        turned = lambda x, sign=1.0: _complex_turn(x, s["pos"], inv_freq, axis, case["adjacent"], sign)  # noqa: E731
    if case["op"] == "turn":
        return turned(_exact_norm(s["x"], s["weight"]))
    if case["op"] == "slope":
        x, w = s["x"].double(), s["weight"].double()
        g = turned(s["dy"].double(), -1.0)
        d = x.shape[-1]
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        dx = g * w / rms - x * (g * w * x).sum(-1, keepdim=True) / (d * rms ** 3)
        return {"dx": dx, "dweight": torch.einsum("thd,thd->d", g, x / rms)}
    if case["op"] == "store":
        return {"q": turned(_exact_norm(s["q"], s["q_weight"])), "k": _stored(turned(_exact_norm(s["k"], s["weight"]))),
                "v": _stored(s["v"])}
    new, total = _lengths(case)
    page, table = case["page"], s["table"].long()
    starts = [sum(new[:b]) for b in range(len(new))]
    out = torch.zeros((sum(new), case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    group, every = case["heads"] // case["kv_heads"], _all_scales()

    def held(name, b, place, head):
        at = (table[b, place // page], place % page)
        byte = s[name + "_pool"][at][:, head].long()
        code = torch.empty((byte.shape[0], case["dim"]), dtype=torch.float64, device="cuda")
        code[:, 0::2], code[:, 1::2] = byte % 16 - 8, byte // 16 - 8
        return code * every[s[name + "_scale"][at][:, head].long()].repeat_interleave(case["dim"] // GROUPS, -1)

    for b, (at, n, t) in enumerate(zip(starts, new, total)):
        place = torch.arange(t, device="cuda")
        for h in range(case["heads"]):
            if h % group == 0:
                k, v = held("k", b, place, h // group), held("v", b, place, h // group)
            logits = s["q"][at:at + n, h].double() @ k.t() / math.sqrt(case["dim"])
            if case["causal"]:
                logits += torch.triu(torch.full((n, t), -math.inf, dtype=torch.float64, device="cuda"), t - n + 1)
            out[at:at + n, h] = torch.softmax(logits, -1) @ v
            lse[at:at + n, h] = torch.logsumexp(logits, -1)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}

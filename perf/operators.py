"""The attention-side operators of the decoder as measured cases: rotary positions with several
axes, appending rotated keys and values to a paged cache, and attention of new tokens over that
cache.

Each case names one call with its sizes and types.  ``run`` makes that call: in the plain form
(elementary torch operations in 32 bits, rounded once at the end) where ``own`` is false, through
the library's entry points where it is true.

  rope    x [T][H][D] -> the same shape.  For pair i of a head: (a, b) -> (a cos t - b sin t,
          b cos t + a sin t), t = pos[axis[i]][token] * inv_freq[i]; the pair is (i, i + R/2)
          within the first R = rotary elements, or (2i, 2i + 1) where "adjacent"; elements past R
          pass through.  "inverse" rotates by -t (the gradient's direction).
  append  k, v [T][Hkv][D] of the new tokens go to their sequences' pages; k is rotated on the
          way, q [T][H][D] too (returned), all rounded to the cache's type.
  attend  q [T][H][D] of the new tokens against every key of their sequence in the paged cache
          (causal: up to their own position); query head h reads key head h // (H / Hkv).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases

def _rope(name, tokens, heads, dim, rotary, axes, src, dst, adjacent=False, inverse=False):
    return {"op": "rope", "name": name, "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary, "axes": axes,
            "src": src, "dst": dst, "adjacent": adjacent, "inverse": inverse}


def _append(name, seqs, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, rotary, axes, page, src, cache,
            adjacent=False):
    return {"op": "append", "name": name, "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
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
        _rope("rope_step", 1, 24, 256, 64, 3, "f32", "bf16"),
        # a video clip's patches in an image tower: time, height and width share an 80-wide head
        _rope("rope_video", 16128, 16, 80, 80, 3, "bf16", "bf16"),
        # the gradient of a training sequence's rotation, one token past 4096
        _rope("rope_gradient", 4097, 24, 256, 64, 3, "f32", "f32", inverse=True),
        # one decoded token: its query, key and value in one call
        _append("append_step", 1, 1, 1, 4100, 4100, 24, 4, 256, 64, 3, 64, "f32", "bf16"),
        # a serving batch of single tokens at ragged positions, small pages
        _append("append_batch", 64, 1, 1, 17, 4000, 24, 4, 256, 64, 3, 16, "f32", "bf16"),
        # prompts of several users in one call
        _append("append_prompts", 3, 1300, 4096, 0, 0, 32, 8, 128, 128, 1, 128, "bf16", "f16", adjacent=True),
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
        # whole prompts of several users, nothing in the cache before them
        _attend("attend_prompts", 4, 700, 4096, 0, 0, 32, 8, 128, 128, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend"))
    dim = rng.choice((64, 80, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 8))
    page = rng.choice((16, 32, 48, 64, 128))
    cache = rng.choice(("bf16", "f16"))
    rotary, axes = rng.choice((dim, dim // 2, dim // 4)) // 4 * 4, rng.choice((1, 2, 3))
    if op == "rope":
        src = rng.choice(("f32", "bf16", "f16"))
        tokens = min(_log(rng, 1, 16000), (1 << 25) // (heads * dim))
        return {k: v for k, v in _rope("", tokens, heads, dim, rotary, axes, src, rng.choice((src, "f32", "bf16")),
                                       rng.random() < 0.3, rng.random() < 0.3).items() if k != "name"}
    seqs = _log(rng, 1, 64)
    if op == "append":
        new = _log(rng, 1, max(1, 8000 // seqs))
        past = _log(rng, 1, 4000)
        case = _append("", seqs, max(1, new // 3), new, past // 5, past, heads, kv_heads, dim, rotary, axes, page,
                       rng.choice(("f32", "bf16", "f16")), cache, rng.random() < 0.3)
    else:
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 4000 // seqs))
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
    if case["op"] == "rope":
        s["x"] = _normal(gen, (case["tokens"], case["heads"], case["dim"]), case["src"])
        s["pos"] = _positions(case, gen, case["tokens"])
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
    shape = (order.numel(), page, case["kv_heads"], case["dim"])
    s["k_pool"] = _normal(gen, shape, case["cache"])
    s["v_pool"] = _normal(gen, shape, case["cache"])
    if case["op"] == "append":
        s["k"] = _normal(gen, (tokens, case["kv_heads"], case["dim"]), case["src"])
        s["v"] = _normal(gen, (tokens, case["kv_heads"], case["dim"]), case["src"])
        s["q"] = _normal(gen, (tokens, case["heads"], case["dim"]), case["src"])
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
        if case["op"] != "rope":
            s["cache"] = hrb.PagedKV(s["k_pool"], s["v_pool"])
            s["batch"] = hrb.KVBatch(s["q_offsets"], s["kv_lens"], s["table"])
    return s


# ------------------------------------------------------------------ one pass

def _plain_rotate(x, pos, inv_freq, axis, adjacent, inverse):
    """float32 [T][H][D].  The angles are formed in 64 bits: at position 10^5 a 32-bit product is off by 2^-8."""
    r = 2 * inv_freq.numel()
    angle = pos.to(torch.float64)[axis].t() * inv_freq.to(torch.float64)
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    sin = -sin if inverse else sin
    x = x.float()
    y = x.clone()
    first = slice(0, r, 2) if adjacent else slice(0, r // 2)
    second = slice(1, r, 2) if adjacent else slice(r // 2, r)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _sequence_of(q_offsets, tokens):
    return torch.bucketize(torch.arange(tokens, device=q_offsets.device, dtype=q_offsets.dtype), q_offsets, right=True) - 1


def _plain_append(s, case):
    dtype, page, tokens = TYPES[case["cache"]], case["page"], s["k"].shape[0]
    turn = lambda x: _plain_rotate(x, s["pos"], s["inv_freq"], s["axis"], case["adjacent"], False)  # noqa: E731
    seq = _sequence_of(s["q_offsets"], tokens)
    place = s["kv_lens"][seq] - s["q_offsets"][seq + 1] + torch.arange(tokens, device="cuda")
    pages, slots = s["table"][seq, place // page].long(), place % page
    s["k_pool"][pages, slots] = turn(s["k"]).to(dtype)
    s["v_pool"][pages, slots] = s["v"].to(dtype)
    return {"k": s["k_pool"], "v": s["v_pool"], "q": turn(s["q"]).to(dtype)}


def _plain_attend(s, case):
    q, offsets, lens = s["q"].float(), s["q_offsets"].long(), s["kv_lens"].long()
    tokens, heads, dim = q.shape
    seqs, kv_heads = lens.numel(), case["kv_heads"]
    group, most_new = heads // kv_heads, case["new_hi"]
    k, v = (p[s["table"].long()].flatten(1, 2).float() for p in (s["k_pool"], s["v_pool"]))
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
    if case["op"] == "rope":
        if own:
            return s["rope"].apply(s["x"], s["pos"], dtype=TYPES[case["dst"]], inverse=case["inverse"])
        return _plain_rotate(s["x"], s["pos"], s["inv_freq"], s["axis"], case["adjacent"], case["inverse"]).to(TYPES[case["dst"]])
    if case["op"] == "append":
        if own:
            q = s["cache"].append(s["k"], s["v"], s["batch"], rope=s["rope"], pos=s["pos"], q=s["q"])
            return {"k": s["k_pool"], "v": s["v_pool"], "q": q}
        return _plain_append(s, case)
    if own:
        out, lse = s["cache"].attend(s["q"], s["batch"], causal=case["causal"], dtype=TYPES[case["dst"]], lse=s["lse"]), s["lse"]
    else:
        out, lse = _plain_attend(s, case)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def work(case):
    """Bytes of each input read once and each output written once; attention's flops over the visible pairs."""
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * case["dim"] * (SIZE[case["src"]] + SIZE[case["dst"]]) + 4 * case["axes"] * case["tokens"],
                "flops": 3 * n * case["rotary"]}
    new, total = _lengths(case)
    tokens, rows = sum(new), 4 * (2 * case["seqs"] + 1)
    if case["op"] == "append":
        n = tokens * case["dim"] * (case["heads"] + 2 * case["kv_heads"])
        return {"bytes": n * (SIZE[case["src"]] + 2) + 4 * (case["axes"] + 1) * tokens + rows,
                "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    pairs = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in zip(new, total))
    bytes_ = sum(total) * case["kv_heads"] * case["dim"] * 4 + sum(-(-t // case["page"]) for t in total) * 4 + rows
    bytes_ += tokens * case["heads"] * (case["dim"] * (2 + SIZE[case["dst"]]) + (4 if case["lse"] else 0))
    return {"bytes": bytes_, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ in 64 bits

def _turned(x, pos, inv_freq, axis, adjacent, sign):
    """Rotation as a product of complex numbers, 64 bits."""
    r = 2 * len(inv_freq)
    x = x.double()
    head, rest = x[..., :r], x[..., r:]
    pairs = head.unflatten(-1, (-1, 2)) if adjacent else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turn = torch.stack([pos[a].double() * f for f, a in zip(inv_freq, axis)], -1) * sign
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(turn), turn)[:, None, :]
    z = torch.view_as_real(z)
    z = z.flatten(-2) if adjacent else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, rest], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "attend":
        inv_freq, axis = _frequencies(case)
    if case["op"] == "rope":
        return _turned(s["x"], s["pos"], inv_freq, axis, case["adjacent"], -1.0 if case["inverse"] else 1.0)
    new, total = _lengths(case)
    page, table = case["page"], s["table"].long()
    starts = [sum(new[:b]) for b in range(len(new))]
    if case["op"] == "append":
        k, v = s["k_pool"].double(), s["v_pool"].double()
        rotated = _turned(s["k"], s["pos"], inv_freq, axis, case["adjacent"], 1.0)
        for b, (at, n, t) in enumerate(zip(starts, new, total)):
            place = torch.arange(t - n, t, device="cuda")
            k[table[b, place // page], place % page] = rotated[at:at + n]
            v[table[b, place // page], place % page] = s["v"][at:at + n].double()
        return {"k": k, "v": v, "q": _turned(s["q"], s["pos"], inv_freq, axis, case["adjacent"], 1.0)}
    out = torch.zeros((sum(new), case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    for b, (at, n, t) in enumerate(zip(starts, new, total)):
        place = torch.arange(t, device="cuda")
        k, v = (s[p][table[b, place // page], place % page].double() for p in ("k_pool", "v_pool"))
        for h in range(case["heads"]):
            logits = s["q"][at:at + n, h].double() @ k[:, h // group].t() / math.sqrt(case["dim"])
            if case["causal"]:
                logits += torch.triu(torch.full((n, t), -math.inf, dtype=torch.float64, device="cuda"), t - n + 1)
            out[at:at + n, h] = torch.softmax(logits, -1) @ v[:, h // group]
            lse[at:at + n, h] = torch.logsumexp(logits, -1)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}

"""The attention side where it once went wrong, or could: one test for each fault.

Definitions, bounds and inputs are those of test_attention_side.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from test_attention_side import (  # noqa: E402,F401
    attend64, attend64_long, attend_case, check_attended, check_long, fill_past, freqs, generator, gpu, hrb, make_batch, make_pools, shared_pages,
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


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("first,last", [(0.0, 300.0), (300.0, 0.0)])
def test_what_is_not_finite_does_not_depend_on_the_cut(hrb, dtype, new, first, last):
    """A NaN or an infinity among values whose weights underflow against another part's: one sequence,
    cut over all SMs, and as many as there are SMs, each in one part."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    length = 20000
    for seqs in (1, sms):
        batch, offsets, kp, vp, q = shared_pages(hrb, generator(33), seqs, new, [length] * seqs, 64, 1, 2, 64, dtype)
        q[..., 0] = 1.0
        at = torch.arange(length, device="cuda")
        where = batch.table[0, at // 64].long(), at % 64
        kp[where[0], where[1], 0, 0] = torch.where(at < length // 2, 8 * first, 8 * last).to(dtype)
        light = 1000 if first < last else length - 1000  # a key that weighs nothing
        vp[where[0][light], where[1][light], 0, 5] = math.nan
        vp[where[0][light], where[1][light], 0, 6] = math.inf
        cache = hrb.PagedKV(kp, vp)
        for out_dtype in (dtype, torch.float32):
            got = cache.attend(q, batch, dtype=out_dtype)
            assert bool(torch.isnan(got[..., 5:7]).all())
            assert bool(torch.isfinite(got[..., :5]).all()) and bool(torch.isfinite(got[..., 7:]).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_parts_without_a_key_for_some_rows(hrb, dtype):
    """Prompts cut inside their last row tiles: a later part holds keys that earlier rows do not see."""
    for dim, heads, new, length in ((64, 1, 128, 200), (128, 4, 96, 170), (256, 2, 64, 4000), (256, 1, 128, 300)):
        batch, offsets, kp, vp, q = attend_case(hrb, dim, 16, 1, heads, [new, 1, new], [length, 7, length + 5], dtype, 34)
        check_long(hrb, batch, offsets, kp, vp, q, [length, 7, length + 5], 1 / math.sqrt(dim), dtype)


@gpu
def test_rope_is_ready_when_it_is_created(hrb):
    """A handle's frequencies are in place for a stream that does not wait for the default one."""
    from test_attention_side import check_rotated

    gen = generator(35)
    side = torch.cuda.Stream()
    x = torch.randn((2, 1, 4096), generator=gen, device="cuda")
    pos = torch.tensor([[3, 70000]], dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(x) for _ in range(40)]
    torch.cuda.synchronize()
    made = []
    for i, out in enumerate(outs):
        inv_freq = freqs(2048, 1e4 + 100 * i)
        made.append((hrb.Rope(inv_freq), inv_freq))
        with torch.cuda.stream(side):
            made[-1][0].apply(x, pos, out=out)
    torch.cuda.synchronize()
    for (_, inv_freq), out in list(zip(made, outs))[::13]:
        check_rotated(out, x, pos, inv_freq, [0] * 2048, False)


@gpu
def test_an_index_error_after_a_cleared_one_is_kept(hrb):
    """Clearing the flag does not race with the next call on a stream of its own."""
    gen = generator(36)
    kp, vp = make_pools(gen, 4, 8, 1, 64, torch.bfloat16)
    cache = hrb.PagedKV(kp, vp)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.randn((1, 1, 64), generator=gen, device="cuda")
    bad = hrb.KVBatch(i32([0, 1]), i32([1]), i32([[4]]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(100):
        with torch.cuda.stream(side):
            cache.append(k, k, bad)
        assert cache.get_error() == hrb.BITLIN_EINDEX
    assert cache.get_error() == 0


@gpu
def test_closed_handles_are_refused(hrb):
    """A closed Rope is not the same as none: nothing is written."""
    gen = generator(37)
    kp, vp = make_pools(gen, 4, 8, 1, 64, torch.bfloat16)
    cache = hrb.PagedKV(kp, vp)
    rope = hrb.Rope(freqs(32))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    batch, pos = hrb.KVBatch(i32([0, 1]), i32([1]), i32([[2]])), i32([3])
    k = torch.randn((1, 1, 64), generator=gen, device="cuda")
    q = k.bfloat16()
    before = kp.clone(), vp.clone()
    rope.close()
    with pytest.raises(ValueError, match="closed"):
        cache.append(k, k, batch, rope=rope, pos=pos, q=k)
    with pytest.raises(ValueError, match="closed"):
        rope.apply(k, pos)
    cache.close()
    with pytest.raises(ValueError, match="closed"):
        cache.append(k, k, batch)
    with pytest.raises(ValueError, match="closed"):
        cache.attend(q, batch)
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])


def stream_of_memory(t):
    """The stream whose blocks of torch's allocator a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@gpu
def test_new_outputs_lie_on_the_stream_of_the_call(hrb):
    """With `stream` and no output given, the output's memory is that stream's."""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 2, 4, [3, 1], [60, 9], torch.bfloat16, 38)
    cache, rope = hrb.PagedKV(kp, vp), hrb.Rope(freqs(32))
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    k = torch.randn((4, 2, 64), generator=generator(39), device="cuda").bfloat16()
    calls = (lambda s: rope.apply(q, pos, stream=s), lambda s: cache.append(k, k, batch, rope=rope, pos=pos, q=q, stream=s),
             lambda s: cache.attend(q, batch, stream=s), lambda s: cache.attend(q, batch, dtype=torch.float32, stream=s))
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = call(side)
        assert stream_of_memory(got) == side.cuda_stream
        assert stream_of_memory(call(torch.cuda.current_stream())) == torch.cuda.current_stream().cuda_stream
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        with torch.cuda.stream(side):
            assert stream_of_memory(call(None)) == side.cuda_stream
        torch.cuda.synchronize()


@gpu
def test_new_outputs_of_projections_lie_on_the_stream_of_the_call(hrb):
    """The same for the one-bit matrices, which the attention side stands between."""
    gen = generator(40)

    def linear(n, k):
        bits = torch.randint(-2**31, 2**31, (n, k // 32), generator=gen, device="cuda").to(torch.int32)
        scales = (torch.rand((n, k // 128), generator=gen, device="cuda") * 0.02 + 0.005).half()
        return hrb.BitLinear(bits, scales, torch.ones(k, device="cuda"))

    lin, up = linear(1024, 1024), linear(2048, 1024)
    x = torch.randn((2, 1024), generator=gen, device="cuda")
    ids = torch.tensor([3, 1000], dtype=torch.int32, device="cuda")
    for call in (lambda s: lin(x, stream=s), lambda s: lin.argmax(x, stream=s), lambda s: lin.embed(ids, stream=s),
                 lambda s: hrb.mlp_forward(up, lin, x, stream=s)):
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = call(side)
        assert stream_of_memory(got) == side.cuda_stream
        assert stream_of_memory(call(torch.cuda.current_stream())) == torch.cuda.current_stream().cuda_stream
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        torch.cuda.synchronize()


def test_batch_tensors_of_two_devices_are_refused(hrb):
    """Checked by what the tensors say of themselves: no device is needed."""
    class Elsewhere:
        dtype, is_cuda = torch.int32, True

        def __init__(self, index):
            self.device = torch.device("cuda", index)

    for at in ((0, 0, 1), (0, 1, 0), (1, 0, 0)):
        with pytest.raises(ValueError, match="one device"):
            hrb.KVBatch(*(Elsewhere(i) for i in at))


@gpu
def test_tensors_of_another_device_are_refused(hrb):
    """Handles that live on a second device, as far as the binding knows, refuse tensors of the first."""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 2, 4, [1], [9], torch.bfloat16, 41)
    cache, rope = hrb.PagedKV(kp, vp), hrb.Rope(freqs(32))
    here, there = cache.device, torch.device("cuda", 1)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.zeros((1, 2, 64), device="cuda").bfloat16()
    calls = (lambda: cache.append(k, k, batch), lambda: cache.append(k, k, batch, rope=rope, pos=pos), lambda: cache.attend(q, batch))
    rope.device = there
    with pytest.raises(ValueError, match="x must be on the handle's device"):
        rope.apply(q, pos)
    with pytest.raises(ValueError, match="the rope must be on the cache's device"):
        cache.append(k, k, batch, rope=rope, pos=pos)
    cache.device = there
    for call in calls:
        with pytest.raises(ValueError, match="the batch must be on the cache's device"):
            call()
    batch.device = there
    for call in calls:
        with pytest.raises(ValueError, match="must be on the handle's device"):
            call()
    rope.device = cache.device = batch.device = here
    for call in calls:
        call()
    assert cache.get_error() == 0


@gpu
def test_tensors_that_handles_point_to_cannot_be_replaced(hrb):
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 1, 2, [1], [40], torch.bfloat16, 42)
    cache = hrb.PagedKV(kp, vp)
    want = cache.attend(q, batch)
    for handle, names in ((batch, ("q_offsets", "kv_lens", "table")), (cache, ("k", "v"))):
        for name in names:
            held = getattr(handle, name)
            with pytest.raises(AttributeError, match=name):
                setattr(handle, name, held.clone())
            assert getattr(handle, name) is held
    assert torch.equal(cache.attend(q, batch), want)
    # contents may change, also in the form that assigns the same tensor again
    batch.kv_lens -= 8
    assert cache.k is kp and cache.v is vp
    ref = attend64(q, kp, vp, offsets, [32], batch.table, 0.125, True)
    check_attended(cache.attend(q, batch), None, ref, torch.bfloat16)


class InvalidCapture:
    """A stream whose capture has been made invalid (by a wait, which a capture does not allow):
    launches into it fail on the host."""

    ERROR = 901  # cudaErrorStreamCaptureInvalidated

    def __enter__(self):
        import ctypes

        self.cuda = ctypes.CDLL("libcuda.so.1")
        self.stream = torch.cuda.Stream()
        self.raw, self.graph = ctypes.c_void_p(self.stream.cuda_stream), ctypes.c_void_p()
        torch.cuda.synchronize()
        assert self.cuda.cuStreamBeginCapture_v2(self.raw, 2) == 0
        assert self.cuda.cuStreamSynchronize(self.raw) != 0
        return self.stream

    def __exit__(self, *_):
        import ctypes

        assert self.cuda.cuStreamEndCapture(self.raw, ctypes.byref(self.graph)) == self.ERROR


def calls_of(hrb, seed):
    """A cache, and each call of the attention side on a stream, with outputs that are given."""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 2, 4, [1], [9], torch.bfloat16, seed)
    cache, rope = hrb.PagedKV(kp, vp), hrb.Rope(freqs(32))
    cache.attend(q, batch)
    out, pos = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.zeros((1, 2, 64), device="cuda").bfloat16()
    return cache, (lambda s: rope.apply(q, pos, out=out, stream=s), lambda s: cache.append(k, k, batch, stream=s),
                   lambda s: cache.attend(q, batch, out=out, stream=s))


@gpu
def test_a_failed_call_does_not_fail_a_later_one(hrb):
    cache, calls = calls_of(hrb, 43)
    bits = torch.zeros((8, 32), dtype=torch.int32, device="cuda")
    scales, signs = torch.ones((8, 8), device="cuda").half(), torch.ones(1024, device="cuda")
    for call in calls:
        with InvalidCapture() as stream:
            with pytest.raises(hrb.BitlinError):
                call(stream)
        hrb.BitLinear(bits, scales, signs).close()  # (asks for the last error of its launches)
        call(stream)
    assert cache.get_error() == 0


@gpu
def test_errors_name_the_cuda_error_of_their_own_call(hrb):
    for i in range(3):
        cache, calls = calls_of(hrb, 44)
        with InvalidCapture() as stream:
            with pytest.raises(hrb.BitlinError, match=f"cudaError {InvalidCapture.ERROR}"):
                calls[i](stream)
        calls[i](stream)  # the handle goes on
        with pytest.raises(hrb.BitlinError) as refused:  # an argument error has no such code
            cache.attend(torch.zeros((1, 3, 64), device="cuda").bfloat16(), hrb.KVBatch(*(
                torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1], [1], [[0]]))))
        assert "cudaError" not in str(refused.value)
        assert cache.get_error() == 0


@gpu
def test_positions_in_another_order_are_refused(hrb):
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 2, 4, [5], [9], torch.bfloat16, 45)
    cache, rope = hrb.PagedKV(kp, vp), hrb.Rope(freqs(32), axis=[i % 3 for i in range(32)])
    pos = torch.randint(0, 99, (3, 5), generator=generator(46), device="cuda", dtype=torch.int32)
    k = q[:, :2].contiguous()
    before = kp.clone()
    for bad in (pos.t().contiguous(), pos[None], pos.view(1, 15)):
        with pytest.raises(ValueError, match="axes"):
            rope.apply(q, bad)
        with pytest.raises(ValueError, match="axes"):
            cache.append(k, k, batch, rope=rope, pos=bad)
    assert torch.equal(kp, before)
    assert torch.equal(rope.apply(q, pos.view(-1)), rope.apply(q, pos))


def without_torch(code):
    """Run in a Python of its own that finds no torch."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", "import sys\nsys.modules['torch'] = None\n" + code], cwd=root,
                          capture_output=True, text=True, timeout=600)
    assert done.returncode == 0, done.stderr


def test_the_library_builds_without_torch(hrb):
    without_torch("from hadamard_rotated_binary_gb300 import build\n"
                  "assert build.build() == build.LIB\n"
                  "import hadamard_rotated_binary_gb300 as m\n"
                  "assert m.lib().bitlin_version() >= 100\n")


def test_import_star_without_torch(hrb):
    without_torch("from hadamard_rotated_binary_gb300 import *\n"
                  "BitLinear, load_q1g128, PATH_AUTO\n"
                  "assert 'Rope' not in globals()\n")
    names = {}
    exec("from hadamard_rotated_binary_gb300 import *", names)
    assert {"BitLinear", "Rope", "PagedKV", "KVBatch", "PAIRS_HALF", "PAIRS_ADJACENT"} <= set(names)


@gpu
def test_caches_share_a_workspace(hrb):
    """Layers with heads of several sizes and types on one workspace, their calls in turn, each against a
    cache of its own; handles closed in any order; no memory of their own."""
    cases = [attend_case(hrb, dim, 16, 2, 4, new, lens, dtype, 47 + dim)
             for dim, new, lens, dtype in ((256, [3, 1], [900, 5000], torch.bfloat16), (64, [1, 40], [7000, 300], torch.float16),
                                           (128, [1, 1], [20, 30000], torch.bfloat16), (200, [2, 2], [3000, 3000], torch.bfloat16))]
    want = []
    for batch, _, kp, vp, q in cases:
        cache = hrb.PagedKV(kp, vp)
        want.append((cache.attend(q, batch), cache.attend(q, batch, dtype=torch.float32)))
        cache.close()
    first = hrb.PagedKV(cases[0][2], cases[0][3])
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    layers = [first] + [hrb.PagedKV(kp, vp, share=first) for _, _, kp, vp, _ in cases[1:]]
    more = [hrb.PagedKV(cases[0][2], cases[0][3], share=layers[-1]) for _ in range(8)]
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] < 16 << 20  # (one workspace has 40 MB)
    for _ in range(3):
        for cache, (batch, _, _, _, q), (out, wide) in zip(layers, cases, want):
            assert torch.equal(cache.attend(q, batch), out)
            assert torch.equal(cache.attend(q, batch, dtype=torch.float32), wide)
    first.close()
    layers[2].close()
    for i in (1, 3):
        assert torch.equal(layers[i].attend(cases[i][4], cases[i][0]), want[i][0])
    assert torch.equal(more[5].attend(cases[0][4], cases[0][0]), want[0][0])
    assert all(c.get_error() == 0 for c in [layers[1], layers[3]] + more)
    # a workspace for smaller heads is refused, and so is a closed cache's
    small = hrb.PagedKV(cases[1][2], cases[1][3])
    for other in (small, first):
        with pytest.raises(hrb.BitlinError):
            hrb.PagedKV(cases[0][2], cases[0][3], share=other)


@gpu
def test_a_timeout_is_one_of_all_caches_that_share(hrb):
    batch, offsets, kp, vp, q = attend_case(hrb, 128, 16, 2, 4, [40, 1], [300, 20], torch.bfloat16, 22)
    one = hrb.PagedKV(kp, vp)
    two, apart = hrb.PagedKV(kp, vp, share=one), hrb.PagedKV(kp, vp)
    want = two.attend(q, batch)
    assert one.get_error() == two.get_error() == 0
    one.set_wait_budget(2_000_000)
    one.test_stall(True)
    one.attend(q, batch)
    for cache in (two, one):
        assert cache.get_error() == hrb.BITLIN_ETIMEOUT
        with pytest.raises(hrb.BitlinError):
            cache.attend(q, batch)
    assert apart.get_error() == 0 and torch.equal(apart.attend(q, batch), want)


@gpu
def test_the_first_call_can_be_captured(hrb):
    """Nothing is allocated or loaded by a handle's first call, of either output type."""
    batch, offsets, kp, vp, q = attend_case(hrb, 72, 16, 2, 4, [3, 1], [900, 50], torch.float16, 48)
    ref = attend64(q, kp, vp, offsets, [900, 50], batch.table, 72**-0.5, True)
    for out_dtype in (torch.float16, torch.float32):
        cache, out = hrb.PagedKV(kp, vp), torch.zeros(q.shape, dtype=out_dtype, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.attend(q, batch, out=out)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            check_attended(out, None, ref, torch.float16)
        assert cache.get_error() == 0


def angles_mod_turn(inv_freq, positions):
    """pos * freq modulo 2 pi, in f64, from 100 digits; [positions][freqs]."""
    from decimal import Decimal, getcontext

    getcontext().prec = 100

    def arctan_inverse(x):
        total = term = Decimal(1) / x
        n = 1
        while abs(term) > Decimal(10) ** -99:
            term /= -x * x
            n += 2
            total += term / n
        return total

    turn = 2 * (16 * arctan_inverse(5) - 4 * arctan_inverse(239))
    rows = []
    for p in positions:
        exact = [Decimal(float(torch.tensor(f, dtype=torch.float32))) * p / turn for f in inv_freq]
        rows.append([float((x - x.to_integral_value()) * turn) for x in exact])
    return torch.tensor(rows, dtype=torch.float64)


@gpu
@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_bound_at_every_position_and_frequency(hrb, adjacent):
    """The documented bound, of a pair's norm: for an f32 output the angle's 24 bits of half a turn
    (2^-26 of a turn, 2^-32 cut off, 2^-31 from the frequency's rounding: 9.8e-8), sine and cosine
    to one unit in the last place (sqrt(2) 2^-24), a product's and the sum's rounding (2 * 2^-24):
    3.1e-7; for a 16-bit one the hardware's sine and cosine (2^-21.4 and 2^-21.2) and the angle's
    rounding to radians instead: 1e-6, then its own."""
    inv_freq = [1.0, -0.25, 7.5, 1e-9, 6.25, 6.2831855, 100.0, -31415.926, 3e38, 1e-45, 0.0, 1e10, 0.7, 1.25e-3, -1e20, 2.0**60]
    positions = [0, 1, -1, 777, 131071, 2**24 + 1, 2**28 + 5, 2**31 - 1, -2**31, -2**31 + 1, 1234567891]
    heads, pairs = 64, len(inv_freq)
    x = torch.randn((len(positions), heads, 2 * pairs), generator=generator(49), device="cuda")
    pos = torch.tensor([positions], dtype=torch.int32, device="cuda")
    t = angles_mod_turn(inv_freq, positions)[:, None, :]
    first, second = (slice(0, None, 2), slice(1, None, 2)) if adjacent else (slice(0, pairs), slice(pairs, None))
    rope = hrb.Rope(inv_freq, adjacent=adjacent)
    for dtype, rel, own, tiny in ((torch.float32, 3.1e-7, 0.0, 0.0), (torch.bfloat16, 1e-6, 2.0**-8, 0.0), (torch.float16, 1e-6, 2.0**-11, 2.0**-25)):
        for inverse in (False, True):
            y = rope.apply(x, pos, dtype=dtype, inverse=inverse).double().cpu()
            a, b = x[..., first].double().cpu(), x[..., second].double().cpu()
            sin = -torch.sin(t) if inverse else torch.sin(t)
            norm = torch.sqrt(a * a + b * b)
            for got, want in ((y[..., first], a * torch.cos(t) - b * sin), (y[..., second], b * torch.cos(t) + a * sin)):
                bound = rel * norm
                bound = bound + own * (want.abs() + bound) + tiny
                assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / norm).max())


@gpu
def test_pools_of_one_head_or_one_page(hrb):
    """A dimension of one may have any stride, and another one in k than in v."""
    for pages, kvh in ((6, 1), (1, 2), (1, 1)):
        gen = generator(50)
        lens = [16 * pages - 3]
        batch, offsets, _ = make_batch(hrb, gen, [2], lens, 16, spare=0)
        k, v = make_pools(gen, pages, 16, kvh, 64, torch.bfloat16)
        q = torch.randn((2, 2 * kvh, 64), generator=gen, device="cuda").bfloat16()
        want = hrb.PagedKV(k, v).attend(q, batch)
        odd = [s if n > 1 else 1 for n, s in zip(k.shape, k.stride())]
        far = [s if n > 1 else 8 * s + 8 for n, s in zip(k.shape, k.stride())]
        for a, b in ((odd, odd), (odd, far), (far, k.stride())):
            cache = hrb.PagedKV(k.as_strided(k.shape, a), v.as_strided(v.shape, b))
            assert torch.equal(cache.attend(q, batch), want)
            new = torch.randn((2, kvh, 64), generator=gen, device="cuda")
            keep = k.clone(), v.clone()
            cache.append(new, new, batch)
            at = torch.arange(lens[0] - 2, lens[0], device="cuda")
            assert torch.equal(v[batch.table[0, at // 16].long(), at % 16], new.bfloat16())
            k.copy_(keep[0])
            v.copy_(keep[1])
            assert cache.get_error() == 0


# ------------------------------------------------------------------ forms that had no test

@gpu
@pytest.mark.parametrize("dim,kvh,heads,rotary", [(64, 2, 6, 32), (80, 1, 3, 40), (256, 4, 24, 64)])
def test_append_of_a_fused_projection(hrb, dim, kvh, heads, rotary):
    """Queries, keys and values as slices of one projection, by head or side by side, and a table whose
    rows are farther apart than they are long."""
    from test_attention_side import check_rotated

    gen = generator(51)
    new, lens = [3, 1, 20], [40, 17, 20]
    batch, offsets, pages = make_batch(hrb, gen, new, lens, 16)
    apart = torch.full((3, batch.table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    apart[:, :-5] = batch.table
    batch = hrb.KVBatch(batch.q_offsets, batch.kv_lens, apart[:, :-5])
    T, inv_freq = offsets[-1], freqs(rotary // 2)
    pos = torch.randint(0, 9000, (1, T), generator=gen, device="cuda", dtype=torch.int32)
    rope = hrb.Rope(inv_freq)
    for src in (torch.float32, torch.bfloat16):
        side_by_side = torch.randn((T, (heads + 2 * kvh) * dim + 4), generator=gen, device="cuda").to(src)
        parts = side_by_side[:, 2:-2].split((heads * dim, kvh * dim, kvh * dim), -1)
        slices = [tuple(p.unflatten(-1, (-1, dim)) for p in parts)]
        by_head = torch.randn((T, kvh, heads // kvh + 2, dim), generator=gen, device="cuda").to(src)
        slices.append((by_head[:, :, 0], by_head[:, :, -2], by_head[:, :, -1]))
        for q, k, v in slices:
            assert not k.is_contiguous() and not v.is_contiguous()
            kp, vp = make_pools(gen, pages, 16, kvh, dim, torch.bfloat16)
            before = kp.clone(), vp.clone()
            cache = hrb.PagedKV(kp, vp)
            q_out = cache.append(k, v, batch, rope=rope, pos=pos, q=q)
            check_rotated(q_out, q, pos, inv_freq, [0] * (rotary // 2), False)
            at = [(s, lens[s] - new[s] + i) for s in range(3) for i in range(new[s])]
            where = (torch.stack([apart[s, p // 16] for s, p in at]).long(), torch.tensor([p % 16 for _, p in at], device="cuda"))
            check_rotated(kp[where], k, pos, inv_freq, [0] * (rotary // 2), False)
            assert torch.equal(vp[where], v.bfloat16())
            before[0][where], before[1][where] = kp[where], vp[where]
            assert torch.equal(before[0], kp) and torch.equal(before[1], vp)
            if q.shape[1] == heads:  # attention reads the same table
                ref = attend64(q_out, kp, vp, offsets, lens, apart, dim**-0.5, True)
                check_attended(cache.attend(q_out, batch), None, ref, torch.bfloat16)
            assert cache.get_error() == 0


@gpu
@pytest.mark.parametrize("seqs", [31, 32, 33, 1023, 1024, 1025, 2500])
def test_append_and_attend_of_many_sequences(hrb, seqs):
    """The search for a token's sequence: 32 boundaries a round, over one, two and three rounds, with
    sequences of no new token among them (the first, the last and runs of them)."""
    from test_attention_side import check_rotated

    gen = generator(52)
    new = [0 if i in (0, seqs - 1) or i % 7 in (2, 3) or 500 < i < 560 else 1 + (i % 11 == 4) * 2 for i in range(seqs)]
    lens = [n + (3 * i) % 29 for i, n in enumerate(new)]
    batch, offsets, pages = make_batch(hrb, gen, new, lens, 8)
    kp, vp = make_pools(gen, pages, 8, 1, 64, torch.float16)
    T, inv_freq = offsets[-1], freqs(16)
    k, v, q = (torch.randn((T, h, 64), generator=gen, device="cuda") for h in (1, 1, 2))
    cache = hrb.PagedKV(kp, vp)
    q_out = cache.append(k, v, batch, rope=hrb.Rope(inv_freq), q=q)
    seq = torch.repeat_interleave(torch.arange(seqs), torch.tensor(new)).cuda()
    place = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lens)]).cuda()
    where = batch.table[seq, place // 8].long(), place % 8
    check_rotated(kp[where], k, place[None], inv_freq, [0] * 16, False)
    check_rotated(q_out, q, place[None], inv_freq, [0] * 16, False)
    assert torch.equal(vp[where], v.half())
    out = cache.attend(q_out, batch, dtype=torch.float32)
    check_attended(out, None, attend64(q_out, kp, vp, offsets, lens, batch.table, 0.125, True), torch.float16)
    assert cache.get_error() == 0


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,kvh,heads", [(64, 2, 8), (128, 1, 3), (256, 1, 6)])
def test_attend_prompts_beside_single_tokens(hrb, dtype, dim, kvh, heads):
    """A serving step that mixes a prompt with single tokens."""
    new, lens = [1, 150, 1, 1, 9, 1], [500, 150, 33, 1, 300, 129]
    batch, offsets, kp, vp, q = attend_case(hrb, dim, 16, kvh, heads, new, lens, dtype, 53, q_scale=2.0)
    fill = attend64(q, kp, vp, offsets, lens, batch.table, dim**-0.5, True)
    cache = hrb.PagedKV(kp, vp)
    for out_dtype in (dtype, torch.float32):
        lse = torch.empty(q.shape[:2], device="cuda")
        check_attended(cache.attend(q, batch, dtype=out_dtype, lse=lse), lse, fill, dtype)
    assert cache.get_error() == 0


@gpu
@pytest.mark.parametrize("dtype,most", [(torch.float16, 3.9e7), (torch.bfloat16, 6.9e8)])
def test_scores_as_large_as_documented(hrb, dtype, most):
    """Keys alike, with scores up to the documented size of either sign: the mean of the values, within the
    weights' and the output's rounding.  (The reference is rounded before it is subtracted.)"""
    batch, offsets, kp, vp, q = attend_case(hrb, 64, 16, 1, 2, [1, 3], [500, 40], dtype, 54)
    kp.fill_(0.0)
    kp[..., 0] = 1024.0
    q.fill_(0.0)
    q[:, 0, 0], q[:, 1, 0] = 1000.0, -1000.0
    cache = hrb.PagedKV(kp, vp)
    for i in range(25):
        scale = most * (0.5 + i / 48) / 1.024e6
        out, lse, _, size = attend64(q, kp, vp, offsets, [500, 40], batch.table, scale, True)
        for out_dtype in (dtype, torch.float32):
            got_lse = torch.empty(q.shape[:2], device="cuda")
            got = cache.attend(q, batch, scale=scale, dtype=out_dtype, lse=got_lse).double().cpu()
            u = 2.0**-8 if dtype == torch.bfloat16 else 2.0**-11
            digits = u if out_dtype == dtype else u * u
            own = u if out_dtype == dtype else 2.0**-24
            assert bool(((got - out).abs() <= size * (digits + 2.0**-18) + own * (out.abs() + digits * size)).all())
            assert bool(((got_lse.double().cpu() - lse).abs() <= 2.0**-21 * lse.abs()).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,heads", [(64, 1), (128, 6), (256, 8)])
@pytest.mark.parametrize("heavy", [0, 1])
def test_f32_outputs_of_single_tokens_hold_whole_weights(hrb, dtype, dim, heads, heavy):
    """Two keys of exact scores, one of weight 1 and value 0, one of weight w and value 1: w / (1 + w).

    In units of 2^-24 of w: the argument of 2^x for |x| < 8 is rounded (4) and its factor too (8), ex2 is
    good to 3, the digits hold all bits or 22 (2), the sum of two products is cut at 2, and sum,
    reciprocal and product round three times (3): with x's by ln 2, 18.3 units, 1.1e-6.  (Two digits of
    bf16 are off by up to 7.6e-6.)"""
    seqs = 300
    gen = generator(55)
    batch, offsets, pages = make_batch(hrb, gen, [1] * seqs, [2] * seqs, 8)
    kp, vp = make_pools(gen, pages, 8, 1, dim, dtype, fill=0.0)
    score = torch.linspace(-5.4, 5.4 if heavy else 0.0, seqs, device="cuda").to(dtype)
    page = batch.table[:, 0].long()
    kp[page, heavy, 0, 0] = score
    vp[page, heavy] = 1.0
    q = torch.zeros((seqs, heads, dim), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    got = hrb.PagedKV(kp, vp).attend(q, batch, scale=1.0, dtype=torch.float32).double().cpu()
    w = torch.exp(score.double().cpu())[:, None, None]
    want = (w / (1 + w)).expand_as(got)
    assert bool(((got - want).abs() <= 1.1e-6 * want).all()), float(((got - want).abs() / want).max())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 0, 0, 1], [0, 4, 0, 0], [0, 0, 1, 0], [2, 0, 0, 0], [60] + [0] * 58 + [1]])
@pytest.mark.parametrize("kvh,heads", [(1, 8), (2, 10), (1, 6), (2, 2), (1, 9)])
def test_f32_outputs_of_few_tokens_however_spread(hrb, dtype, new, kvh, heads):
    """As many tokens as sequences, or fewer, spread in any way, and more than were counted on."""
    lens = [n + (37 * i + 5) % 300 for i, n in enumerate(new)]
    batch, offsets, kp, vp, q = attend_case(hrb, 72, 16, kvh, heads, new, lens, dtype, 56, q_scale=2.0)
    fill_past(batch, kp, vp, lens, math.nan)
    cache = hrb.PagedKV(kp, vp)
    for causal in (True, False):
        ref = attend64(q, kp, vp, offsets, lens, batch.table, 72**-0.5, causal)
        lse = torch.empty(q.shape[:2], device="cuda")
        out = cache.attend(q, batch, causal=causal, dtype=torch.float32, lse=lse)
        check_attended(out, lse, ref, dtype)
        assert torch.equal(out, cache.attend(q, batch, causal=causal, dtype=torch.float32))
    assert cache.get_error() == 0

"""Binding of the attention side: rotary positions, norms of heads, the paged caches in 16 and in
4 bits and attention over them.

Handles live here (ctypes, as in ``_binding``); the calls on tensors are marshalled by the compiled
``_paged_native`` (csrc/paged_native.cpp)."""
from __future__ import annotations

import ctypes

import torch

from ._binding import BITLIN_OK, Batch, BitlinError, QuantPools, lib

lib()  # libbitlin.so first: the compiled binding is linked against it

from . import _paged_native as native  # noqa: E402

F32, BF16, F16 = 0, 1, 2
PAIRS_HALF, PAIRS_ADJACENT = 0, 1

_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


class Rope:
    """Rotary positions with one or several axes (a bitlin_rope handle on the current device).

    inv_freq  R/2 numbers: pair i turns by pos[axis[i]] * inv_freq[i]
    axis      R/2 axis indices, or None: one axis
    adjacent  pairs (2i, 2i + 1) instead of (i, i + R/2)
    """

    def __init__(self, inv_freq, axis=None, adjacent: bool = False):
        freq = [float(f) for f in inv_freq]
        of = None if axis is None else [int(a) for a in axis]
        if of is not None and len(of) != len(freq):
            raise ValueError("axis must name one axis per frequency")
        self.rotary_dim = 2 * len(freq)
        self.axes = 1 if not of else max(of) + 1
        self.device = torch.device("cuda", torch.cuda.current_device())
        h = ctypes.c_void_p()
        st = lib().bitlin_rope_create(ctypes.byref(h), self.rotary_dim, self.axes,
                                      (ctypes.c_float * len(freq))(*freq),
                                      None if of is None else (ctypes.c_int32 * len(of))(*of),
                                      PAIRS_ADJACENT if adjacent else PAIRS_HALF)
        if st != BITLIN_OK:
            raise BitlinError(st, "bitlin_rope_create")
        self._h = h.value

    def apply(self, x, pos, out=None, dtype=None, inverse: bool = False, stream=None, norm=None, eps: float = 1e-6):
        """bitlin_rope_apply: x [tokens][heads][dim] rotated by pos (int32 [axes][tokens]), into `out`
        (x itself is allowed) or a new tensor of `dtype` (x's where None).

        norm  float32 [dim]: each head is first divided by its root mean square (eps added to the
              mean, 0 .. 1e38) and multiplied by this weight, in the same pass
              (bitlin_rope_apply_normed).

        Autograd does not record the call: the gradient is apply with inverse=True, or, with a norm,
        `gradient`.
        """
        return native.rope_apply(self._h, self.device.index, self.axes, x, pos, out, dtype, inverse, stream, norm, eps)

    def gradient(self, dy, x, pos, norm, eps: float = 1e-6, dx=None, stream=None):
        """bitlin_rope_gradient: the gradient of apply(x, pos, norm=norm, eps=eps) from that of its
        output: (dx in x's type, the weight's in float32).  dx: x, dy, or a tensor to write to.  Neither result
        requires a gradient: hand them to a torch.autograd.Function's backward."""
        return native.rope_gradient(self._h, self.device.index, self.axes, dy, x, pos, norm, eps, dx, stream)

    def close(self):
        if getattr(self, "_h", None):
            lib().bitlin_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _held(name: str):
    """A tensor whose address a handle keeps: its contents may change, the tensor itself may not
    (the old one's memory would be freed under the calls that read it).  Assigning the same tensor
    again, as `batch.kv_lens += 1` does, is no change."""

    def get(self):
        return self.__dict__["_" + name]

    def put(self, value):
        if value is not self.__dict__.get("_" + name, value):
            raise AttributeError(f"{name} cannot be replaced: change its contents, or make a new {type(self).__name__}")
        self.__dict__["_" + name] = value

    return property(get, put)


class KVBatch:
    """The new tokens of a batch of sequences (a bitlin_kv_batch; holds the tensors).

    q_offsets  int32 CUDA [seqs + 1]: sequence s owns token rows q_offsets[s] .. q_offsets[s + 1] - 1
    kv_lens    int32 CUDA [seqs]: tokens in the cache, the new ones with them
    table      int32 CUDA [seqs][pages per sequence]

    Calls read the tensors on the device: their contents may change between calls, the tensors stay.
    """

    q_offsets, kv_lens, table = _held("q_offsets"), _held("kv_lens"), _held("table")

    def __init__(self, q_offsets, kv_lens, table):
        for t in (q_offsets, kv_lens, table):
            if t.dtype != torch.int32 or not t.is_cuda:
                raise ValueError("q_offsets, kv_lens and table must be int32 CUDA tensors")
            if t.device != kv_lens.device:
                raise ValueError("q_offsets, kv_lens and table must be on one device")
        seqs = kv_lens.numel()
        if not (q_offsets.is_contiguous() and kv_lens.is_contiguous()) or q_offsets.numel() != seqs + 1:
            raise ValueError("q_offsets [seqs + 1] and kv_lens [seqs] must be contiguous")
        if table.dim() != 2 or table.shape[0] != seqs or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be [seqs][pages] with contiguous rows")
        if table.stride(0) < table.shape[1] and seqs > 1:
            raise ValueError("table's rows must not overlap")
        self.q_offsets, self.kv_lens, self.table = q_offsets, kv_lens, table
        self.device = kv_lens.device
        # the row length bounds what is read; rows of a wider table may be longer apart
        self._c = Batch(seqs, q_offsets.data_ptr(), kv_lens.data_ptr(), table.data_ptr(), table.shape[1],
                        table.stride(0))
        self.address = ctypes.addressof(self._c)


def _same_kind(cache, kind, name: str):
    """A handle reaches the library as an address, which does not say what lies there."""
    if cache is not None and not isinstance(cache, kind):
        raise ValueError(f"{name} must be a {kind.__name__}")


def _rope_of(rope: Rope | None, device):
    """(handle, axes) of an append's rope."""
    if rope is None:
        return None, 0
    _same_kind(rope, Rope, "rope")
    if not rope._h:
        raise ValueError("the rope's handle is closed")  # (None would mean no rotation)
    if rope.device != device:
        raise ValueError("the rope must be on the cache's device")
    return rope._h, rope.axes


class PagedKV:
    """One layer's paged cache (a bitlin_kv handle on the caller's pools, which it keeps alive).

    k, v  bfloat16 or float16 CUDA tensors [pages][page_size][kv_heads][head_dim] with the same
          strides, head_dim contiguous (a permuted view of another page layout is fine)
    share another layer's cache, with heads at least as large, whose workspace to use (40 MB at
          head_dim 256) in place of one of its own: the calls on both must then follow one
          another in stream order
    """

    k, v = _held("k"), _held("v")

    def __init__(self, k, v, share: PagedKV | None = None):
        # a dimension of one has no stride that matters
        strides = [[s if n > 1 else t.shape[-1] for n, s in zip(t.shape, t.stride())] for t in (k, v)]
        if k.dim() != 4 or k.shape != v.shape or strides[0] != strides[1] or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages][page_size][kv_heads][head_dim] of one type and layout")
        if not (k.is_cuda and v.is_cuda) or k.stride(3) != 1 or k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("k and v must be bfloat16 or float16 CUDA tensors with contiguous heads")
        if k.device != v.device:
            raise ValueError("k and v must be on one device")
        _same_kind(share, PagedKV, "share")
        self.k, self.v = k, v
        self.device, self.dtype = k.device, k.dtype
        pages, page_size, self.kv_heads, self.head_dim = k.shape
        page_stride, slot_stride, head_stride = strides[0][:3]
        h = ctypes.c_void_p()
        with torch.cuda.device(k.device):
            st = lib().bitlin_kv_create(ctypes.byref(h), k.data_ptr(), v.data_ptr(), pages, page_size, self.kv_heads,
                                        self.head_dim, _CODES[k.dtype], page_stride, slot_stride, head_stride)
            if st != BITLIN_OK:
                raise BitlinError(st, "bitlin_kv_create")
            self._h = h.value
            if share is not None:
                self._check(lib().bitlin_kv_share(self._h, share._h), "bitlin_kv_share")

    def _check(self, st: int, what: str):
        if st != BITLIN_OK:
            raise BitlinError(st, what, lib().bitlin_kv_cuda_error(self._h))

    def _address_of(self, batch: KVBatch) -> int:
        if batch.device != self.device:
            raise ValueError("the batch must be on the cache's device")
        return batch.address

    def append(self, k, v, batch: KVBatch, rope: Rope | None = None, pos=None, q=None, q_out=None, stream=None,
               q_norm=None, k_norm=None, eps: float = 1e-6):
        """bitlin_kv_append: k and v [tokens][kv_heads][head_dim] to their places, k rotated; q
        [tokens][heads][head_dim], when given, is rotated too and returned in the cache's type.

        q_norm, k_norm  float32 [head_dim]: each head of q and of k is normed before its rotation,
                        in the same pass (see Rope.apply).
        """
        r, axes = _rope_of(rope, self.device)
        return native.kv_append(self._h, self.device.index, self.kv_heads, self.head_dim, self.dtype,
                                self._address_of(batch), k, v, r, axes, pos, q, q_out, stream, q_norm, k_norm, eps)

    def attend(self, q, batch: KVBatch, scale: float | None = None, causal: bool = True, out=None, dtype=None,
               lse=None, stream=None):
        """bitlin_kv_attend: attention of q [tokens][heads][head_dim] over the batch's sequences, into
        `out` or a new tensor of `dtype` (the cache's type, or float32); lse: float32 [tokens][heads]."""
        return native.kv_attend(self._h, self.device.index, self.head_dim, self.dtype, self._address_of(batch), q, scale,
                                causal, out, dtype, lse, stream)

    def set_wait_budget(self, ns: int):
        self._check(lib().bitlin_kv_set_wait_budget(self._h, int(ns)), "bitlin_kv_set_wait_budget")

    def test_stall(self, on: bool):
        self._check(lib().bitlin_kv_test_stall(self._h, 1 if on else 0), "bitlin_kv_test_stall")

    def get_error(self) -> int:
        return lib().bitlin_kv_get_error(self._h)

    def close(self):
        if getattr(self, "_h", None):
            lib().bitlin_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class QuantKV:
    """One layer's paged cache in 4 bits (a bitlin_kvq handle on the caller's pools, which it keeps
    alive).  `QuantKV.pools` makes pools in the layout that is read fastest.

    k, v              uint8 CUDA tensors [pages][page_size][kv_heads][head_dim / 2], head_dim 64, 128
                      or 256, with the same strides (multiples of 16): two elements a byte
    k_scale, v_scale  uint8 CUDA tensors [pages][page_size][kv_heads][4] with the same strides
                      (multiples of 4): a scale for each quarter of a head
    dtype             bfloat16 or float16: of queries, and of outputs unless they are asked for in
                      float32
    share             another 4-bit cache, whose workspace to use in place of one of its own: the
                      calls on both must then follow one another in stream order
    """

    k, v, k_scale, v_scale = _held("k"), _held("v"), _held("k_scale"), _held("v_scale")

    def __init__(self, k, v, k_scale, v_scale, dtype=torch.bfloat16, share: QuantKV | None = None):
        parts = (k, v, k_scale, v_scale)
        if any(t.dtype != torch.uint8 or not t.is_cuda or t.dim() != 4 or t.device != k.device for t in parts):
            raise ValueError("k, v and their scales must be 4-dimensional uint8 CUDA tensors on one device")
        if k.shape != v.shape or k_scale.shape != v_scale.shape or k_scale.shape != k.shape[:3] + (4,):
            raise ValueError("k and v must be [pages][page_size][kv_heads][head_dim / 2], the scales [pages][page_size][kv_heads][4]")
        if any(t.stride(3) != 1 for t in parts):
            raise ValueError("heads must be contiguous")
        # a dimension of one has no stride that matters
        strides = [[s if n > 1 else max(t.shape[3], 16) for n, s in zip(t.shape, t.stride())][:3] for t in parts]
        if strides[0] != strides[1] or strides[2] != strides[3]:
            raise ValueError("k and v must have one layout, and their scales one")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be bfloat16 or float16")
        _same_kind(share, QuantKV, "share")
        self.k, self.v, self.k_scale, self.v_scale = parts
        self.device, self.dtype = k.device, dtype
        pages, page_size, self.kv_heads, self.head_dim = *k.shape[:3], 2 * k.shape[3]
        pools = QuantPools(*(t.data_ptr() for t in parts), pages, page_size, self.kv_heads, self.head_dim,
                           *strides[0], *strides[2])
        h = ctypes.c_void_p()
        with torch.cuda.device(k.device):
            st = lib().bitlin_kvq_create(ctypes.byref(h), ctypes.byref(pools), _CODES[dtype])
            if st != BITLIN_OK:
                raise BitlinError(st, "bitlin_kvq_create")
            self._h = h.value
            if share is not None:
                st = lib().bitlin_kvq_share(self._h, share._h)
                if st != BITLIN_OK:
                    raise BitlinError(st, "bitlin_kvq_share", lib().bitlin_kvq_cuda_error(self._h))

    @staticmethod
    def pools(pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        """(k, v, k_scale, v_scale) of zeros, the slots of a head side by side in memory."""
        def pool(n):
            return torch.zeros((pages, kv_heads, page_size, n), dtype=torch.uint8, device=device).transpose(1, 2)
        return pool(head_dim // 2), pool(head_dim // 2), pool(4), pool(4)

    def _address_of(self, batch: KVBatch) -> int:
        if batch.device != self.device:
            raise ValueError("the batch must be on the cache's device")
        return batch.address

    def append(self, k, v, batch: KVBatch, rope: Rope | None = None, pos=None, q=None, q_out=None, stream=None,
               q_norm=None, k_norm=None, eps: float = 1e-6):
        """bitlin_kvq_append: as PagedKV.append, to 4 bits; q is returned in the handle's dtype."""
        r, axes = _rope_of(rope, self.device)
        return native.kvq_append(self._h, self.device.index, self.kv_heads, self.head_dim, self.dtype,
                                 self._address_of(batch), k, v, r, axes, pos, q, q_out, stream, q_norm, k_norm, eps)

    def read(self, batch: KVBatch, tokens: int, k=None, v=None, dtype=None, stream=None):
        """bitlin_kvq_read: what the cache holds at the places of the batch's rows, as (k, v)
        [tokens][kv_heads][head_dim], into `k` and `v` or new tensors of `dtype` (the handle's)."""
        return native.kvq_read(self._h, self.device.index, self.kv_heads, self.head_dim, self._address_of(batch), tokens,
                               k, v, dtype or self.dtype, stream)

    def attend(self, q, batch: KVBatch, scale: float | None = None, causal: bool = True, out=None, dtype=None,
               lse=None, stream=None, through: PagedKV | None = None, f32_through: bool = False):
        """bitlin_kvq_attend: as PagedKV.attend, over the 4-bit cache.

        through      a 16-bit cache of the same pages, page size, heads and dtype whose pools are
                     scratch (one serves all layers): calls whose sequences bring many tokens
                     read their pages back into it and attend there, faster for prompts
                     (what goes wrong there, get_error of this handle tells)
        f32_through  whether float32 outputs go through it too: as exact as PagedKV.attend's
                     (up to 3e-6 off) and 2 to 7 times faster, where without it they are as
                     exact as float32 arithmetic
        """
        _same_kind(through, PagedKV, "through")
        if through is not None and not through._h:
            raise ValueError("through's handle is closed")
        return native.kvq_attend(self._h, self.device.index, self.head_dim, self.dtype, self._address_of(batch), q, scale,
                                 causal, out, dtype, lse, stream, None if through is None else through._h, f32_through)

    def get_error(self) -> int:
        return lib().bitlin_kvq_get_error(self._h)

    def close(self):
        if getattr(self, "_h", None):
            lib().bitlin_kvq_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

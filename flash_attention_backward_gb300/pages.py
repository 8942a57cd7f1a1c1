"""PyTorch-facing wrappers of fa_paged_ext.h: who holds which page, bounds of the pages' keys and the selection of
pages by them, and the axes of a rotation's pairs.

Conventions are those of paged.py, whose calls take what these make: cache_append() the slots of pages_extend(),
paged_decode() the pages of page_select(), qk_norm_rope() and cache_append() the axes of rope_sections().
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _native as nat
from . import paged
from .api import FaBackError, Workspace, _check
from .paged import _F32, _I32, _act, _call, _empty, _expect, _heads, _index, _int32


def rope_sections(sections: Sequence[int], *, interleaved: bool = False, device="cuda") -> torch.Tensor:
    """The axis of each rotation pair (uint8 [pairs]), as rope_axes takes them: sections[a] pairs for axis a, one axis
    after another, or with interleaved in turn while an axis has pairs left."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 8 or min(left) < 0:
        raise FaBackError("sections: the pairs of one to eight axes expected")
    if not interleaved:
        out = [a for a, n in enumerate(left) for _ in range(n)]
    else:
        out = []
        while any(left):
            for a, n in enumerate(left):
                if n:
                    out.append(a)
                    left[a] -= 1
    return torch.tensor(out, dtype=torch.uint8).to(device)


class _Held:
    """An object of the tensors that it was made with: the kernels are given their addresses."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise FaBackError(f"{name}: a {type(self).__name__} keeps what it was made with; make another one")
        super().__setattr__(name, value)


class PageLists(_Held):
    """Who holds which page of a pool of free.numel() pages of page_size positions: page_table (int32 [B][max_pages]) and
    seq_lens (int32 [B]; negative: a slot without a request), which PagedCache and paged_decode() take, and the pages that
    nobody holds, free[:num_free] (int32 [num_pages], [1]), the last one to be taken first.  num_pages and page_size are those
    of the cache that the pages are of; no call sees both to compare them.  Holds the tensors, which
    pages_extend() and pages_trim() edit in place; a request is taken in by setting its length to 0."""

    def __init__(self, page_table: torch.Tensor, seq_lens: torch.Tensor, free: torch.Tensor, num_free: torch.Tensor, *,
                 page_size: int):
        if page_table.dim() != 2 or free.dim() != 1:
            raise FaBackError("page_table: int32 [B][max_pages], free: int32 [num_pages] expected")
        self.page_table, self.seq_lens, self.free, self.num_free, self.page_size = page_table, seq_lens, free, num_free, page_size
        self.B, self.max_pages = page_table.shape
        self.num_pages, self.device = free.shape[0], page_table.device
        for name, n in (("page_table", max(page_table.shape)), ("free", self.num_pages), ("page_size", page_size)):
            _int32(name, "sizes below 2^31", n)
        self.c = nat.fa_page_lists(
            _expect("page_table", page_table, _I32, tuple(page_table.shape), self.device),
            _expect("seq_lens", seq_lens, _I32, (self.B,), self.device), _expect("free", free, _I32, tuple(free.shape), self.device),
            _expect("num_free", num_free, _I32, (1,), self.device), self.num_pages, page_size, self.B, self.max_pages)
        self._at, self._index = ctypes.addressof(self.c), self.device.index

    @classmethod
    def empty(cls, B: int, max_pages: int, num_pages: int, page_size: int, *, device="cuda") -> "PageLists":
        """B slots without a request, and all pages free (page 0 the first to be taken)."""
        def ints(*shape):
            return torch.full(shape, -1, dtype=_I32, device=device)
        return cls(ints(B, max_pages), ints(B), torch.arange(num_pages - 1, -1, -1, dtype=_I32, device=device),
                   torch.tensor([num_pages], dtype=_I32, device=device), page_size=page_size)


def pages_extend(lists: PageLists, new_tokens: torch.Tensor, T: int, *, stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Make room for new_tokens [B] (int32) further tokens of each request, in all at most T: the lists are edited in
    place, and {"seq", "pos", "row": int32 [T], "starts": int32 [B + 1], "first": int32 [B]} says where the tokens go.
    Token t is position pos[t] of request seq[t] (-1, -1 where there is none: padding for cache_append()) and lies in row
    row[t] of the pools; request b's tokens are starts[b] .. starts[b + 1] - 1.  A request for whose tokens there is no
    room gets none of them: first[b] is the length before, or -1 for a request that gets no tokens."""
    if stream is None and lists._index is not None and (paged._plain or paged._bind()):
        got = paged._fast.extend(lists._at, lists._index, new_tokens, T)
        if got is not None:
            return got
    dev = lists.device
    p_new = _expect("new_tokens", new_tokens, _I32, (lists.B,), dev)
    _int32("T", "a number of tokens", T, 0)
    _index(dev)

    def run(s):
        o = {n: _empty((m,), dtype=_I32, device=dev) for n, m in (("seq", T), ("pos", T), ("row", T), ("starts", lists.B + 1), ("first", lists.B))}
        _check(nat.fa_pages_extend(lists.c, p_new, T, o["starts"].data_ptr(), o["first"].data_ptr(), o["seq"].data_ptr(),
                                   o["pos"].data_ptr(), o["row"].data_ptr(), s))
        return o

    return _call(run, dev, stream)


def pages_trim(lists: PageLists, keep: torch.Tensor, *, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Shorten each request to keep [B] (int32) positions, where that is less than it has, and give the pages behind
    them back: drafts that were rejected, or 0 for a request that has ended.  A negative keep leaves a request as it is."""
    if stream is None and lists._index is not None and (paged._plain or paged._bind()) and paged._fast.trim(
            lists._at, lists._index, keep):
        return
    p_keep = _expect("keep", keep, _I32, (lists.B,), lists.device)
    _check(_call(lambda s: nat.fa_pages_trim(lists.c, p_keep, s), lists.device, stream))


class PageBounds(_Held):
    """The bounds of a cache's keys page by page: codes (int8 [num_pages][Hkv][2][D]) and scales (f32
    [num_pages][Hkv][D / 32]): the largest value of a component in a page is about codes[..., 0, :] times its block's
    scale, the smallest codes[..., 1, :] times it, rounded outward.  They bound the keys but for f32's roundings of scale and
    quotient (2^-22 of the block's largest magnitude); a block without a magnitude above 1e-30 counts as zeros, and a NaN is
    left out.  Holds the tensors."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 4 or codes.shape[2] != 2 or codes.shape[3] % 32:
            raise FaBackError("codes: int8 [num_pages][Hkv][2][D] expected")
        n, Hkv, _, D = codes.shape
        self.codes, self.scales, self.device = codes, scales, codes.device
        self.c = nat.fa_page_bounds_pool(_expect("codes", codes, torch.int8, (n, Hkv, 2, D), codes.device),
                                         _expect("scales", scales, _F32, (n, Hkv, D // 32), codes.device))
        self._at, self._dims = ctypes.addressof(self.c), (n, Hkv, D, codes.device)

    @classmethod
    def of(cls, cache: "paged.PagedCache") -> "PageBounds":
        """Room for the bounds of a cache's pages, none of which is known yet."""
        n, Hkv, D, dev = cache._dims
        return cls(torch.zeros((n, Hkv, 2, D), dtype=torch.int8, device=dev), torch.zeros((n, Hkv, D // 32), dtype=_F32, device=dev))

    def _fits(self, cache: "paged.PagedCache") -> None:
        if self._dims != cache._dims:
            raise FaBackError("bounds: of %d pages, %d KV heads of %d on %s, the cache has %d, %d of %d on %s" % (*self._dims, *cache._dims))


def page_bounds(cache: "paged.PagedCache", bounds: PageBounds, seq_lens: torch.Tensor, *, first: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Bring the bounds of the pages of positions first [B] .. seq_lens [B] - 1 (int32) up to date, from the keys that the
    cache holds: after every cache_append(), with the `first` of pages_extend() (None: of all pages; a negative one: of
    none of that sequence)."""
    bounds._fits(cache)
    if stream is None and cache._index is not None and (paged._plain or paged._bind()) and paged._fast.bounds(
            cache._at, cache._index, bounds._at, seq_lens, first):
        return
    dev = cache.device
    p_len = _expect("seq_lens", seq_lens, _I32, (cache.B,), dev)
    p_first = None if first is None else _expect("first", first, _I32, (cache.B,), dev)
    _check(_call(lambda s: nat.fa_page_bounds(cache.c, bounds.c, p_first, p_len, s), dev, stream))


def page_select(q: torch.Tensor, cache: "paged.PagedCache", bounds: PageBounds, seq_lens: torch.Tensor, K: int, *,
                scale: float, first: int = 1, last: int = 1, alibi_slopes: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """For each query q [B][H][D] (as paged_decode() takes it) and KV head, the K pages of its sequence whose bounds promise
    the largest scores, the sequence's `first` first and `last` last ones always among them: int32 [B][Hkv][K], ascending,
    -1 behind the last where the sequence has fewer; what paged_decode() takes as pages, with the same scale (finite, of
    either sign).  The choice is exact: the score is defined to the bit, and of equal ones the lowest page is taken."""
    bounds._fits(cache)
    if stream is None and out is None and workspace is None and cache._index is not None and (paged._plain or paged._bind()):
        got = paged._fast.select(q, cache._at, cache._index, bounds._at, seq_lens, K, scale, first, last, alibi_slopes)
        if got is not None:
            return got
    dev, B, dtype = cache.device, cache.B, q.dtype
    act = _act(dtype)
    H, q_row, q_head = _heads("q", q, B, cache.D, dtype, dev)
    p_len = _expect("seq_lens", seq_lens, _I32, (B,), dev)
    p_alibi = None if alibi_slopes is None else _expect("alibi_slopes", alibi_slopes, _F32, (H,), dev)
    for name, n in (("K", K), ("first", first), ("last", last)):
        _int32(name, "a number of pages", n)
    _index(dev)

    def run(s):
        o = out
        if o is None:
            o = _empty((B, cache.Hkv, max(K, 0)), dtype=_I32, device=dev)
        p_o = _expect("out", o, _I32, (B, cache.Hkv, max(K, 0)), dev)
        need = nat.fa_page_select_workspace_size(cache.c, H, K)
        ws = _empty((need,), dtype=torch.uint8, device=dev) if workspace is None else workspace.get(need)
        _check(nat.fa_page_select(q.data_ptr(), act, q_row, q_head, cache.c, bounds.c, p_len, H, scale, p_alibi, K, first, last,
                                  p_o, ws.data_ptr(), need, s))
        return o

    return _call(run, dev, stream)

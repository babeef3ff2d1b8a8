"""Pages of the paged caches: copying, forking, growing and ending requests,
compacting (Python binding).

A pool of pages is shared by all layers: page ``p`` is block ``p`` of every
array of a ``PageSet``. ``refs`` (int32 ``[num_blocks]``) counts who holds each
page, 0 being free, and request ``r`` holds the first ``ceil(seq_lens[r] /
block_size)`` entries of row ``r`` of ``block_table``. The table and the lengths
have one row for each request here. All calls decide on the device and leave
nothing for the host to wait for, so that a decode step with them can be
captured; they return new tables, lengths and counts, or write them into the
``out_`` tensors, which may be the inputs except where noted. The checks and
the allocations are in the compiled module ``_binding`` (csrc/binding.cpp).
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from ._lib import PageArrayDesc, binding, check, load
from .attention import KVCache, _on

PAGE_UNITS = 2 ** 24 - 1024  # of a page of one array


class PageSet:
    """The arrays whose blocks are the pages of one pool.

    ``caches`` are the layers' ``KVCache`` objects (keys, values and their
    scales). ``arrays`` are any other CUDA tensors ``[num_blocks, ...]`` of the
    same pool, such as the indexer's keys and their scales: each page contiguous
    and of a multiple of 4 bytes, pages any distance apart; of at most 2^24 - 1024
    units of 16 bytes, or of 4 where an address, distance or size is no multiple of
    16 (256 or 64 MB). ``block_size`` is that of the caches, or is given where there
    are none. The object keeps the tensors.
    """

    def __init__(self, caches: Sequence[KVCache] = (), arrays: Sequence[torch.Tensor] = (), *,
                 block_size: Optional[int] = None):
        self.caches, self.arrays = tuple(caches), tuple(arrays)
        every = [(f"caches[{i}]", c.device, c.num_blocks) for i, c in enumerate(self.caches)]
        for i, t in enumerate(self.arrays):
            if not t.is_cuda:
                raise ValueError(f"arrays[{i}] must be on a CUDA device, got {t.device}")
            if t.dim() < 1 or t.numel() == 0:
                raise ValueError(f"arrays[{i}] must be [num_blocks, ...]")
            if not t[0].is_contiguous():
                raise ValueError(f"arrays[{i}] needs contiguous pages")
            if t[0].nbytes % 4:
                raise ValueError(f"arrays[{i}] needs pages of a multiple of 4 bytes")
            if t.shape[0] > 1 and t.stride(0) < t[0].numel():
                raise ValueError(f"arrays[{i}] needs pages that do not overlap")
            step = t.stride(0) * t.element_size() if t.shape[0] > 1 else 0
            unit = 4 if (t.data_ptr() | step | t[0].nbytes) % 16 else 16
            if t[0].nbytes > unit * PAGE_UNITS:
                raise ValueError(f"arrays[{i}] needs pages of {unit * PAGE_UNITS} bytes at most, got {t[0].nbytes}")
            every.append((f"arrays[{i}]", t.device, t.shape[0]))
        if not every:
            raise ValueError("a pool needs at least one cache or array")
        name, self.device, self.num_blocks = every[0]
        for other, device, blocks in every[1:]:
            if device != self.device or blocks != self.num_blocks:
                raise ValueError(f"{other} has {blocks} blocks on {device}, {name} {self.num_blocks} on {self.device}")
        sizes = {c.block_size for c in self.caches} | ({int(block_size)} if block_size is not None else set())
        if len(sizes) != 1:
            raise ValueError("caches of one block_size are needed, or block_size for arrays alone" if not sizes else
                             f"caches and block_size differ: {sorted(sizes)}")
        self.block_size = sizes.pop()
        descs = []
        four = (PageArrayDesc * 4)()
        for c in self.caches:
            n = load().sai_cache_page_arrays(c._ref, ctypes.addressof(four))
            if n < 0:
                check(n, "sai_cache_page_arrays")
            descs += [PageArrayDesc.from_buffer_copy(four[i]) for i in range(n)]
        for t in self.arrays:
            page = t[0].nbytes
            step = t.stride(0) * t.element_size() if t.shape[0] > 1 else page
            descs.append(PageArrayDesc(t.data_ptr(), step, (0, 0), (1, 1), page, -1))
        self._descs = (PageArrayDesc * len(descs))(*descs)
        # an empty copy: the checks of the arrays alone
        check(load().sai_copy_pages(ctypes.addressof(self._descs), len(descs), self.num_blocks, None, None, 0, None), "PageSet")
        self._args = (ctypes.addressof(self._descs), len(descs), self.num_blocks, self.block_size, self.device.index)


def copy_pages(pages: PageSet, src: torch.Tensor, dst: torch.Tensor, *, stream=None) -> None:
    """Page ``dst[i]`` becomes a copy of page ``src[i]`` in every array.

    ``src`` and ``dst`` are int32 ``[n]`` on the pages' device; pairs with a
    negative id, or of a page with itself, are left out. A page may be a source
    more than once; one that is two targets, or a source and a target, ends up
    with a mixture.
    """
    if stream is not None:
        with _on(stream, pages.device):
            return copy_pages(pages, src, dst)
    return binding().copy_pages(*pages._args, src, dst)


def fork_pages(block_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor, *,
               block_size: int, out_table: Optional[torch.Tensor] = None, out_lens: Optional[torch.Tensor] = None,
               out_refs: Optional[torch.Tensor] = None, stream=None):
    """The batch whose request ``i`` continues request ``parents[i]`` (int32;
    -1: none), sharing all its pages; requests that none continues are freed.

    Returns ``(table [children, width], lens [children], refs)``. No page is
    copied: ``resize_pages`` copies a shared, partly filled last page when one of
    its requests grows. ``out_refs`` may be ``refs``; ``out_table`` and
    ``out_lens`` may not overlap the inputs.
    """
    if stream is not None:
        with _on(stream, block_table.device):
            return fork_pages(block_table, seq_lens, refs, parents, block_size=block_size, out_table=out_table,
                              out_lens=out_lens, out_refs=out_refs)
    return binding().fork_pages(block_table, seq_lens, refs, parents, block_size, out_table, out_lens, out_refs)


def resize_pages_workspace(num_blocks: int, requests: int) -> int:
    """Workspace bytes of ``resize_pages`` for these sizes."""
    return int(load().sai_resize_pages_workspace(num_blocks, requests))


def resize_pages(pages: PageSet, block_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor,
                 refs: torch.Tensor, *, out_table: Optional[torch.Tensor] = None, out_lens: Optional[torch.Tensor] = None,
                 out_refs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gives each request the pages that ``new_lens[r]`` tokens need, before
    ``append_kv`` fills them, and takes back those past them (0: all).

    A growing request whose partly filled last page is held by others too gets
    a copy of it first. Pages are taken lowest id first, in the order of requests.
    Returns ``(table, lens, refs)``; ``lens[r]`` is ``new_lens[r]``, or still
    ``seq_lens[r]`` where the pool had no pages left for this request (or one
    before it), which also sets status bit 8. Freed pages can be taken from the
    next call on.
    """
    if stream is not None:
        with _on(stream, pages.device):
            return resize_pages(pages, block_table, seq_lens, new_lens, refs, out_table=out_table, out_lens=out_lens,
                                out_refs=out_refs, workspace=workspace)
    return binding().resize_pages(*pages._args, block_table, seq_lens, new_lens, refs, out_table, out_lens, out_refs,
                                  workspace)


def compact_pages_workspace(num_blocks: int) -> int:
    """Workspace bytes of ``compact_pages`` for these sizes."""
    return int(load().sai_compact_pages_workspace(num_blocks))


def compact_pages(pages: PageSet, block_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor, *,
                  out_table: Optional[torch.Tensor] = None, out_refs: Optional[torch.Tensor] = None,
                  out_moves: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Moves the held pages to the lowest ids, contents, table and counts.

    Held pages at or above their number move, in ascending order, to the free
    ids below it. Returns ``(table, refs, moves)``; ``moves[p]`` (int32
    ``[num_blocks]``) is page ``p``'s new id, -1 for a free one, for whatever else
    names pages.
    """
    if stream is not None:
        with _on(stream, pages.device):
            return compact_pages(pages, block_table, seq_lens, refs, out_table=out_table, out_refs=out_refs,
                                 out_moves=out_moves, workspace=workspace)
    return binding().compact_pages(*pages._args, block_table, seq_lens, refs, out_table, out_refs, out_moves, workspace)

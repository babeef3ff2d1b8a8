"""Paged key/value caches and the attention over them (Python binding).

``KVCache`` names one layer's cache arrays; ``append_kv`` rotates the step's
keys and queries and writes keys and values into it, ``sparse_attention``
attends over the slots that ``index_score_topk`` or ``topk_transform`` picked,
and ``paged_attention`` over all keys of a row or a sliding window of them.
Rows, ``seq_lens``, ``row_to_batch`` and ``block_table`` mean what they mean
for ``index_score_topk``. As everywhere in this package, the computation runs
in libsai.so; this module checks arguments and allocates.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._lib import KVCacheDesc, check, load

_BF16, _E4M3 = 0, 1


class KVCache:
    """One layer's paged cache.

    ``k`` and ``v`` are ``[num_blocks, kv_heads, block_size, dim]`` CUDA
    tensors, torch.bfloat16 or e4m3 codes (torch.uint8 or
    torch.float8_e4m3fn); any strides that keep ``dim`` contiguous and rows 16
    bytes apart work, so a ``[blocks, block_size, heads, dim]`` array is passed
    as ``x.transpose(1, 2)``. An e4m3 cache needs ``k_scale`` and ``v_scale``,
    fp32 ``[num_blocks, kv_heads]``. ``block_size`` is 16, 32, 64 or 128,
    ``dim`` 64 or 128. The object keeps the tensors; their contents are updated
    in place by ``append_kv``.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        self.device = k.device
        if not k.is_cuda or v.device != k.device:
            raise ValueError(f"k and v must be on one CUDA device, got {k.device} and {v.device}")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [num_blocks, kv_heads, block_size, dim]")
        if v.dtype != k.dtype or k.dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
            raise ValueError(f"k and v must both be bfloat16 or e4m3 codes, got {k.dtype} and {v.dtype}")
        f8 = k.dtype != torch.bfloat16
        if f8 != (k_scale is not None) or f8 != (v_scale is not None):
            raise ValueError("k_scale and v_scale go with an e4m3 cache, and only with one")
        blocks, heads, bs, dim = k.shape
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and (t.device != k.device or t.dtype != torch.float32 or t.shape != (blocks, heads)
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous float32 [{blocks}, {heads}] on {k.device}")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v need unit stride along dim")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_blocks, self.heads, self.block_size, self.dim = blocks, heads, bs, dim
        self.dtype = _E4M3 if f8 else _BF16
        self._desc = KVCacheDesc(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if f8 else None, v_scale.data_ptr() if f8 else None, blocks,
            (ctypes.c_int64 * 3)(*k.stride()[:3]), (ctypes.c_int64 * 3)(*v.stride()[:3]), heads, bs, dim, self.dtype)
        self._ref = ctypes.addressof(self._desc)


def _tensor(t, name, dtype, dev, ndim):
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _row_index(t, name, rows, dev):
    _tensor(t, name, torch.int32, dev, 1)
    if t.shape[0] != rows or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{rows}]")
    return t.data_ptr()


def _heads(t, name, rows, heads, cache):
    """Row stride of a bf16 [rows, heads, dim] tensor whose heads are contiguous."""
    _tensor(t, name, torch.bfloat16, cache.device, 3)
    shape, st = t.shape, t.stride()
    if shape[0] != rows or shape[2] != cache.dim or (heads and shape[1] != heads):
        raise ValueError(f"{name} must be [{rows}, {heads or 'heads'}, {cache.dim}], got {list(shape)}")
    if st[2] != 1 or (st[1] != cache.dim and shape[1] > 1):
        raise ValueError(f"{name} needs contiguous heads")
    return st[0] if rows > 1 else shape[1] * cache.dim


def _table(block_table, dev):
    _tensor(block_table, "block_table", torch.int32, dev, 2)
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    return block_table.data_ptr(), block_table.shape[0], block_table.shape[1]


class _On:
    """The launch stream, with the cache's device current; what is allocated
    for a call on another stream than torch's current one is kept for it."""

    __slots__ = ("stream", "handle", "other")

    def __init__(self, stream, dev):
        if dev.index != torch.cuda.current_device():
            raise ValueError(f"the current device is cuda:{torch.cuda.current_device()}, the cache is on {dev}")
        if stream is None:
            self.handle, self.other = torch.cuda.current_stream(dev).cuda_stream, False
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        self.stream, self.handle = stream, stream.cuda_stream
        self.other = self.handle != torch.cuda.current_stream(dev).cuda_stream

    def empty(self, shape, dtype, dev):
        t = torch.empty(shape, dtype=dtype, device=dev)
        if self.other:
            t.record_stream(self.stream)
        return t


def append_kv(cache: KVCache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
              cos_sin: Optional[torch.Tensor] = None, *, q: Optional[torch.Tensor] = None,
              out_q: Optional[torch.Tensor] = None, row_to_batch: Optional[torch.Tensor] = None,
              interleaved: bool = False, stream=None) -> Optional[torch.Tensor]:
    """Rotate ``k`` (and ``q``) by each row's position ``seq_lens[i] - 1`` and
    write ``k`` and ``v`` into the cache at that position of the row's request.

    ``k`` and ``v`` are bf16 ``[rows, kv_heads, dim]``, ``q`` bf16 ``[rows,
    q_heads, dim]`` (any row stride); ``cos_sin`` fp32 ``[max_pos, rot_dim]``
    holds each position's cosines, then its sines (None: no rotation).
    ``interleaved`` pairs dims (2j, 2j+1) instead of (j, j + rot_dim/2). An
    e4m3 cache's block scales are powers of two that grow as the block fills.
    The rows of one request that meet in one block are neighbours, in order.
    Returns the rotated queries (None without ``q``).
    """
    dev = cache.device
    on = _On(stream, dev)
    rows = k.shape[0]
    k_row = _heads(k, "k", rows, cache.heads, cache)
    v_row = _heads(v, "v", rows, cache.heads, cache)
    lens = _row_index(seq_lens, "seq_lens", rows, dev)
    r2b = None if row_to_batch is None else _row_index(row_to_batch, "row_to_batch", rows, dev)
    bt, bt_rows, bt_stride = _table(block_table, dev)
    q_ptr = oq_ptr = cs = None
    q_row = q_heads = max_pos = rot = 0
    if q is not None:
        q_row, q_heads, q_ptr = _heads(q, "q", rows, 0, cache), q.shape[1], q.data_ptr()
        if out_q is None:
            out_q = on.empty(q.shape, torch.bfloat16, dev)
        elif out_q.shape != q.shape or out_q.dtype != torch.bfloat16 or out_q.device != dev or \
                not out_q.is_contiguous():
            raise ValueError("out_q must be contiguous bfloat16 like q")
        oq_ptr = out_q.data_ptr()
    elif out_q is not None:
        raise ValueError("out_q goes with q")
    if cos_sin is not None:
        _tensor(cos_sin, "cos_sin", torch.float32, dev, 2)
        if not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous")
        cs, (max_pos, rot) = cos_sin.data_ptr(), cos_sin.shape
    st = load().sai_append_kv(cache._ref, k.data_ptr(), k_row, v.data_ptr(), v_row, q_ptr, q_row, q_heads, oq_ptr, cs,
                              max_pos, rot, int(interleaved), bt, bt_rows, bt_stride, r2b, lens, rows, on.handle)
    check(st, "sai_append_kv")
    return out_q


@functools.lru_cache(maxsize=1024)
def _paged_workspace(dev, rows, q_heads, heads, dim, dtype, max_seq_len, window, sinks, packed) -> int:
    return int(load().sai_paged_attention_workspace(rows, q_heads, heads, dim, dtype, max_seq_len, window, sinks,
                                                    packed))


def paged_attention_workspace(rows: int, q_heads: int, cache: KVCache, *, max_seq_len: int, window: int = 0,
                              sinks: int = 0, packed: bool = False) -> int:
    """Workspace bytes of ``paged_attention`` for these sizes."""
    return _paged_workspace(cache.device.index, rows, q_heads, cache.heads, cache.dim, cache.dtype, max_seq_len, window,
                            sinks, int(packed))


@functools.lru_cache(maxsize=1024)
def _sparse_workspace(dev, rows, q_heads, heads, dim, dtype, k) -> int:
    return int(load().sai_sparse_attention_workspace(rows, q_heads, heads, dim, dtype, k))


def sparse_attention_workspace(rows: int, q_heads: int, cache: KVCache, k: int) -> int:
    """Workspace bytes of ``sparse_attention`` for these sizes."""
    return _sparse_workspace(cache.device.index, rows, q_heads, cache.heads, cache.dim, cache.dtype, k)


def _attention_args(q, cache, out, want_lse, out_lse, workspace, need, on):
    dev, rows, heads = cache.device, q.shape[0], q.shape[1]
    if out is None:
        out = on.empty((rows, heads, cache.dim), torch.bfloat16, dev)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be contiguous bfloat16 like q")
    if out_lse is None:
        if want_lse:
            out_lse = on.empty((rows, heads), torch.float32, dev)
    elif out_lse.shape != (rows, heads) or out_lse.dtype != torch.float32 or out_lse.device != dev or \
            not out_lse.is_contiguous():
        raise ValueError(f"out_lse must be contiguous float32 [{rows}, {heads}]")
    if workspace is None:
        if need:
            workspace = on.empty((need,), torch.uint8, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}")
    return out, out_lse, workspace


def paged_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                    max_seq_len: int, row_to_batch: Optional[torch.Tensor] = None, packed: bool = False,
                    window: int = 0, sinks: int = 0, sm_scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, want_lse: bool = False,
                    out_lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of each row over the first ``seq_lens[i]`` keys of its request.

    ``q`` is bf16 ``[rows, q_heads, dim]`` (any row stride; ``q_heads`` a
    multiple of the cache's heads). With ``window`` a row sees its last
    ``window`` keys and the request's first ``sinks``. ``packed`` (prefill,
    needs ``row_to_batch``) takes neighbouring rows as tiles. ``sm_scale``
    defaults to ``dim ** -0.5``. Returns ``out`` (bf16, like ``q``), or ``(out,
    lse)`` with ``want_lse`` or ``out_lse`` (fp32 ``[rows, q_heads]``). A row
    that sees no key gives zeros and -inf.
    """
    dev = cache.device
    on = _On(stream, dev)
    rows = q.shape[0]
    q_row = _heads(q, "q", rows, 0, cache)
    lens = _row_index(seq_lens, "seq_lens", rows, dev)
    r2b = None if row_to_batch is None else _row_index(row_to_batch, "row_to_batch", rows, dev)
    if packed and r2b is None:
        raise ValueError("packed rows need row_to_batch")
    bt, bt_rows, bt_stride = _table(block_table, dev)
    heads = q.shape[1]
    max_seq_len, window, sinks, packed = int(max_seq_len), int(window), int(sinks), int(packed)
    need = _paged_workspace(dev.index, rows, heads, cache.heads, cache.dim, cache.dtype, max_seq_len, window, sinks,
                            packed)
    out, out_lse, workspace = _attention_args(q, cache, out, want_lse, out_lse, workspace, need, on)
    st = load().sai_paged_attention(
        q.data_ptr(), q_row, heads, cache._ref, bt, bt_rows, bt_stride, r2b, lens, rows, max_seq_len, window, sinks,
        cache.dim ** -0.5 if sm_scale is None else float(sm_scale), packed, out.data_ptr(),
        None if out_lse is None else out_lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), on.handle)
    check(st, "sai_paged_attention")
    return out if out_lse is None else (out, out_lse)


def sparse_attention(q: torch.Tensor, cache: KVCache, slots: torch.Tensor, *, sm_scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, want_lse: bool = False,
                     out_lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of each row over the cache cells ``slots[i, j] >= 0`` (int32
    ``[rows, k]``, unit column stride: the slots of ``index_score_topk`` or of
    ``topk_transform`` with the cache's block size). Otherwise as
    ``paged_attention``."""
    dev = cache.device
    on = _On(stream, dev)
    rows, heads = q.shape[0], q.shape[1]
    q_row = _heads(q, "q", rows, 0, cache)
    _tensor(slots, "slots", torch.int32, dev, 2)
    k = slots.shape[1]
    if slots.shape[0] != rows or (k > 1 and slots.stride(1) != 1):
        raise ValueError(f"slots must be [{rows}, k] with unit column stride")
    need = _sparse_workspace(dev.index, rows, heads, cache.heads, cache.dim, cache.dtype, k)
    out, out_lse, workspace = _attention_args(q, cache, out, want_lse, out_lse, workspace, need, on)
    st = load().sai_sparse_attention(
        q.data_ptr(), q_row, heads, cache._ref, slots.data_ptr(), slots.stride(0) if rows > 1 else k, k, rows,
        cache.dim ** -0.5 if sm_scale is None else float(sm_scale), out.data_ptr(),
        None if out_lse is None else out_lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), on.handle)
    check(st, "sai_sparse_attention")
    return out if out_lse is None else (out, out_lse)

"""Paged key/value caches and the attention over them (Python binding).

``KVCache`` names one layer's cache arrays; ``append_kv`` rotates the step's
keys and queries and writes keys and values into it, ``sparse_attention``
attends over the slots that ``index_score_topk`` or ``topk_transform`` picked,
and ``paged_attention`` over all keys of a row or a sliding window of them.
Rows, ``seq_lens``, ``row_to_batch`` and ``block_table`` mean what they mean
for ``index_score_topk``; the table may be columns of a wider one, and a length
past its columns makes a bad row. As everywhere in this package, the
computation runs in libsai.so; the checks and the allocations of the calls are
in the compiled module ``_binding`` (csrc/binding.cpp), because a decode step
makes them once a layer.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._lib import KVCacheDesc, binding, load

_BF16, _E4M3 = 0, 1
PACKED_TILES = 2


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
        self._ref, self._index = ctypes.addressof(self._desc), k.device.index


def _on(stream, device):
    """Makes ``stream`` (a torch stream or a cudaStream_t as an integer) the current one, so that the outputs and the
    workspace of a call belong to it."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


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
    if stream is not None:
        with _on(stream, cache.device):
            return append_kv(cache, k, v, block_table, seq_lens, cos_sin, q=q, out_q=out_q, row_to_batch=row_to_batch,
                             interleaved=interleaved)
    return binding().append_kv(cache._ref, cache._index, k, v, block_table, seq_lens, cos_sin, q, out_q, row_to_batch,
                               interleaved)


def paged_attention_workspace(rows: int, q_heads: int, cache: KVCache, *, max_seq_len: int, window: int = 0,
                              sinks: int = 0, packed: int = False) -> int:
    """Workspace bytes of ``paged_attention`` for these sizes."""
    return int(load().sai_paged_attention_workspace(rows, q_heads, cache.heads, cache.dim, cache.dtype, max_seq_len,
                                                    window, sinks, int(packed)))


def sparse_attention_workspace(rows: int, q_heads: int, cache: KVCache, k: int) -> int:
    """Workspace bytes of ``sparse_attention`` for these sizes."""
    return int(load().sai_sparse_attention_workspace(rows, q_heads, cache.heads, cache.dim, cache.dtype, k))


def paged_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                    max_seq_len: int, row_to_batch: Optional[torch.Tensor] = None, packed: int = False,
                    window: int = 0, sinks: int = 0, sm_scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, want_lse: bool = False,
                    out_lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of each row over the first ``seq_lens[i]`` keys of its request.

    ``q`` is bf16 ``[rows, q_heads, dim]`` (any row stride; ``q_heads`` a
    multiple of the cache's heads). With ``window`` a row sees its last
    ``window`` keys and the request's first ``sinks``. ``packed`` (prefill,
    needs ``row_to_batch``) takes neighbouring rows as tiles where their sizes
    make that faster, ``packed=PACKED_TILES`` whatever they are. ``sm_scale``
    defaults to ``dim ** -0.5``. Returns ``out`` (bf16, like ``q``), or ``(out,
    lse)`` with ``want_lse`` or ``out_lse`` (fp32 ``[rows, q_heads]``). A row
    that sees no key gives zeros and -inf.
    """
    if stream is not None:
        with _on(stream, cache.device):
            return paged_attention(q, cache, block_table, seq_lens, max_seq_len=max_seq_len, row_to_batch=row_to_batch,
                                   packed=packed, window=window, sinks=sinks, sm_scale=sm_scale, out=out,
                                   want_lse=want_lse, out_lse=out_lse, workspace=workspace)
    return binding().paged_attention(cache._ref, cache._index, q, block_table, seq_lens, max_seq_len, row_to_batch,
                                     packed, window, sinks, sm_scale, out, want_lse, out_lse, workspace)


def sparse_attention(q: torch.Tensor, cache: KVCache, slots: torch.Tensor, *, sm_scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, want_lse: bool = False,
                     out_lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of each row over the cache cells ``slots[i, j] >= 0`` (int32
    ``[rows, k]``, unit column stride: the slots of ``index_score_topk`` or of
    ``topk_transform`` with the cache's block size). Otherwise as
    ``paged_attention``."""
    if stream is not None:
        with _on(stream, cache.device):
            return sparse_attention(q, cache, slots, sm_scale=sm_scale, out=out, want_lse=want_lse, out_lse=out_lse,
                                    workspace=workspace)
    return binding().sparse_attention(cache._ref, cache._index, q, slots, sm_scale, out, want_lse, out_lse, workspace)

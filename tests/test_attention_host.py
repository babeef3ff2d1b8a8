"""Host-side argument checks of the cache and attention entry points (CPU)."""

import ctypes

import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_top_gb300 import _lib, build

    build.build()
    return _lib.load()


def _desc(**kw):
    from sparse_attention_indexer_top_gb300._lib import KVCacheDesc

    a = dict(k=P, v=P, k_scale=None, v_scale=None, num_blocks=8, k_stride=(2 * 128 * 128, 128 * 128, 128),
             v_stride=(2 * 128 * 128, 128 * 128, 128), heads=2, block_size=128, dim=128, dtype=0)
    a.update(kw)
    d = KVCacheDesc(a["k"], a["v"], a["k_scale"], a["v_scale"], a["num_blocks"], (ctypes.c_int64 * 3)(*a["k_stride"]),
                    (ctypes.c_int64 * 3)(*a["v_stride"]), a["heads"], a["block_size"], a["dim"], a["dtype"])
    return d


def _paged(lib, d, q=P, q_row=8 * 128, hq=8, bt=P, bt_rows=4, r2b=None, lens=P, rows=4, window=0, sinks=0, sm=0.1,
           packed=0, out=P, lse=None):
    return lib.sai_paged_attention(q, q_row, hq, None if d is None else ctypes.addressof(d), bt, bt_rows, 8, r2b, lens,
                                   rows, 1024, window, sinks, sm, packed, out, lse, None, 0, None)


def _sparse(lib, d, slots=P, stride=512, k=512, rows=4, hq=8):
    return lib.sai_sparse_attention(P, hq * 128, hq, ctypes.addressof(d), slots, stride, k, rows, 0.1, P, None, None, 0,
                                    None)


def _append(lib, d, k=P, k_row=256, q=None, oq=None, hq=0, cs=None, rot=0, max_pos=0, bt_rows=4, rows=4):
    return lib.sai_append_kv(ctypes.addressof(d), k, k_row, P, 256, q, hq * 128, hq, oq, cs, max_pos, rot, 0, P,
                             bt_rows, 8, None, P, rows, None)


def test_cache_descriptor(lib):
    assert _paged(lib, None) == -1
    for call in (_paged, _sparse, _append):
        assert call(lib, _desc(dtype=2)) == -3
        assert call(lib, _desc(dim=96)) == -3
        assert call(lib, _desc(block_size=100)) == -3
        assert call(lib, _desc(block_size=8)) == -3
        assert call(lib, _desc(heads=0)) == -2
        assert call(lib, _desc(num_blocks=0)) == -2
        assert call(lib, _desc(num_blocks=1 << 25)) == -2  # slots are 32 bits
        assert call(lib, _desc(k=None)) == -1
        assert call(lib, _desc(dtype=1)) == -1  # an 8-bit cache needs its scales
        assert call(lib, _desc(k=P + 8)) == -7
        assert call(lib, _desc(v_stride=(2 * 128 * 128, 128 * 128, 132))) == -7
        assert call(lib, _desc(k_stride=(-1, 0, 0))) == -2


def test_paged_attention_arguments(lib):
    d = _desc()
    assert _paged(lib, d, rows=-1) == -2
    assert _paged(lib, d, hq=7) == -2
    assert _paged(lib, d, window=-1) == -2
    assert _paged(lib, d, sinks=-1) == -2
    assert _paged(lib, d, sm=float("inf")) == -2
    assert _paged(lib, d, q=None) == -1
    assert _paged(lib, d, q=P + 4) == -7
    assert _paged(lib, d, q_row=1000) == -2
    assert _paged(lib, d, q_row=1028) == -7
    assert _paged(lib, d, out=None) == -1
    assert _paged(lib, d, bt=None) == -1
    assert _paged(lib, d, bt_rows=3) == -2
    assert _paged(lib, d, packed=1) == -1  # tiles need row_to_batch
    assert _paged(lib, d, packed=2) == -1
    assert _paged(lib, d, packed=3) == -3
    assert _paged(lib, d, lse=P + 2) == -7
    assert _paged(lib, d, rows=0, q=None, out=None, bt=None, lens=None) == 0


def test_sparse_attention_arguments(lib):
    d = _desc()
    assert _sparse(lib, d, k=0) == -2
    assert _sparse(lib, d, k=65537, stride=65537) == -2
    assert _sparse(lib, d, slots=None) == -1
    assert _sparse(lib, d, stride=511) == -2
    assert _sparse(lib, d, slots=P + 2) == -7
    assert _sparse(lib, d, hq=3) == -2
    assert _sparse(lib, d, rows=0, slots=None) == 0


def test_append_arguments(lib):
    d = _desc()
    assert _append(lib, d, k=None) == -1
    assert _append(lib, d, k_row=128) == -2
    assert _append(lib, d, k=P + 2) == -7
    assert _append(lib, d, rot=24, cs=P, max_pos=8) == -3
    assert _append(lib, d, rot=256, cs=P, max_pos=8) == -3
    assert _append(lib, d, rot=64) == -1
    assert _append(lib, d, rot=64, cs=P, max_pos=0) == -2
    assert _append(lib, d, rot=64, cs=P + 4, max_pos=8) == -7
    assert _append(lib, d, q=P) == -1  # queries without a place for them
    assert _append(lib, d, q=P, oq=P, hq=0) == -2
    assert _append(lib, d, bt_rows=3) == -2
    assert _append(lib, d, rows=0) == 0


def test_workspace_queries_without_sizes(lib):
    assert lib.sai_paged_attention_workspace(0, 8, 2, 128, 0, 100, 0, 0, 0) == 0
    assert lib.sai_sparse_attention_workspace(4, 8, 2, 128, 0, 0) == 0


def test_host_tensors_are_refused():
    x = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        sai.KVCache(x, x)

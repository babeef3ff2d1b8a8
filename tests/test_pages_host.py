"""Host-side argument checks of the page entry points, and the oracle's invariants (CPU)."""

import ctypes
import random

import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import pages as O

P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_top_gb300 import _lib, build

    build.build()
    return _lib.load()


def _array(**kw):
    from sparse_attention_indexer_top_gb300._lib import PageArrayDesc

    a = dict(base=P, page_stride=65536, stride=(32768, 256), count=(2, 128), row_bytes=256, cells=1)
    a.update(kw)
    return (PageArrayDesc * 1)(PageArrayDesc(a["base"], a["page_stride"], a["stride"], a["count"], a["row_bytes"], a["cells"]))


def _copy(lib, a, n=1, blocks=8, src=P, dst=P, pairs=4):
    return lib.sai_copy_pages(None if a is None else ctypes.addressof(a), n, blocks, src, dst, pairs, None)


def _resize(lib, a=None, n=1, blocks=8, bs=128, table=P, reqs=4, width=4, stride=4, lens=P + 4096, new=P + 8192, refs=P + 12288,
            out=P + 16384, ostride=4, olens=P + 20480, orefs=P + 24576, ws=P, ws_bytes=1 << 20):
    a = _array() if a is None else a
    return lib.sai_resize_pages(ctypes.addressof(a), n, blocks, bs, table, reqs, width, stride, lens, new, refs, out, ostride,
                                olens, orefs, ws, ws_bytes, None)


def _compact(lib, a=None, blocks=8, bs=128, table=P, lens=P + 4096, refs=P + 12288, out=P + 16384, orefs=P + 24576,
             moves=P + 28672, ws=P, ws_bytes=1 << 20):
    a = _array() if a is None else a
    return lib.sai_compact_pages(ctypes.addressof(a), 1, blocks, bs, table, 4, 4, 4, lens, refs, out, 4, orefs, moves, ws,
                                 ws_bytes, None)


def _fork(lib, table=P, reqs=4, width=4, stride=4, lens=P + 4096, bs=128, refs=P + 12288, blocks=8, parents=P + 8192, kids=4,
          out=P + 16384, ostride=4, olens=P + 20480, orefs=P + 24576):
    return lib.sai_fork_pages(table, reqs, width, stride, lens, bs, refs, blocks, parents, kids, out, ostride, olens, orefs, None)


def test_copy_arguments(lib):
    assert _copy(lib, None) == -1
    assert _copy(lib, _array(base=None)) == -1
    assert _copy(lib, _array(), src=None) == -1
    assert _copy(lib, _array(), dst=P + 2) == -7
    assert _copy(lib, _array(), pairs=-1) == -2
    assert _copy(lib, _array(), blocks=0) == -2
    assert _copy(lib, _array(), n=-1) == -2
    assert _copy(lib, _array(base=P + 2)) == -7
    assert _copy(lib, _array(row_bytes=250)) == -7
    assert _copy(lib, _array(page_stride=65538)) == -7
    assert _copy(lib, _array(stride=(32768, 258))) == -7
    assert _copy(lib, _array(stride=(32768, 128))) == -2  # rows that overlap
    assert _copy(lib, _array(count=(0, 128))) == -2
    assert _copy(lib, _array(row_bytes=0)) == -2
    assert _copy(lib, _array(cells=2)) == -2
    assert _copy(lib, _array(count=(1 << 20, 128))) == -2  # a page above 256 MB
    assert _copy(lib, _array(), pairs=0, src=None, dst=None) == 0


def test_fork_arguments(lib):
    assert _fork(lib, table=None) == -1
    assert _fork(lib, refs=None) == -1
    assert _fork(lib, parents=None) == -1
    assert _fork(lib, olens=None) == -1
    assert _fork(lib, width=0) == -2
    assert _fork(lib, stride=3) == -2
    assert _fork(lib, ostride=3) == -2
    assert _fork(lib, bs=0) == -2
    assert _fork(lib, blocks=0) == -2
    assert _fork(lib, kids=-1) == -2
    assert _fork(lib, out=P + 16) == -2  # over rows that are still to be read
    assert _fork(lib, olens=P + 4096) == -2
    assert _fork(lib, olens=P + 8192) == -2
    assert _fork(lib, orefs=P + 12292) == -2
    assert _fork(lib, lens=P + 4098) == -7


def test_resize_and_compact_arguments(lib):
    for call in (_resize, _compact):
        assert call(lib, blocks=0) == -2
        assert call(lib, blocks=(1 << 28) + 1) == -2
        assert call(lib, bs=0) == -2
        assert call(lib, table=None) == -1
        assert call(lib, refs=None) == -1
        assert call(lib, refs=P + 12289) == -7
        assert call(lib, orefs=P + 12292) == -2  # partly over the counts
        assert call(lib, out=P + 16) == -2  # partly over the table
        assert call(lib, ws=None) == -4
        assert call(lib, ws=P + 8) == -4
        assert call(lib, ws_bytes=16) == -4
    assert _resize(lib, new=None) == -1
    assert _resize(lib, width=0) == -2
    assert _resize(lib, olens=P + 4100) == -2
    assert _resize(lib, bs=64) == -2  # the array's tokens are 128 a page
    assert _resize(lib, out=P, ostride=5) == -2  # in place, but of another stride
    assert _compact(lib, moves=None) == -1
    assert _compact(lib, moves=P + 12288) == -2


def test_workspace_queries(lib):
    assert lib.sai_resize_pages_workspace(0, 4) == 0
    assert lib.sai_compact_pages_workspace(0) == 0
    assert lib.sai_resize_pages_workspace(100, 0) > 0
    assert lib.sai_compact_pages_workspace(1 << 28) > 1 << 28


def test_host_tensors_are_refused():
    x = torch.zeros((4, 16), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        sai.PageSet(arrays=[x], block_size=16)
    with pytest.raises(ValueError, match="at least one"):
        sai.PageSet()
    with pytest.raises(ValueError, match="CUDA device"):
        sai.fork_pages(x, x[:, 0].contiguous(), x[0], x[0], block_size=16)


def _held_counts(table, lens, bs, blocks):
    refs = [0] * blocks
    for row, n in zip(table, lens):
        for p in row[:O.pages_of(n, bs)]:
            refs[p] += 1
    return refs


@pytest.mark.parametrize("seed", range(20))
def test_oracle_keeps_the_counts_true(seed):
    """Whatever is forked, grown, ended and compacted, refs count the holders and a page that is written to has one."""
    rng = random.Random(seed)
    bs, blocks, width = rng.choice([1, 4, 16]), 60, 12
    table, lens, refs = [[-1] * width for _ in range(5)], [0] * 5, [0] * blocks
    for step in range(30):
        op = rng.choice(["fork", "resize", "resize", "compact"])
        if op == "fork":
            table, lens, refs = O.fork(table, lens, refs, [rng.randrange(-1, 5) for _ in range(5)], bs)
        elif op == "resize":
            new = [rng.choice([n, n + 1, rng.randint(0, n), rng.randint(0, width * bs)]) for n in lens]
            new = [min(n, width * bs) for n in new]
            before = [list(r) for r in table]
            table, out, refs, copies, refused = O.resize(table, lens, new, refs, bs)
            for r, n in enumerate(lens):
                if r in refused:
                    assert out[r] == n and table[r] == before[r]
                elif new[r] > n:  # the cells to be written lie in pages of its own
                    for j in range(n // bs, O.pages_of(new[r], bs)):
                        assert refs[table[r][j]] == 1
            lens = out
        else:
            table, refs, moves, copies = O.compact(table, lens, refs, bs)
            assert all((r > 0) == (p < sum(x > 0 for x in refs)) for p, r in enumerate(refs))
        assert refs == _held_counts(table, lens, bs, blocks)

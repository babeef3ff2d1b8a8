"""GPU parity of the page operators with the oracle: tables, lengths and counts exactly, contents byte by byte."""

import random

import numpy as np
import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import pages as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _t(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pool:
    """Caches of several layouts and other arrays over one pool, filled with random bytes."""

    def __init__(self, seed, blocks, *, bs=16, hkv=2, dim=64, kinds=("bf16", "e4m3"), nhd=False, extra=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda shape: torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        self.bs, self.blocks, self.token, self.whole = bs, blocks, [], []
        caches = []
        for kind in kinds:
            shape = (blocks, bs, hkv, dim) if nhd else (blocks, hkv, bs, dim)
            raw = [rnd(shape + (2,) if kind == "bf16" else shape) for _ in range(2)]
            kv = [x.view(torch.bfloat16).squeeze(-1) if kind == "bf16" else x for x in raw]
            self.token += [(x, 1 if nhd else 2) for x in raw]
            sc = [rnd((blocks, hkv, 4)).view(torch.float32).squeeze(-1) for _ in range(2)] if kind == "e4m3" else []
            self.whole += [x.view(torch.uint8) for x in sc]
            caches.append(sai.KVCache(*((x.transpose(1, 2) if nhd else x) for x in kv), *sc))
        arrays = []
        if extra:  # pages of odd sizes and distances
            arrays = [rnd((blocks, 37, 4)), rnd((blocks, 3, 7, 16)), rnd((blocks, 260))[:, :52]]
            self.whole += arrays
        self.set = sai.PageSet(caches, arrays, block_size=bs)

    def snapshot(self):
        return [(x.cpu().clone(), axis) for x, axis in self.token] + [(x.cpu().clone(), None) for x in self.whole]

    def check(self, before, copies):
        """copies: (from, to, cells of keys and values or None for whole pages)."""
        for (old, axis), new in zip(before, [x for x, _ in self.token] + self.whole):
            want = old.clone()
            for a, b, n in copies:
                if axis is None or n is None:
                    want[b] = old[a]
                else:
                    sl = (slice(None),) * (axis - 1) + (slice(0, n),)
                    want[b][sl] = old[a][sl]
            assert torch.equal(new.cpu(), want)


def _state(seed, requests, blocks, bs, width, share=3, most=None):
    """Random table, lengths and counts in which groups of requests share pages."""
    rng = random.Random(seed)
    ids = list(range(blocks))
    rng.shuffle(ids)
    table, lens, refs = [], [], [0] * blocks
    while len(table) < requests:
        n = rng.choice([0, 1, bs, rng.randint(0, (most or width * bs))])
        pages = [ids.pop() if ids else None for _ in range(O.pages_of(n, bs))]
        if None in pages:
            n, pages = 0, []
        for _ in range(rng.randint(1, share)):
            if len(table) < requests:
                table.append(pages + [-1] * (width - len(pages)))
                lens.append(n)
                for p in pages:
                    refs[p] += 1
    order = list(range(requests))
    rng.shuffle(order)
    return [table[i] for i in order], [lens[i] for i in order], refs


@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("bs,hkv,dim", [(16, 1, 64), (32, 3, 64), (128, 2, 128), (16, 5, 128)])
def test_copy_pages(bs, hkv, dim, nhd):
    p = Pool(bs + hkv, 40, bs=bs, hkv=hkv, dim=dim, nhd=nhd)
    before = p.snapshot()
    src, dst = [3, 3, 7, -1, 9, 5, 39, 12], [0, 1, 2, 4, -5, 5, 38, 11]
    sai.copy_pages(p.set, _t(src), _t(dst))
    p.check(before, [(a, b, None) for a, b in zip(src, dst) if a >= 0 and b >= 0 and a != b])
    assert sai.device_status() == 0
    sai.copy_pages(p.set, _t([]), _t([]))
    before = p.snapshot()
    sai.copy_pages(p.set, _t([40, 1, 2]), _t([3, 40, 4]))
    p.check(before, [(2, 4, None)])
    assert sai.device_status() == 4


def test_copy_more_arrays_than_a_launch_takes():
    g = torch.Generator(device=DEV).manual_seed(1)
    arrays = [torch.randint(0, 99, (9, 1 + i), generator=g, device=DEV, dtype=torch.int32) for i in range(70)]
    before = [x.clone() for x in arrays]
    sai.copy_pages(sai.PageSet(arrays=arrays, block_size=1), _t([0, 1]), _t([8, 7]))
    for x, y in zip(arrays, before):
        y[8], y[7] = y[0], y[1]
        assert torch.equal(x, y)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,children,blocks,bs,width", [(1, 1, 1, 16, 1), (5, 9, 300, 16, 20), (70, 3, 9001, 1, 40),
                                                              (40, 130, 5000, 128, 33), (3, 0, 100, 16, 9),
                                                              (300, 520, 90001, 16, 70)])
def test_fork(requests, children, blocks, bs, width, in_place):
    table, lens, refs = _state(requests, requests, blocks, bs, width)
    rng = random.Random(children)
    parents = [rng.randrange(-1, requests) for _ in range(children)]
    want = O.fork(table, lens, refs, parents, bs)
    wide = torch.full((requests, width + 5), 77, dtype=torch.int32, device=DEV)
    wide[:, :width] = _t(table)
    t_refs = _t(refs)
    got = sai.fork_pages(wide[:, :width], _t(lens), t_refs, _t(parents), block_size=bs, out_refs=t_refs if in_place else None)
    assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2]
    assert in_place == (got[2].data_ptr() == t_refs.data_ptr()) and (in_place or t_refs.tolist() == refs)
    assert sai.device_status() == 0


def test_fork_bad_metadata():
    table, lens, refs = [[0, 1], [2, 99], [3, -7]], [20, 32, 40], [1, 1, 1, 1, 0]
    got = sai.fork_pages(_t(table), _t(lens), _t(refs), _t([0, 1, 2, 3, -2, 0]), block_size=16)
    # request 2 is too long, 3 and -2 are no requests, page 99 is none
    assert got[0].tolist() == [[0, 1], [2, 99], [-1, -1], [-1, -1], [-1, -1], [0, 1]]
    assert got[1].tolist() == [20, 32, 0, 0, 0, 20] and got[2].tolist() == [2, 2, 1, 1, 0]
    assert sai.device_status() == 1 + 4


def _resize_case(seed, requests, blocks, bs, width, *, nhd=False, in_place=False, free=None):
    rng = random.Random(seed)
    table, lens, refs = _state(seed, requests, blocks, bs, width, most=max(1, min(width * bs, blocks * bs // (2 * requests))))
    top = width * bs
    new = [min(top, rng.choice([n, n + 1, n + 1, n + 1, 0, rng.randint(0, n), n + rng.randint(0, 3 * bs)])) for n in lens]
    if free is not None:  # all but so many of the free pages are held by others
        for page in [p for p, r in enumerate(refs) if r == 0][free:]:
            refs[page] = 1
    p = Pool(seed, blocks, bs=bs, nhd=nhd, kinds=("bf16", "e4m3") if blocks < 50000 else ())
    before = p.snapshot()
    want = O.resize(table, lens, new, refs, bs)
    tt, tl, tn, tr = _t(table), _t(lens), _t(new), _t(refs)
    kw = dict(out_table=tt, out_lens=tl, out_refs=tr) if in_place else {}
    got = sai.resize_pages(p.set, tt, tl, tn, tr, **kw)
    for a, b in zip(got, want):
        assert a.tolist() == b
    p.check(before, want[3])
    assert sai.device_status() == (8 if want[4] else 0)
    if not in_place:
        assert tt.tolist() == table and tl.tolist() == lens and tr.tolist() == refs
    return want


@pytest.mark.parametrize("nhd,in_place", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("requests,blocks,bs,width", [(1, 1, 16, 1), (7, 90, 16, 30), (60, 900, 32, 40), (33, 200, 128, 9),
                                                      (600, 20000, 16, 70), (1100, 20000, 32, 60), (50, 90001, 16, 30)])
def test_resize(requests, blocks, bs, width, nhd, in_place):
    for seed in range(3):
        _resize_case(100 * seed + requests, requests, blocks, bs, width, nhd=nhd, in_place=in_place)


def test_resize_when_the_pool_runs_out():
    for seed in range(12):
        assert _resize_case(seed, 30, 200, 16, 12, free=seed)[4]


def test_resize_last_holder_keeps_the_page():
    p = Pool(1, 8)
    grow = lambda refs, new: sai.resize_pages(p.set, _t([[5, -1]] * 3), _t([10, 10, 12]), _t(new), _t(refs))
    before = p.snapshot()
    table, lens, refs = grow([0, 0, 0, 0, 0, 3, 0, 0], [11, 12, 13])
    assert table.tolist() == [[0, -1], [1, -1], [5, -1]] and refs.tolist() == [1, 1, 0, 0, 0, 1, 0, 0]
    p.check(before, [(5, 0, 10), (5, 1, 10)])
    before = p.snapshot()
    # held by someone else too: all three get copies; and without pages for those before it the last one waits
    table, lens, refs = grow([0, 0, 1, 0, 0, 4, 0, 0], [11, 12, 13])
    assert table.tolist() == [[0, -1], [1, -1], [3, -1]] and refs.tolist() == [1, 1, 1, 1, 0, 1, 0, 0]
    p.check(before, [(5, 0, 10), (5, 1, 10), (5, 3, 12)])
    assert sai.device_status() == 0
    before = p.snapshot()
    table, lens, refs = grow([1, 1, 0, 1, 1, 3, 1, 1], [11, 12, 13])
    assert table.tolist() == [[2, -1], [5, -1], [5, -1]] and lens.tolist() == [11, 10, 12]
    assert refs.tolist() == [1, 1, 1, 1, 1, 2, 1, 1]
    p.check(before, [(5, 2, 10)])
    assert sai.device_status() == 8


def test_resize_bad_metadata():
    p = Pool(2, 6)
    table = [[0, -1], [9, -1], [2, -1], [3, 7], [4, -1]]
    got = sai.resize_pages(p.set, _t(table), _t([16, 5, -1, 20, 3]), _t([33, 6, 4, 16, 3]), _t([1, 0, 1, 1, 1, 0]))
    # too long; a last page that is none; a negative length; a page given back that is none; unchanged
    assert got[0].tolist() == [[0, -1], [9, -1], [2, -1], [3, -1], [4, -1]]
    assert got[1].tolist() == [16, 5, -1, 16, 3] and got[2].tolist() == [1, 0, 1, 1, 1, 0]
    assert sai.device_status() == 1 + 4


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,blocks,bs,width", [(1, 1, 16, 1), (4, 33, 16, 9), (30, 500, 32, 20), (9, 8193, 16, 70),
                                                      (90, 30000, 16, 100), (200, 80000, 16, 90)])
def test_compact(requests, blocks, bs, width, in_place):
    for seed in range(3):
        table, lens, refs = _state(seed, requests, blocks, bs, width)
        if seed == 1:  # most of the pool held by others
            rng = random.Random(5)
            refs = [r or int(rng.random() < 0.7) for r in refs]
        p = Pool(seed, blocks, bs=bs, kinds=("e4m3",) if blocks < 50000 else ())
        before = p.snapshot()
        want = O.compact(table, lens, refs, bs)
        tt, tr = _t(table), _t(refs)
        got = sai.compact_pages(p.set, tt, _t(lens), tr, **(dict(out_table=tt, out_refs=tr) if in_place else {}))
        for a, b in zip(got, want):
            assert a.tolist() == b
        p.check(before, [(a, b, None) for a, b in want[3]])
        assert sai.device_status() == 0


@pytest.mark.parametrize("every", [0, 1])
def test_compact_empty_and_full_pools(every):
    p = Pool(3, 70)
    before = p.snapshot()
    got = sai.compact_pages(p.set, _t([[-1]]), _t([0]), _t([every] * 70))
    assert got[0].tolist() == [[-1]] and got[1].tolist() == [every] * 70
    assert got[2].tolist() == (list(range(70)) if every else [-1] * 70)
    p.check(before, [])


def test_compact_bad_metadata():
    p = Pool(4, 6)
    table = [[5, -9], [3, 8], [1, -1], [5, 0]]
    got = sai.compact_pages(p.set, _t(table), _t([16, 32, 16, 99]), _t([0, 0, 0, 1, 0, 1]))
    assert got[0].tolist() == [[1, -9], [0, 8], [-1, -1], [5, 0]]  # no page 8; page 1 is free; too long
    assert got[1].tolist() == [1, 1, 0, 0, 0, 0] and got[2].tolist() == [-1, -1, -1, 0, -1, 1]
    assert sai.device_status() == 1 + 4


def test_more_arrays_than_a_launch_takes():
    """Rows are written by the first launch of a call, copies by each."""
    p = Pool(8, 60, kinds=("e4m3", "bf16") * 7)
    before = p.snapshot()
    table, lens, refs = [[59, 40, -1], [59, 40, -1], [7, -1, -1]], [20, 30, 16], [0] * 60
    refs[59] = refs[40] = 2
    refs[7] = 1
    new = [21, 33, 17]
    want = O.resize(table, lens, new, refs, 16)
    got = sai.resize_pages(p.set, _t(table), _t(lens), _t(new), _t(refs))
    assert [x.tolist() for x in got] == list(want[:3])
    p.check(before, want[3])
    before = p.snapshot()
    want = O.compact(want[0], want[1], want[2], 16)
    got = sai.compact_pages(p.set, *got)
    assert [x.tolist() for x in got] == list(want[:3]) and want[3]
    p.check(before, [(a, b, None) for a, b in want[3]])
    assert sai.device_status() == 0


def test_no_requests():
    p = Pool(9, 20)
    none, row, refs = torch.zeros((0, 3), dtype=torch.int32, device=DEV), _t([]), [0] * 20
    refs[4], refs[19] = 1, 3
    before = p.snapshot()
    got = sai.resize_pages(p.set, none, row, row, _t(refs))
    assert got[0].shape == (0, 3) and got[2].tolist() == refs
    got = sai.fork_pages(none, row, _t(refs), _t([-1, -1]), block_size=16)
    assert [x.tolist() for x in got] == [[[-1] * 3] * 2, [0, 0], refs]
    got = sai.fork_pages(none, row, _t(refs), row, block_size=16)
    assert got[0].shape == (0, 3) and got[2].tolist() == refs
    p.check(before, [])
    got = sai.compact_pages(p.set, none, row, _t(refs))
    assert got[1].tolist() == [1, 3] + [0] * 18 and got[2].tolist() == [-1] * 4 + [0] + [-1] * 14 + [1]
    p.check(before, [(4, 0, None), (19, 1, None)])
    assert sai.device_status() == 0


def test_a_large_pool_has_longer_chunks():
    blocks = 5_000_001  # above 512 chunks of 8192 pages
    refs = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    refs[:4_990_000] = 1
    x = torch.arange(blocks, dtype=torch.int32, device=DEV)
    pages = sai.PageSet(arrays=[x], block_size=1)
    table, lens, out = sai.resize_pages(pages, _t([[-1] * 3, [-1] * 3]), _t([0, 0]), _t([3, 2]), refs)
    assert table.tolist() == [[4_990_000, 4_990_001, 4_990_002], [4_990_003, 4_990_004, -1]] and int(out.sum()) == 4_990_005
    refs[:] = 0
    refs[[7, 4_000_000, 5_000_000]] = _t([1, 2, 3])
    table, out, moves = sai.compact_pages(pages, _t([[5_000_000, 7]]), _t([2]), refs)
    assert moves[[7, 4_000_000, 5_000_000]].tolist() == [0, 1, 2] and out[:4].tolist() == [1, 2, 3, 0]
    assert table.tolist() == [[2, 0]] and x[:3].tolist() == [7, 4_000_000, 5_000_000]
    assert sai.device_status() == 0


def test_graph_of_a_decode_step():
    """fork, resize and compact captured together and replayed on changed inputs."""
    bs, blocks, width, n = 16, 64, 6, 8
    p = Pool(6, blocks, bs=bs)
    table, lens, refs = _state(3, n, blocks, bs, width, most=60)
    tt, tl, tr, parents, plus = _t(table), _t(lens), _t(refs), _t(list(range(n))), _t([0] * n)
    stream = torch.cuda.Stream()

    def step():
        t, l, r = sai.fork_pages(tt, tl, tr, parents, block_size=bs)
        t, l, r = sai.resize_pages(p.set, t, l, l + plus, r)
        t2, r2, m = sai.compact_pages(p.set, t, l, r)
        return t2, l, r2, m

    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
    rng = random.Random(9)
    for _ in range(3):
        pv = [rng.randrange(-1, n) for _ in range(n)]
        parents.copy_(_t(pv))
        t, l, r = O.fork(table, lens, refs, pv, bs)
        add = [min(rng.randint(0, 20), width * bs - x) for x in l]
        plus.copy_(_t(add))
        before = p.snapshot()
        graph.replay()
        torch.cuda.synchronize()
        t, l, r, copies, refused = O.resize(t, l, [a + b for a, b in zip(l, add)], r, bs)
        t, r, m, moved = O.compact(t, l, r, bs)
        assert [x.tolist() for x in got] == [t, l, r, m] and not refused
        state = [(x.clone(), a) for x, a in before]
        for x, axis in state:
            src = x.clone()
            for a, b, c in copies:
                if axis is None:
                    x[b] = src[a]
                else:
                    sl = (slice(None),) * (axis - 1) + (slice(0, c),)
                    x[b][sl] = src[a][sl]
        p.check(state, [(a, b, None) for a, b in moved])


def test_streams_and_refusals():
    p = Pool(7, 8)
    t, l, r = _t([[0, 1]]), _t([20]), _t([1, 1, 0, 0, 0, 0, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = sai.resize_pages(p.set, t, l, _t([32]), r, stream=s)
    s.synchronize()
    assert out[1].tolist() == [32]
    with pytest.raises(ValueError, match="must be torch.int32"):
        sai.copy_pages(p.set, l.long(), l)
    with pytest.raises(ValueError, match="one length"):
        sai.copy_pages(p.set, l, t[0])
    with pytest.raises(ValueError, match="refs must be contiguous"):
        sai.resize_pages(p.set, t, l, l, r[:7])
    with pytest.raises(ValueError, match="seq_lens must be contiguous"):
        sai.resize_pages(p.set, t, t[0], l, r)
    with pytest.raises(ValueError, match="out_table must be"):
        sai.compact_pages(p.set, t, l, r, out_table=_t([[1]]))
    with pytest.raises(ValueError, match="workspace"):
        sai.compact_pages(p.set, t, l, r, workspace=torch.zeros(4, dtype=torch.uint8))
    with pytest.raises(sai.SaiError, match="workspace"):
        sai.compact_pages(p.set, t, l, r, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(sai.SaiError):
        sai.fork_pages(t, l, r, _t([0]), block_size=16, out_table=t)
    with pytest.raises(sai.SaiError):
        sai.fork_pages(t, l, r, _t([0]), block_size=0)
    with pytest.raises(ValueError, match="blocks"):
        sai.PageSet(p.set.caches, [torch.zeros((9, 4), device=DEV)])
    with pytest.raises(ValueError, match="multiple of 4"):
        sai.PageSet(p.set.caches, [torch.zeros((8, 3), device=DEV, dtype=torch.uint8)])
    with pytest.raises(ValueError, match="contiguous pages"):
        sai.PageSet(p.set.caches, [torch.zeros((8, 4, 4), device=DEV).transpose(1, 2)])
    with pytest.raises(ValueError, match="differ"):
        sai.PageSet(p.set.caches, block_size=32)
    assert sai.device_status() == 0

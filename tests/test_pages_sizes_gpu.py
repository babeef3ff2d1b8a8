"""GPU tests of the page operators at sizes where they change their ways: many requests, large pages."""

import random

import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import pages as O
from test_pages_gpu import DEV, Pool, _state, _t
from timing import least_us

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests", [127, 128, 129, 512, 513, 2049, 5000])
@pytest.mark.parametrize("short", [False, True])
def test_resize_of_many_requests_that_share_last_pages(requests, short):
    """Groups of up to four requests on one page, spread over all requests, all growing or not, held by others too or not."""
    bs, width, blocks = 16, 3, 3 * requests + 100
    rng = random.Random(requests)
    table, lens, refs = _state(requests, requests, blocks, bs, width, share=4, most=2 * bs - 1)
    new = [min(width * bs, n + rng.choice([1, 1, 1, 5, 20, 0])) for n in lens]
    for page in rng.sample(range(blocks), blocks // 50):
        refs[page] += refs[page] > 0
    if short:  # the pool runs out
        for page in [p for p, r in enumerate(refs) if r == 0][requests // 2:]:
            refs[page] = 1
    p = Pool(requests, blocks, bs=bs, kinds=("bf16",), extra=False)
    before = p.snapshot()
    want = O.resize(table, lens, new, refs, bs)
    kept = sum(1 for r, row in enumerate(table) if new[r] > lens[r] and lens[r] % bs and refs[row[lens[r] // bs]] > 1
               and want[0][r][lens[r] // bs] == row[lens[r] // bs] and want[1][r] == new[r])
    assert kept > requests // 200 and short == bool(want[4])  # the last holder's rule is at work
    got = sai.resize_pages(p.set, _t(table), _t(lens), _t(new), _t(refs))
    assert [x.tolist() for x in got] == list(want[:3])
    p.check(before, want[3])
    assert sai.device_status() == (8 if want[4] else 0)


def _growing(requests):
    """Pairs of requests, far apart, on one partly filled page each; all of them grow."""
    half = requests // 2
    table = torch.arange(half, dtype=torch.int32, device=DEV).repeat(2)[:, None].contiguous()
    refs = torch.zeros(requests + 8, dtype=torch.int32, device=DEV)
    refs[:half] = 2
    lens = torch.full((requests,), 3, dtype=torch.int32, device=DEV)
    pages = sai.PageSet(arrays=[torch.arange(requests + 8, dtype=torch.int32, device=DEV)], block_size=16)
    return pages, table, lens, lens + 1, refs


def test_resize_time_grows_with_the_requests_alone():
    def us(n):
        pages, table, lens, new, refs = _growing(n)
        got = sai.resize_pages(pages, table, lens, new, refs)
        half = n // 2
        assert torch.equal(got[0][:, 0], torch.cat([torch.arange(half, n), torch.arange(half)]).int().to(DEV))
        assert int(got[2].sum()) == n and int(got[2].max()) == 1
        return least_us(lambda: sai.resize_pages(pages, table, lens, new, refs))

    small, large = us(16384), us(131072)
    assert large < 20 * small, (small, large)  # eight times the requests


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,children", [(3, 5000), (300, 320), (300, 321), (5000, 9000), (200, 300)])
def test_fork_of_many_children(requests, children, in_place):
    bs, width, blocks = 16, 5, 2 * requests + 50  # 64 children a column
    table, lens, refs = _state(requests, requests, blocks, bs, width, most=30)
    rng = random.Random(children)
    parents = [rng.randrange(-1, requests) for _ in range(children)]
    counts = [0] * requests
    for r in parents:
        if r >= 0:
            counts[r] += 1
    want = list(refs)
    for r, row in enumerate(table):
        for page in row[:O.pages_of(lens[r], bs)]:
            want[page] += counts[r] - 1
    t_refs = _t(refs)
    got = sai.fork_pages(_t(table), _t(lens), t_refs, _t(parents), block_size=bs, out_refs=t_refs if in_place else None)
    assert got[0].tolist() == [table[r] if r >= 0 else [-1] * width for r in parents]
    assert got[1].tolist() == [lens[r] if r >= 0 else 0 for r in parents] and got[2].tolist() == want
    assert sai.device_status() == 0


@pytest.mark.parametrize("blocks,width", [(6912, 20), (6913, 20), (2000, 64), (2000, 65)])
def test_fork_in_a_cluster_and_in_two_launches(blocks, width):
    """Up to 8192 entries, of the 64 rows among them, and 64 columns are one launch."""
    table, lens, refs = _state(blocks, 30, blocks, 16, width)
    rng = random.Random(blocks)
    for _ in range(3):
        parents = [rng.randrange(-1, 30) for _ in range(34)]
        want = O.fork(table, lens, refs, parents, 16)
        got = sai.fork_pages(_t(table), _t(lens), _t(refs), _t(parents), block_size=16)
        assert [x.tolist() for x in got] == list(want)
    assert sai.device_status() == 0


def test_fork_of_many_children_with_bad_metadata():
    table, lens, refs = [[0, 1], [2, 99], [3, -7]], [20, 32, 40], [1, 1, 1, 1, 0]
    parents = [0, 1, 2, 3, -2] + [0] * 5000 + [1] * 9
    got = sai.fork_pages(_t(table), _t(lens), _t(refs), _t(parents), block_size=16)
    # request 2 is too long, 3 and -2 are no requests, page 99 is none
    assert got[0][:6].tolist() == [[0, 1], [2, 99], [-1, -1], [-1, -1], [-1, -1], [0, 1]] and got[0][-1].tolist() == [2, 99]
    assert got[1][:6].tolist() == [20, 32, 0, 0, 0, 20] and got[2].tolist() == [5001, 5001, 10, 1, 0]
    assert sai.device_status() == 1 + 4


def test_fork_time_grows_with_the_requests_alone():
    def us(n):
        table = torch.arange(n, dtype=torch.int32, device=DEV)[:, None].contiguous()
        lens, refs = torch.full((n,), 5, dtype=torch.int32, device=DEV), torch.ones(n, dtype=torch.int32, device=DEV)
        parents = torch.arange(n, dtype=torch.int32, device=DEV).flip(0).contiguous()
        got = sai.fork_pages(table, lens, refs, parents, block_size=16)
        assert torch.equal(got[0], table.flip(0)) and torch.equal(got[2], refs)
        return least_us(lambda: sai.fork_pages(table, lens, refs, parents, block_size=16))

    small, large = us(65536), us(524288)
    assert large < 20 * small, (small, large)  # eight times the requests


def test_page_sizes_are_refused_by_their_units():
    """Pages of 2^24 - 1024 units at most, of 16 bytes, or of 4 where something is no multiple of 16."""
    wide, narrow = 16 * (2 ** 24 - 1024), 4 * (2 ** 24 - 1024)
    raw = torch.zeros(wide + 64, dtype=torch.uint8, device=DEV)
    sai.PageSet(arrays=[raw[:wide][None]], block_size=1)
    sai.PageSet(arrays=[raw[4:4 + narrow][None]], block_size=1)
    sai.PageSet(arrays=[raw[:narrow][None]], block_size=1)
    for x in (raw[:wide + 16][None], raw[4:8 + narrow][None], raw[:narrow + 4][None], raw[4:4 + wide][None],
              torch.as_strided(raw, (2, narrow + 16), (narrow + 20, 1))):
        with pytest.raises(ValueError, match="bytes at most"):
            sai.PageSet(arrays=[x], block_size=1)

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

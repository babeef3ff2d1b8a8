"""GPU parity of the attention with changed scores and masks against the float64 oracle.

The error bound is that of test_attention_gpu.py, with a larger score error d: the cap's slope is at most 1, so it hands
on the product's error, and is off itself by 8 * 2^-24 of |x| (near 0) or of the cap (beyond: exp2, reciprocal, one
product and one sum of fp32 each); the bias is off by 4 * 2^-24 of the largest slope * distance (slope in log2 units,
the distance's product in two parts, one sum), and the sums that hold cap and bias round once more.
"""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import attention as A
from test_attention_gpu import DEV, LENS, Case, _lens

pytestmark = pytest.mark.gpu


def _check(case, q64, cells, out, lse, sm, *, softcap=0.0, slopes=None):
    """cells: for each row the (request, length, positions) it sees."""
    out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    sl = None if slopes is None else slopes.double().cpu().numpy()
    for i, (b, n, at) in enumerate(cells):
        if not len(at):
            assert (out[i] == 0).all() and np.isneginf(lse[i]).all(), i
            continue
        k, v = (x[at] for x in case.kv[b])
        dist = np.abs(n - 1 - at).astype(np.float64)
        ref, rl, mag = A.attend_changed(q64[i], k, v, sm, softcap, sl, dist)
        grp = q64.shape[1] // case.hkv
        heads = range(q64.shape[1])
        size = np.array([np.abs(k[:, a // grp]).dot(np.abs(q64[i, a])).max() for a in heads]) * abs(sm)
        d = (case.dim + 8) * 2.0 ** -23 * size
        top = np.array([np.abs(k[:, a // grp].dot(q64[i, a])).max() for a in heads]) * abs(sm)
        if softcap:
            d = d + 8 * 2.0 ** -24 * (np.minimum(top, softcap) if (top <= softcap).all() else softcap)
        if sl is not None:
            d = d + 2.0 ** -24 * (4 * np.abs(sl) * dist.max() + top)
        d = d[:, None]
        err = np.abs(out[i] - ref)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 4 * d) * mag
        assert (err <= tol).all(), (i, float((err / tol).max()))
        assert (np.abs(lse[i] - rl) <= 2 * d[:, 0] + 2.0 ** -19 * (1 + np.abs(rl))).all(), (i, np.abs(lse[i] - rl).max())


def _slopes(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq)


MODS = [dict(softcap=30.0), dict(slopes=True), dict(softcap=3.0, slopes=True)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("hkv,group,bs,dim", [(2, 1, 128, 64), (2, 3, 16, 128), (1, 16, 64, 128), (2, 17, 32, 64), (1, 64, 128, 128),
                                              (1, 70, 128, 64)])
def test_decode_rows(dtype, mod, hkv, group, bs, dim):
    c = Case(10 + dim + group, LENS, dtype=dtype, hkv=hkv, dim=dim, bs=bs)
    q, q64 = c.queries(len(LENS), hkv * group)
    slopes = _slopes(hkv * group) if mod.get("slopes") else None
    cap = mod.get("softcap", 0.0)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(LENS), max_seq_len=1000, want_lse=True, softcap=cap, slopes=slopes)
    _check(c, q64, [(b, n, A.span(n)) for b, n in enumerate(LENS)], out, lse, dim ** -0.5, softcap=cap, slopes=slopes)
    assert sai.device_status() == 0


def _spans(seed, totals, rows, docs=True, prefixes=True):
    """Random rows of the requests, neighbours in order: (request, length, start, prefix), some empty or all alone."""
    rng = np.random.default_rng(seed)
    got = []
    for b, t in enumerate(totals):
        for n in sorted(rng.integers(0, t + 1, rows)):
            start = int(rng.integers(0, n + 2)) if docs and rng.random() < 0.8 else 0
            prefix = int(rng.integers(0, t + 1)) if prefixes and rng.random() < 0.6 else 0
            got.append((b, int(n), min(start, t), prefix))
    return got


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("packed", [0, 1, sai.PACKED_TILES])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (130, 70), (1, 1), (3000, 5)])
def test_documents_and_prefixes(dtype, packed, window, sinks):
    totals = [700, 1, 333]
    c = Case(50 + window, totals, dtype=dtype, bs=32, hkv=2)
    spans = _spans(window + sinks, totals, 60)
    q, q64 = c.queries(len(spans), 8)
    b, n, start, prefix = (_lens(list(x)) for x in zip(*spans))
    cells = [(b, n, A.span(n, window, sinks, s, p)) for b, n, s, p in spans]
    for mod in (dict(), dict(softcap=10.0), dict(slopes=_slopes(8)), dict(softcap=10.0, slopes=_slopes(8))):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=700, row_to_batch=b, packed=packed, window=window,
                                       sinks=sinks, want_lse=True, row_starts=start, prefix_lens=prefix, **mod)
        _check(c, q64, cells, out, lse, 128 ** -0.5, **mod)
    # one of the two alone
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=700, row_to_batch=b, packed=packed, window=window,
                                   sinks=sinks, want_lse=True, row_starts=start)
    _check(c, q64, [(b, n, A.span(n, window, sinks, s, 0)) for b, n, s, p in spans], out, lse, 128 ** -0.5)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=700, row_to_batch=b, packed=packed, window=window,
                                   sinks=sinks, want_lse=True, prefix_lens=prefix)
    _check(c, q64, [(b, n, A.span(n, window, sinks, 0, p)) for b, n, s, p in spans], out, lse, 128 ** -0.5)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("hkv,group,dim,bs", [(1, 1, 128, 64), (2, 7, 64, 128), (1, 64, 128, 16), (1, 128, 64, 32), (4, 8, 128, 128)])
def test_packed_tiles(dtype, mod, hkv, group, dim, bs):
    totals = [300, 41, 129]
    c = Case(70 + group, totals, dtype=dtype, hkv=hkv, dim=dim, bs=bs)
    rows = [(b, n) for b, t in enumerate(totals) for n in range(max(1, t - 40), t + 1)] + [(0, 0)]
    q, q64 = c.queries(len(rows), hkv * group)
    slopes = _slopes(hkv * group) if mod.get("slopes") else None
    cap = mod.get("softcap", 0.0)
    b, n = (_lens(list(x)) for x in zip(*rows))
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=300, row_to_batch=b, packed=sai.PACKED_TILES, want_lse=True,
                                   softcap=cap, slopes=slopes)
    _check(c, q64, [(b, n, A.span(n)) for b, n in rows], out, lse, dim ** -0.5, softcap=cap, slopes=slopes)
    assert sai.device_status() == 0


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_long_rows_are_split_and_joined(dtype, packed):
    total, rows = 9000, 5
    c = Case(80, [total], dtype=dtype, bs=64, hkv=1)
    q, q64 = c.queries(rows, 4, sigma=4.0)
    n = list(range(total - rows + 1, total + 1))
    start, prefix = [0, 4000, 8990, 17, 9000], [0, 0, 9000, 8999, 0]
    slopes = 0.01 * _slopes(4)
    zero = _lens([0] * rows)
    for w, s in ((0, 0), (3001, 200)):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(n), max_seq_len=total, row_to_batch=zero, packed=packed,
                                       want_lse=True, softcap=20.0, slopes=slopes, row_starts=_lens(start),
                                       prefix_lens=_lens(prefix), window=w, sinks=s)
        _check(c, q64, [(0, m, A.span(m, w, s, a, p)) for m, a, p in zip(n, start, prefix)], out, lse, 128 ** -0.5, softcap=20.0,
               slopes=slopes)


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("dtype,any_scales", [("bf16", False), ("e4m3", False), ("e4m3", True)])
@pytest.mark.parametrize("cap,sigma", [(0.5, 8.0), (2.0, 2.0), (1000.0, 2.0), (1e6, 2.0)])
def test_caps_far_below_and_above_the_scores(packed, dtype, any_scales, cap, sigma):
    lens = [200, 129, 77, 1]
    c = Case(90, lens, dtype=dtype, bs=16, any_scales=any_scales, vscales=(-8, -5) if dtype == "bf16" else (-12, -2))
    q, q64 = c.queries(4, 8, sigma=sigma)
    slopes = _slopes(8)
    r2b = _lens([0, 1, 2, 3])
    for sl in (None, slopes):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=200, row_to_batch=r2b, packed=packed,
                                       want_lse=True, softcap=cap, slopes=sl)
        _check(c, q64, [(b, n, A.span(n)) for b, n in enumerate(lens)], out, lse, 128 ** -0.5, softcap=cap, slopes=sl)


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("cap", [0.0, 7.0, 60.0])
def test_slopes_of_either_sign_and_zero(packed, dtype, cap):
    """Slopes below 0 favour far keys: every tile then moves the maximum; prefixes put keys on both sides of the position."""
    totals = [900, 500]
    c = Case(91, totals, dtype=dtype, bs=64, hkv=1)
    rows = [(0, n, 0) for n in range(850, 901, 7)] + [(0, 300, 900), (0, 1, 900), (0, 129, 260)] + [(1, n, 0) for n in (1, 2, 130, 500)]
    q, q64 = c.queries(len(rows), 6)
    slopes = torch.tensor([-0.05, -0.001, 0.0, 0.001, 0.3, -2.0], device=DEV)
    b, n, prefix = (_lens(list(x)) for x in zip(*rows))
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=900, row_to_batch=b, packed=packed, want_lse=True,
                                   softcap=cap, slopes=slopes, prefix_lens=prefix)
    _check(c, q64, [(b, n, A.span(n, prefix=p)) for b, n, p in rows], out, lse, 128 ** -0.5, softcap=cap, slopes=slopes)


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
def test_scores_of_zero_under_the_least_cap(packed):
    c = Case(92, [50], dtype="bf16", bs=16, hkv=1)
    q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device=DEV)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([50]), max_seq_len=50, row_to_batch=_lens([0]), packed=packed,
                                   want_lse=True, softcap=1e-30, sm_scale=1e15)
    assert torch.allclose(lse, torch.full_like(lse, float(np.log(50))), atol=1e-5)
    mean = c.kv[0][1].mean(0)
    assert np.abs(out[0].float().cpu().numpy() - mean).max() <= 2.0 ** -6 * np.abs(c.kv[0][1]).mean()


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
def test_infinite_scores_are_capped(packed):
    """A key of infinities: the product is +inf, its capped score the cap; without a cap such a row is NaN."""
    c = Case(95, [60], dtype="bf16", bs=64, hkv=1)
    q = torch.ones((1, 4, 128), dtype=torch.bfloat16, device=DEV)
    c.k[int(c.table[0, 0]), 0, 7] = float("inf")
    c.kv[0][0][7] = 1e30
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([60]), max_seq_len=60, row_to_batch=_lens([0]), packed=packed,
                                   want_lse=True, softcap=5.0)
    ref, rl, mag = A.attend_changed(np.ones((4, 128)), *c.kv[0], 128 ** -0.5, 5.0)
    assert np.abs(lse.cpu().numpy()[0] - rl).max() < 1e-4
    assert (np.abs(out[0].float().cpu().numpy() - ref) <= 2.0 ** -7 * mag + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_nonfinite_values_reach_only_the_rows_that_see_them(dtype, packed):
    totals = [260]
    c = Case(97, totals, dtype=dtype, bs=32)
    at = 100
    c.v.view(torch.uint8 if dtype == "e4m3" else c.v.dtype)[int(c.table[0, at // 32]), :, at % 32, 3] = 0x7F if dtype == "e4m3" else float("nan")
    n = [90, 101, 150, 260, 260, 95]
    start = [0, 0, 101, 100, 200, 0]
    prefix = [0, 0, 0, 0, 0, 101]
    seen = [False, True, False, True, False, True]
    q, q64 = c.queries(6, 4)
    slopes = _slopes(4)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(n), max_seq_len=260, row_to_batch=_lens([0] * 6), packed=packed,
                                   want_lse=True, softcap=8.0, slopes=slopes, row_starts=_lens(start), prefix_lens=_lens(prefix))
    nan = torch.isnan(out[:, :, 3]).cpu()
    assert (nan == torch.tensor(seen)[:, None]).all()
    keep = [d for d in range(128) if d != 3]
    assert torch.isfinite(out[:, :, keep]).all()
    c.kv[0][1][at, :, 3] = 0.0
    out[:, :, 3] = 0.0
    o64 = out.float().cpu().double().numpy()
    for i in range(6):
        cells = A.span(n[i], 0, 0, start[i], prefix[i])
        k, v = (x[cells] for x in c.kv[0])
        ref, rl, mag = A.attend_changed(q64[i], k, v, 128 ** -0.5, 8.0, slopes.double().cpu().numpy(), np.abs(n[i] - 1 - cells))
        ref[:, 3] = mag[:, 3] = 0
        assert (np.abs(o64[i] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag).all(), i


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,k", [(4, 1), (16, 100), (64, 512)])
def test_sparse_softcap(dtype, hq, k):
    lens = [600, 3, 0, 512]
    c = Case(99 + k, lens, dtype=dtype, bs=64)
    q, q64 = c.queries(4, hq, sigma=4.0)
    rng = np.random.default_rng(k)
    slots, cells = np.full((4, k), -1, np.int32), []
    for b, n in enumerate(lens):
        at = rng.permutation(n)[:k]
        slots[b, rng.permutation(k)[:len(at)]] = [c.slot(b, t) for t in at]
        cells.append((b, n, at))
    out, lse = sai.sparse_attention(q, c.cache, torch.from_numpy(slots).to(DEV), want_lse=True, softcap=4.0)
    _check(c, q64, cells, out, lse, 128 ** -0.5, softcap=4.0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("window,sinks", [(0, 0), (65, 9)])
def test_masks_that_hide_nothing_change_nothing(dtype, packed, window, sinks):
    totals = [500, 90]
    c = Case(3, totals, dtype=dtype, bs=32)
    rows = [(b, n) for b, t in enumerate(totals) for n in range(1, t + 1, 3)]
    q, _ = c.queries(len(rows), 8)
    b, n = (_lens(list(x)) for x in zip(*rows))
    kw = dict(max_seq_len=500, row_to_batch=b, packed=packed, window=window, sinks=sinks, want_lse=True)
    plain = sai.paged_attention(q, c.cache, c.t_table, n, **kw)
    same = sai.paged_attention(q, c.cache, c.t_table, n, row_starts=torch.zeros_like(n), prefix_lens=torch.zeros_like(n), **kw)
    assert torch.equal(plain[0], same[0]) and torch.equal(plain[1], same[1])


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
def test_bad_rows_and_pages(packed):
    c = Case(4, [100], dtype="bf16", bs=32)
    q, q64 = c.queries(6, 4)
    n = _lens([50, 50, 50, 50, 50, 100])
    start, prefix = _lens([-1, 0, 101, 0, 3, 0]), _lens([0, 101, 0, -1, 60, 0])
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=100, row_to_batch=_lens([0] * 6), packed=packed,
                                   want_lse=True, row_starts=start, prefix_lens=prefix, softcap=9.0)
    empty = np.arange(0)
    _check(c, q64, [(0, 50, empty)] * 4 + [(0, 50, np.arange(3, 60)), (0, 100, np.arange(100))], out, lse, 128 ** -0.5, softcap=9.0)
    assert sai.device_status() == 1
    table = c.t_table.clone()
    table[0, 1] = 1 << 20
    seen = np.concatenate([np.arange(32), np.arange(64, 100)])
    out, lse = sai.paged_attention(q[:1], c.cache, table, _lens([100]), max_seq_len=100, row_to_batch=_lens([0]), packed=packed,
                                   want_lse=True, softcap=9.0, slopes=_slopes(4))
    _check(c, q64[:1], [(0, 100, seen)], out, lse, 128 ** -0.5, softcap=9.0, slopes=_slopes(4))
    assert sai.device_status() == 4
    # a prefix past the table's columns
    out, lse = sai.paged_attention(q[:1], c.cache, c.t_table, _lens([50]), max_seq_len=1000, row_to_batch=_lens([0]), packed=packed,
                                   want_lse=True, prefix_lens=_lens([500]))
    assert torch.isinf(lse).all() and sai.device_status() == 1


def test_refusals():
    c = Case(5, [100], dtype="bf16", bs=32)
    q, _ = c.queries(1, 4)
    call = lambda **kw: sai.paged_attention(q, c.cache, c.t_table, _lens([100]), max_seq_len=100, **kw)
    for cap in (-1.0, float("nan"), float("inf"), 1e-40, 1e31):
        with pytest.raises(ValueError, match="softcap"):
            call(softcap=cap)
        with pytest.raises(ValueError, match="softcap"):
            sai.sparse_attention(q, c.cache, _lens([[0]]), softcap=cap)
    with pytest.raises(TypeError):
        call(softcap="x")
    with pytest.raises(ValueError, match="slopes"):
        call(slopes=torch.zeros(5, device=DEV))
    with pytest.raises(ValueError, match="slopes"):
        call(slopes=torch.zeros(4, device=DEV, dtype=torch.float64))
    with pytest.raises(ValueError, match="slopes"):
        call(slopes=torch.zeros(8, device=DEV)[::2])
    with pytest.raises(ValueError, match="row_starts"):
        call(row_starts=_lens([0, 0]))
    with pytest.raises(ValueError, match="prefix_lens"):
        call(prefix_lens=_lens([0]).long())
    assert sai.device_status() == 0

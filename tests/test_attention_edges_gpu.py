"""Paged and sparse attention at the edges of what a cache and its queries may hold, against the float64 oracle.

Element bounds are those of test_attention_gpu.py; where a test needs another term, it derives it.
"""

import numpy as np
import pytest
import torch
from test_attention_gpu import Case, _check, _lens

import sparse_attention_indexer_top_gb300 as sai
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _rows(reqs):
    """Lengths and requests of packed rows; reqs: (new rows, total length) of each request."""
    return [t - n + j + 1 for n, t in reqs for j in range(n)], [b for b, (n, _) in enumerate(reqs) for _ in range(n)]


def _check_any(case, q64, cells, out, lse, sm, lse_extra=0.0):
    """_check for values that may be NaN or infinite: the same elements are, the others are within the bounds."""
    out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for i, (b, at) in enumerate(cells):
        if not len(at):
            assert (out[i] == 0).all() and np.isneginf(lse[i]).all(), i
            continue
        k, v = (x[at] for x in case.kv[b])
        with np.errstate(invalid="ignore"):
            ref, rl, mag = A.attend(q64[i], k, v, sm)
        ok = np.isfinite(ref)
        assert np.array_equal(out[i][~ok], ref[~ok], equal_nan=True), (i, out[i][~ok], ref[~ok])
        grp = q64.shape[1] // case.hkv
        size = np.array([np.abs(k[:, a // grp]).dot(np.abs(q64[i, a])).max() for a in range(q64.shape[1])]) * abs(sm)
        d = (case.dim + 8) * 2.0 ** -23 * size[:, None]
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 4 * d) * mag
        assert (np.abs(out[i][ok] - ref[ok]) <= tol[ok]).all(), i
        assert (np.abs(lse[i] - rl) <= 2 * d[:, 0] + 2.0 ** -19 * (1 + np.abs(rl)) + lse_extra).all(), i


# --- value rows that are not finite

def _spoil(c, marks):
    """Sets value elements (request, token, dim) of all kv heads."""
    for b, t, d, x in marks:
        blk = int(c.table[b, t // c.bs])
        if c.dtype == "bf16":
            c.v[blk, :, t % c.bs, d] = x
        else:
            c.v.view(torch.uint8)[blk, :, t % c.bs, d] = 0x7F
        c.kv[b][1][t, :, d] = x if c.dtype == "bf16" else np.nan


NAN, INF = float("nan"), float("inf")
SPOILED = [
    # several requests in one unit of tiles, each with such a token, in the same and in different halves of the dims
    ([(64, 64), (64, 64)], [(0, 10, 3, NAN), (1, 20, 5, NAN)]),
    ([(64, 64), (64, 64)], [(0, 10, 63, INF), (1, 20, 1, NAN), (1, 21, 40, -INF)]),
    ([(20, 20), (20, 40), (20, 60), (30, 50)], [(0, 0, 2, NAN), (1, 25, 3, INF), (2, 55, 4, -INF), (3, 49, 5, NAN)]),
    ([(40, 500), (1, 130), (60, 130)], [(0, 470, 7, INF), (0, 480, 7, -INF), (0, 100, 9, NAN), (2, 100, 9, NAN)]),
    # units that are dealt out and joined
    ([(40, 6000), (24, 5000)], [(0, 5980, 3, NAN), (0, 100, 6, INF), (1, 4985, 3, NAN), (1, 4990, 60, INF)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,group,bs", [(128, 4, 128), (64, 8, 32), (128, 8, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (45, 12)])
@pytest.mark.parametrize("reqs,marks", SPOILED)
def test_seen_nonfinite_values(dtype, dim, group, bs, window, sinks, reqs, marks):
    """Rows that see such a value have it in its dim (and only there), the others are as if it were not there."""
    c = Case(200 + dim + group, [t for _, t in reqs], dtype=dtype, hkv=1, dim=dim, bs=bs)
    # and in the upper half of the dims
    _spoil(c, marks + [(b, t, d + dim // 2, x) for b, t, d, x in marks if d + dim // 2 < dim])
    lens, r2b = _rows(reqs)
    q, q64 = c.queries(len(lens), group)
    cells = [(b, A.seen(n, window, sinks)) for b, n in zip(r2b, lens)]
    for packed in (sai.PACKED_TILES, False):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=max(lens), window=window,
                                       sinks=sinks, row_to_batch=_lens(r2b), packed=packed, want_lse=True)
        _check_any(c, q64, cells, out, lse, dim ** -0.5)


# --- block scales of 0

@pytest.mark.parametrize("packed", [False, True, 2])
@pytest.mark.parametrize("dim,group,bs", [(128, 4, 16), (64, 8, 128), (128, 20, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 9)])
@pytest.mark.parametrize("share", [0.5, 1.0])
def test_zero_scales(packed, dim, group, bs, window, sinks, share):
    """Blocks with a scale of 0 hold zeros. A log-sum-exp may be off by the spacing of the running maximum, which
    carries the value scale's exponent (at most 64 and a few): three roundings of numbers below 128, 3 * 2^-18."""
    reqs = [(90, 400), (1, 150), (64, 64)]
    c = Case(210 + dim, [t for _, t in reqs], dtype="e4m3", hkv=2, dim=dim, bs=bs)
    for x, which in ((c.ks, 0), (c.vs, 1)):
        zero = torch.from_numpy(c.rng.random(tuple(x.shape)) < share).to(DEV)
        x.masked_fill_(zero, 0.0)
        for b, (_, t) in enumerate(reqs):
            for j in range(0, t, bs):
                c.kv[b][which][j:j + bs, zero[int(c.table[b, j // bs])].cpu().numpy()] = 0.0
    lens, r2b = _rows(reqs)
    lens[3] = lens[100] = 0
    q, q64 = c.queries(len(lens), 2 * group)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=400, row_to_batch=_lens(r2b),
                                   packed=packed, window=window, sinks=sinks, want_lse=True)
    _check_any(c, q64, [(b, A.seen(n, window, sinks)) for b, n in zip(r2b, lens)], out, lse, dim ** -0.5, 3 * 2.0 ** -18)

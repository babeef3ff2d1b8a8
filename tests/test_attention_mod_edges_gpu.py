"""GPU tests of the attention with changed scores and masks where it went wrong or slow: infinite values, large scales,
first tokens of several documents, long prefixes under short windows, rows that see nothing, the cap's own error.

Bounds of time compare two calls on the same machine with about the same keys to read; they are far above what the calls
differ by and far below what they differed by while the second one walked keys that no row sees, or walked them alone.
"""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import attention as A
from test_attention_gpu import DEV, Case, _lens
from test_attention_mod_gpu import _check, _slopes
from timing import least_us

pytestmark = pytest.mark.gpu


def _infinite(c, n, dim):
    """Value cell (t, t % dim) becomes infinite, even t up, odd t down: every dim meets one infinity at least, of one sign
    (dim is even), with a weight of its own."""
    for t in range(n):
        inf = float("inf") if t % 2 == 0 else -float("inf")
        c.v[int(c.table[0, t // c.bs]), :, t % c.bs, t % dim] = inf


def _all_infinite(out, dim):
    sign = torch.where(torch.arange(dim, device=DEV) % 2 == 0, float("inf"), -float("inf"))
    return bool((out.float() == sign).all())


INF_MODS = [dict(), dict(softcap=30.0), dict(softcap=5.0, slopes=0.02), dict(slopes=0.02)]


@pytest.mark.parametrize("mod", INF_MODS)
@pytest.mark.parametrize("group,dim", [(1, 128), (8, 64), (12, 128), (17, 64), (70, 128)])
@pytest.mark.parametrize("packed", [0, 1, sai.PACKED_TILES])
def test_visible_infinite_values_stay_infinite(mod, group, dim, packed):
    """A sum of positive weights times values with infinities of one sign is infinite, the key of the largest weight among
    them; scores lie within 60 of one another, so no weight is 0."""
    n = 2 * dim
    c = Case(20 + dim + group, [n], dtype="bf16", hkv=1, dim=dim, bs=64)
    _infinite(c, n, dim)
    q, _ = c.queries(3, group, sigma=1.0)
    kw = dict(mod)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"] * _slopes(group)
    out = sai.paged_attention(q, c.cache, c.t_table, _lens([n, n - 1, n]), max_seq_len=n, row_to_batch=_lens([0, 0, 0]),
                              packed=packed, **kw)
    assert _all_infinite(out, dim)


@pytest.mark.parametrize("cap", [0.0, 4.0])
@pytest.mark.parametrize("group", [4, 16, 64])
def test_sparse_infinite_values_stay_infinite(cap, group):
    c = Case(30 + group, [256], dtype="bf16", hkv=1, bs=64)
    _infinite(c, 256, 128)
    q, _ = c.queries(2, group, sigma=1.0)
    slots = torch.tensor([[c.slot(0, t) for t in range(256)], [c.slot(0, t) for t in range(128)] + [-1] * 128],
                         dtype=torch.int32, device=DEV)
    assert _all_infinite(sai.sparse_attention(q, c.cache, slots, softcap=cap), 128)


@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
def test_an_infinite_value_reaches_its_dim_alone(packed):
    """One infinity on a row that is split over chunks, and another row that does not see it."""
    c = Case(40, [3000], dtype="bf16", hkv=2, bs=128)
    q, q64 = c.queries(2, 8, sigma=1.0)
    at = 2500
    c.v[int(c.table[0, at // 128]), :, at % 128, 9] = float("inf")
    slopes = 0.001 * _slopes(8)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([3000, 2400]), max_seq_len=3000, row_to_batch=_lens([0, 0]),
                                   packed=packed, want_lse=True, softcap=20.0, slopes=slopes)
    assert (out[0, :, 9] == float("inf")).all() and torch.isfinite(out[1]).all()
    out[0, :, 9] = 0.0
    c.kv[0][1][at, :, 9] = 0.0
    for i, n in enumerate((3000, 2400)):
        k, v = (x[:n] for x in c.kv[0])
        ref, _, mag = A.attend_changed(q64[i], k, v, 128 ** -0.5, 20.0, slopes.double().cpu().numpy(), np.arange(n)[::-1])
        if i == 0:
            ref[:, 9] = mag[:, 9] = 0.0
        assert (np.abs(out[i].float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag).all(), i


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("sm,cap", [(1e20, 1e15), (1e30, 1e26), (2.0 ** 60, 2.0 ** 50), (1e-25, 1e-29)])
def test_large_and_small_scales_under_a_cap(dtype, packed, slopes, sm, cap):
    """Scores of 0 at any sm_scale: the weights are even (biased: those of the distances alone)."""
    n = 300
    c = Case(41, [n], dtype=dtype, bs=16, hkv=1)
    q = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device=DEV)
    sl = _slopes(2) if slopes else None
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([n, 200]), max_seq_len=n, row_to_batch=_lens([0, 0]),
                                   packed=packed, want_lse=True, softcap=cap, sm_scale=sm, slopes=sl)
    for i, m in enumerate((n, 200)):
        w = np.exp(-(sl.double().cpu().numpy() if slopes else np.zeros(2))[:, None] * np.arange(m)[::-1])
        ref = w @ c.kv[0][1][:m, 0] / w.sum(1, keepdims=True)
        mag = w @ np.abs(c.kv[0][1][:m, 0]) / w.sum(1, keepdims=True)
        # weights in 16 bits (2^-8 of each at most) and the result's own rounding
        assert (np.abs(out[i].float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag).all(), i
        # distances' products 2^-22 of at most 150, exponentials and sums 2^-20
        assert np.abs(lse[i].cpu().numpy() - np.log(w.sum(1))).max() <= 2.0 ** -14, i


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("packed", [0, sai.PACKED_TILES])
@pytest.mark.parametrize("near", [0.01, 0.2, 0.25, 0.5, 1.0, 2.0, 9.0])
def test_the_cap_alone(dtype, packed, near):
    """256 equal keys with exact products, so that the log-sum-exp is the capped score plus log 256, on both sides of where
    the polynomials change.

    The score may be off by 2^-20 of itself (of the cap, 2^-22, beyond it). The rest is the way through log2 units: scale,
    cap, its inverse, the product, the sum with the logarithm and ln 2 are a rounding each, of at most the log-sum-exp and
    log 256, doubled: 16 * 2^-24."""
    n, cap = 256, 30.0
    c = Case(42, [n], dtype=dtype, bs=128, hkv=1, dim=64)
    blocks = [int(x) for x in c.table[0]]
    one = torch.zeros(64)
    one[:2] = 1.0
    c.k[blocks] = one.to(c.k.dtype).to(DEV)
    if dtype == "e4m3":
        c.ks[blocks] = 1.0
    at = [near * cap * f for f in (0.97, 0.996, 1.0, 1.004, 1.03)]
    q = torch.zeros((len(at) * 2, 1, 64))
    for i, x in enumerate(at):
        hi = torch.tensor(x).bfloat16().float()
        q[2 * i, 0, 0], q[2 * i, 0, 1] = hi, torch.tensor(x - float(hi)).bfloat16().float()
        q[2 * i + 1] = -q[2 * i]
    q = q.to(torch.bfloat16).to(DEV)
    x = q.double().sum(-1).cpu().numpy()[:, 0]
    rows = len(x)
    _, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([n] * rows), max_seq_len=n, row_to_batch=_lens([0] * rows),
                                 packed=packed, want_lse=True, softcap=cap, sm_scale=1.0)
    ref = cap * np.tanh(x / cap) + np.log(n)
    tol = np.where(np.abs(x) <= cap, 2.0 ** -20 * np.abs(x), 2.0 ** -22 * cap) + 2.0 ** -20 * (np.abs(ref) + 2 * np.log(n))
    err = np.abs(lse.cpu().double().numpy()[:, 0] - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", ["two requests", "two documents"])
def test_first_tokens_of_one_document_cost_no_other(dtype, rows):
    """Rows of a window with first tokens: tiles between one row's first tokens and another's are not walked."""
    c = Case(43, [30000, 200], dtype=dtype, bs=128, hkv=1)
    if rows == "two requests":  # a late document of one, a short other one
        spans = [(0, n, 29000) for n in range(29985, 30001)] + [(1, n, 0) for n in range(185, 201)]
    else:
        spans = [(0, n, 0) for n in range(28985, 29001)] + [(0, n, 29000) for n in range(29140, 29156)]
    b, n, start = (_lens(list(x)) for x in zip(*spans))
    q, q64 = c.queries(len(spans), 8)
    kw = dict(max_seq_len=30000, row_to_batch=b, packed=sai.PACKED_TILES, window=128, sinks=4)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, want_lse=True, row_starts=start, **kw)
    _check(c, q64, [(b, n, A.span(n, 128, 4, s)) for b, n, s in spans], out, lse, 128 ** -0.5)
    plain = least_us(lambda: sai.paged_attention(q, c.cache, c.t_table, n, **kw))
    masked = least_us(lambda: sai.paged_attention(q, c.cache, c.t_table, n, row_starts=start, **kw))
    assert masked < 3 * plain, (masked, plain)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("packed", [0, 1])
def test_a_long_prefix_under_a_short_window_is_split(dtype, packed):
    """The row sees the keys from its window's first one to the prefix's end, far more than the window."""
    c = Case(44, [30000], dtype=dtype, bs=128, hkv=1)
    q, q64 = c.queries(1, 8)
    n, prefix = _lens([200]), _lens([30000])
    kw = dict(max_seq_len=30000, row_to_batch=_lens([0]), packed=packed, prefix_lens=prefix)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, want_lse=True, window=128, **kw)
    _check(c, q64, [(0, 200, A.span(200, 128, 0, 0, 30000))], out, lse, 128 ** -0.5)
    whole = least_us(lambda: sai.paged_attention(q, c.cache, c.t_table, n, **kw))
    windowed = least_us(lambda: sai.paged_attention(q, c.cache, c.t_table, n, window=128, **kw))
    assert windowed < 2 * whole, (windowed, whole)


def test_workspaces_of_a_long_prefix():
    """The plain call's workspace for its window is enough; that without a window lets the row be split."""
    c = Case(45, [5000], dtype="bf16", bs=128, hkv=1)
    q, q64 = c.queries(2, 8)
    n, prefix = _lens([100, 4000]), _lens([5000, 0])
    cells = [(0, 100, A.span(100, 64, 0, 0, 5000)), (0, 4000, A.span(4000, 64))]
    for window in (64, 0):
        need = sai.paged_attention_workspace(2, 8, c.cache, max_seq_len=5000, window=window)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=5000, row_to_batch=_lens([0, 0]), window=64,
                                       want_lse=True, prefix_lens=prefix, workspace=ws)
        _check(c, q64, cells, out, lse, 128 ** -0.5)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("mod", ["cap", "bias", "both"])
@pytest.mark.parametrize("empty", ["lengths", "starts"])
def test_rows_that_see_nothing_slow_no_others(dtype, mod, empty):
    """Padding, or documents that start behind their rows, among packed rows with changed scores: NaN queries too."""
    total, rows = 32768, 1024
    c = Case(46, [total], dtype=dtype, bs=128, hkv=1)
    q, q64 = c.queries(rows, 8)
    none = [i for i in range(rows) if i % 50 == 3]
    full = list(range(total - rows + 1, total + 1))
    lens = [0 if i in none and empty == "lengths" else n for i, n in enumerate(full)]
    kw = dict(max_seq_len=total, row_to_batch=_lens([0] * rows), packed=sai.PACKED_TILES, softcap=0.0 if mod == "bias" else 50.0,
              slopes=None if mod == "cap" else 0.01 * _slopes(8))
    starts = _lens([0] * rows)
    n = _lens(full)
    whole = least_us(lambda: sai.paged_attention(q, c.cache, c.t_table, n, row_starts=starts, **kw))
    if empty == "starts":
        starts[none] = total
    n = _lens(lens)
    holes = least_us(lambda: sai.paged_attention(q, c.cache, c.t_table, n, row_starts=starts, **kw))
    assert holes < 1.25 * whole, (holes, whole)
    q[none[0]] = float("nan")
    q[none[1]] = float("inf")
    out, lse = sai.paged_attention(q, c.cache, c.t_table, n, want_lse=True, row_starts=starts, **kw)
    few = [0, 2, 4, 200, rows - 1]
    _check(c, q64[few], [(0, full[i], A.span(full[i])) for i in few], out[few], lse[few], 128 ** -0.5, softcap=kw["softcap"],
           slopes=kw["slopes"])
    assert (out[none] == 0).all() and (lse[none] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("mod", ["masks", "bias", "cap"])
@pytest.mark.parametrize("dim,hkv,group", [(128, 1, 4), (64, 1, 4)])
def test_each_change_alone_on_long_rows(dtype, mod, dim, hkv, group):
    """Few rows, long enough that their tiles are dealt out and joined, for each instance of the tile kernel."""
    total, rows = 9000, 6
    c = Case(47, [total], dtype=dtype, bs=64, hkv=hkv, dim=dim)
    q, q64 = c.queries(rows, group, sigma=3.0)
    n = list(range(total - rows + 1, total + 1))
    start, prefix = [0, 4000, 8990, 17, 9000, 1], [0, 0, 9000, 8999, 0, 0]
    kw, plain = {}, dict(softcap=0.0, slopes=None)
    if mod == "masks":
        kw = dict(row_starts=_lens(start), prefix_lens=_lens(prefix))
    else:
        start = prefix = [0] * rows
        kw = dict(slopes=0.01 * _slopes(group)) if mod == "bias" else dict(softcap=20.0)
        plain.update(kw)
    for w, s in ((0, 0), (3001, 200)):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(n), max_seq_len=total, row_to_batch=_lens([0] * rows),
                                       packed=sai.PACKED_TILES, want_lse=True, window=w, sinks=s, **kw)
        _check(c, q64, [(0, m, A.span(m, w, s, a, p)) for m, a, p in zip(n, start, prefix)], out, lse, dim ** -0.5, **plain)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,hkv,group,bs", [(64, 2, 1, 16), (64, 1, 33, 128), (128, 1, 64, 64), (128, 2, 5, 16)])
@pytest.mark.parametrize("window,sinks", [(130, 70), (3, 300)])
def test_masks_with_windows_of_other_heads(dtype, dim, hkv, group, bs, window, sinks):
    from test_attention_mod_gpu import _spans

    totals = [700, 2, 333]
    c = Case(48 + group, totals, dtype=dtype, bs=bs, hkv=hkv, dim=dim)
    spans = _spans(window + group, totals, 40)
    q, q64 = c.queries(len(spans), hkv * group)
    b, n, start, prefix = (_lens(list(x)) for x in zip(*spans))
    cells = [(b, n, A.span(n, window, sinks, s, p)) for b, n, s, p in spans]
    for packed in (0, sai.PACKED_TILES):
        for mod in (dict(), dict(softcap=10.0), dict(slopes=_slopes(hkv * group))):
            out, lse = sai.paged_attention(q, c.cache, c.t_table, n, max_seq_len=700, row_to_batch=b, packed=packed,
                                           window=window, sinks=sinks, want_lse=True, row_starts=start, prefix_lens=prefix, **mod)
            _check(c, q64, cells, out, lse, dim ** -0.5, **mod)
    assert sai.device_status() == 0

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


# --- small weights beside blocks with large scales

@pytest.mark.parametrize("rows,packed", [(1, False), (2500, False), (200, 2)])
@pytest.mark.parametrize("group", [4, 16, 20])
def test_small_weights_beside_a_large_scale(rows, packed, group):
    """Two kinds of runs in turn (128 tokens for tiles, 64 for single rows' warps): a key of weight 1 in a block of value scale 2^10 whose codes are 0 but in dim
    0, and keys of weights about 2^-16 with value scale 1, which alone fill the other dims.

    The weights of an e4m3 cache go to f16 below a maximum of score plus scale exponent, at least 2^6 there: each is
    off by at most 2^-25 * 2^-6 of 2^(16 + 10) beside its relative 2^-12. With sum e_t the softmax's denominator, that
    is 2^-31 * 2^26 * sum |v_t| / sum e_t for an element, and the bounds' own terms.
    """
    n, dim = 2048, 128
    c = Case(220, [n], dtype="e4m3", hkv=1, dim=dim, bs=16)
    kind = (np.arange(n) // (128 if packed else 64)) % 2  # 0: large scale
    kc, vc = np.zeros((n, dim)), np.zeros((n, dim))
    kc[:, 0] = np.where(kind == 0, np.where(np.arange(n) % 16 == 0, 16.0, -240.0), c.rng.choice([0.0, 0.25, -0.5, 0.75], n))
    vc[kind == 1] = np.exp2(c.rng.integers(-2, 6, (n // 2, dim)))
    vc[kind == 0, 0] = 1.0
    ks, vs = np.ones(n), np.where(kind == 0, 2.0 ** 10, 1.0)
    for x, codes, s, scale in ((c.k, kc, c.ks, ks), (c.v, vc, c.vs, vs)):
        t = torch.from_numpy(codes).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV).view(-1, 16, dim)
        blk = torch.from_numpy(c.table[0]).long().to(DEV)
        x.view(torch.uint8)[blk, 0] = t
        s[blk, 0] = torch.from_numpy(scale[::16]).float().to(DEV)
    q = torch.zeros((rows, group, dim), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    sm = float(np.log(2.0))
    ref, rl, mag = A.attend(q[0].double().cpu().numpy(), kc[:, None], (vc * vs[:, None])[:, None], sm)
    total = np.exp2(kc[:, 0]).sum()
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([n] * rows), max_seq_len=n, row_to_batch=_lens([0] * rows),
                                   packed=packed, sm_scale=sm, want_lse=True)
    tol = 2.0 ** -8 * ref + 2.0 ** -8 * mag + 2.0 ** -5 * (vc * vs[:, None]).sum(0) / total * (np.arange(dim) > 0)
    assert (tol[:, 1:] < 0.5 * ref[:, 1:]).all()  # zeros there would be found out
    err = np.abs(out.double().cpu().numpy() - ref[None])
    assert (err <= tol[None]).all()
    assert (np.abs(lse.double().cpu().numpy() - rl[None]) <= 2.0 ** -15).all()


# --- queries of any size

@pytest.mark.parametrize("packed", [False, 2])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [4, 16, 20])
@pytest.mark.parametrize("power", [-120, -95, 95, 112, 120])
def test_query_sizes(packed, dtype, group, power):
    """Queries times 2^power with sm_scale over it: the same scores."""
    reqs = [(70, 300), (20, 20)]
    c = Case(230, [t for _, t in reqs], dtype=dtype, hkv=1, bs=64)
    lens, r2b = _rows(reqs)
    q, _ = c.queries(len(lens), group)
    scaled = q * 2.0 ** power
    q64 = scaled.double().cpu().numpy() * 2.0 ** -power  # the least ones have lost bits
    out, lse = sai.paged_attention(scaled, c.cache, c.t_table, _lens(lens), max_seq_len=300,
                                   row_to_batch=_lens(r2b), packed=packed, sm_scale=2.0 ** -power * 128 ** -0.5,
                                   want_lse=True)
    _check(c, q64, [(b, np.arange(n)) for b, n in zip(r2b, lens)], out, lse, 128 ** -0.5)


@pytest.mark.parametrize("packed", [False, 2])
@pytest.mark.parametrize("group", [4, 20])
def test_tiny_queries_and_key_scales(packed, group):
    """Scores that are 0 in fp32: every seen key has the same weight."""
    n = 200
    c = Case(231, [n], dtype="e4m3", hkv=1, bs=32)
    c.ks.fill_(2.0 ** -64)
    q, _ = c.queries(n, group)
    out, lse = sai.paged_attention(q * 2.0 ** -90, c.cache, c.t_table, _lens(range(1, n + 1)), max_seq_len=n,
                                   row_to_batch=_lens([0] * n), packed=packed, want_lse=True)
    _check(c, np.zeros((n, group, 128)), [(0, np.arange(i + 1)) for i in range(n)], out, lse, 1.0)


@pytest.mark.parametrize("packed", [False, 2])
@pytest.mark.parametrize("group", [4, 20])
@pytest.mark.parametrize("scales", [(105, 119), (-70, -60), (-62, 36)])
def test_value_scales_of_any_size(packed, group, scales):
    """Up to what append_kv makes of the largest bf16 values. A log-sum-exp may be off by the spacing of the running
    maximum, which carries the value scale's exponent: three roundings of numbers below 128, 3 * 2^-18."""
    reqs = [(70, 300), (20, 20)]
    c = Case(232, [t for _, t in reqs], dtype="e4m3", hkv=1, bs=32, vscales=scales)
    lens, r2b = _rows(reqs)
    q, q64 = c.queries(len(lens), group)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=300, row_to_batch=_lens(r2b),
                                   packed=packed, want_lse=True)
    _check_any(c, q64, [(b, np.arange(n)) for b, n in zip(r2b, lens)], out, lse, 128 ** -0.5, 3 * 2.0 ** -18)


# --- rows all of whose scores are -inf

@pytest.mark.parametrize("packed", [False, 2])
@pytest.mark.parametrize("group,n", [(4, 40), (16, 300), (20, 40), (4, 9000)])
def test_all_scores_minus_infinity(packed, group, n):
    """A row whose sum is 0 gives zeros and -inf, whatever its values are."""
    c = Case(240, [n], dtype="bf16", hkv=1, bs=64)
    q, _ = c.queries(30, group)
    q[:, :, 0] = 1.0
    c.k[:, :, :, 0] = -INF
    c.k[:, :, :, 1:] = 0.0
    _spoil(c, [(0, 5, 3, NAN), (0, n - 35, 70, INF)])
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(range(n - 29, n + 1)), max_seq_len=n,
                                   row_to_batch=_lens([0] * 30), packed=packed, want_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


# --- block tables that are slices of wider ones

@pytest.mark.parametrize("packed", [False, 2])
def test_sliced_block_table(packed):
    """Columns of a wide table, as index_score_topk takes them; what lies beside the slice is never used."""
    reqs = [(70, 300), (20, 20), (1, 256)]
    c = Case(250, [t for _, t in reqs], dtype="bf16", bs=64)
    lens, r2b = _rows(reqs)
    q, q64 = c.queries(len(lens), 8)
    rows, cols = c.table.shape
    wide = torch.zeros((rows, cols + 7), dtype=torch.int32, device=DEV)
    wide[:, 3:3 + cols] = c.t_table
    part = wide[:, 3:3 + cols]
    cells = [(b, np.arange(n)) for b, n in zip(r2b, lens)]
    kw = dict(max_seq_len=1000, row_to_batch=_lens(r2b), packed=packed, want_lse=True)
    sai.device_status()
    out, lse = sai.paged_attention(q, c.cache, part, _lens(lens), **kw)
    _check(c, q64, cells, out, lse, 128 ** -0.5)
    assert sai.device_status() == 0
    # a length that passes the slice, but not the wide table: a bad row
    lens[0] = cols * 64 + 1
    out, lse = sai.paged_attention(q, c.cache, part, _lens(lens), **kw)
    _check(c, q64, [(0, np.arange(0))] + cells[1:], out, lse, 128 ** -0.5)
    assert sai.device_status() == 1
    # one request: the stride of an axis of one means nothing
    sai.paged_attention(q[:1], c.cache, wide[:1, 3:3 + cols], _lens([300]), **dict(kw, row_to_batch=_lens([0])))
    assert sai.device_status() == 0
    for bad in (c.t_table.t().contiguous().t(), c.t_table[:1].expand(rows, cols)):
        with pytest.raises(ValueError, match="block_table"):
            sai.paged_attention(q, c.cache, bad, _lens(lens), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rot", [0, 64])
def test_append_through_a_sliced_block_table(dtype, rot):
    lens = [64, 33, 1]
    a, b = (Case(251, [64, 33, 1], dtype=dtype, dim=64, bs=32) for _ in range(2))
    rows, cols = a.table.shape
    wide = torch.zeros((rows, cols + 5), dtype=torch.int32, device=DEV)
    wide[:, 2:2 + cols] = a.t_table
    k, v = (torch.randn((rows, 2, 64), device=DEV).to(torch.bfloat16) for _ in range(2))
    cs = torch.rand((500, rot), device=DEV) if rot else None
    bits = lambda c: [x.contiguous().view(torch.uint8).clone() for x in (c.k, c.v)]
    sai.device_status()
    sai.append_kv(a.cache, k, v, a.t_table, _lens(lens), cs)
    sai.append_kv(b.cache, k, v, wide[:, 2:2 + cols], _lens(lens), cs)
    assert sai.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(bits(a), bits(b)))
    # past the slice, but not past the wide table: skipped and flagged
    before = bits(b)
    sai.append_kv(b.cache, k, v, wide[:, 2:2 + cols], _lens([cols * 32 + 1, 0, 0]), cs)
    assert sai.device_status() == 1
    assert all(torch.equal(x, y) for x, y in zip(before, bits(b)))


def test_append_with_angles_of_no_dims():
    """They bound no position."""
    c = Case(252, [33], dtype="bf16", dim=64, bs=32)
    x = torch.randn((1, 2, 64), device=DEV).to(torch.bfloat16)
    sai.device_status()
    sai.append_kv(c.cache, x, x, c.t_table, _lens([33]), torch.empty((2, 0), device=DEV))
    assert sai.device_status() == 0
    assert torch.equal(c.k[int(c.table[0, 1]), :, 0], x[0])



@pytest.mark.parametrize("packed", [False, 2])
@pytest.mark.parametrize("window", [0, 1000])
def test_lengths_near_2_to_31(packed, window):
    """A table of 2^24 blocks to a request: lengths whose rounded ends would pass 32 bits are bad rows, the others right."""
    c = Case(253, [300], dtype="bf16", hkv=1, bs=128)
    table = torch.full((1, 1 << 24), int(c.table[0, 0]), dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.t_table
    top = 2 ** 31 - 1
    lens = [300, top, top - 100, 2 ** 31 - 8191, 17]
    q, q64 = c.queries(len(lens), 8)
    sai.device_status()
    out, lse = sai.paged_attention(q, c.cache, table, _lens(lens), max_seq_len=top, row_to_batch=_lens([0] * 5),
                                   packed=packed, window=window, want_lse=True)
    assert sai.device_status() == 1
    cells = [(0, A.seen(n, window, 0)) if n <= 300 else (0, np.arange(0)) for n in lens]
    _check(c, q64, cells, out, lse, 128 ** -0.5)



# --- arguments without a truth value

def test_flags_without_a_truth_value():
    c = Case(260, [10], dtype="bf16", dim=64, bs=16)
    x = torch.ones((1, 2, 64), dtype=torch.bfloat16, device=DEV)
    before = c.k.view(torch.uint8).clone()
    with pytest.raises(RuntimeError, match="ambiguous"):
        sai.append_kv(c.cache, x, x, c.t_table, _lens([10]), interleaved=torch.ones(2))
    assert torch.equal(before, c.k.view(torch.uint8))
    with pytest.raises(RuntimeError, match="ambiguous"):
        sai.paged_attention(x, c.cache, c.t_table, _lens([10]), max_seq_len=10, want_lse=torch.ones(2))
    with pytest.raises(RuntimeError, match="ambiguous"):
        sai.sparse_attention(x, c.cache, _lens([[0]]), want_lse=torch.ones(2))

"""GPU parity of the paged and the sparse attention against the float64 oracle.

Error bound of an output element, from the kernels' roundings: the result is
rounded to bf16 (2^-9 of it), the softmax weights to bf16 or f16 (2^-9 of
each, so of sum w|v|), scores are fp32 sums of dim exact products (at most
(dim + 8) * 2^-23 of sum |q k| sm_scale, which moves a weight by the same
share), and exp2, the sums and the quotient add a few 2^-22. Doubled:
  |got - ref| <= 2^-8 |ref| + (2^-8 + 4 d) sum w|v|,  |lse - ref| <= 2 d + 2^-19 (1 + |ref|)
with d the largest score error of the row.
"""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _bits(x, dtype):
    return torch.from_numpy(x).to(dtype)


class Case:
    """A paged cache with `total` tokens for each request, NaN in every cell that holds none."""

    def __init__(self, seed, totals, *, dtype, hkv=2, dim=128, bs=128, nhd=False, blocks=None, vscales=(-8, -5),
                 any_scales=False):
        rng = np.random.default_rng(seed)
        self.rng, self.bs, self.hkv, self.dim, self.dtype = rng, bs, hkv, dim, dtype
        per = [max(1, -(-t // bs)) for t in totals]
        used = sum(per)
        nb = blocks or used + 2
        ids = np.sort(rng.choice(nb, used, replace=False)) if nb < 100000 else np.arange(nb - used, nb)
        rng.shuffle(ids)
        self.table = np.full((len(totals), max(per)), -1, np.int32)
        i = 0
        for b, n in enumerate(per):
            self.table[b, :n] = ids[i:i + n]
            i += n
        self.ks = self.vs = None
        shape = (nb, bs, hkv, dim) if nhd else (nb, hkv, bs, dim)
        elem = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
        k, v = (torch.empty(shape, dtype=elem, device=DEV) for _ in range(2))
        if nhd:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        if nb < 100000:
            for x in (k, v):
                x.copy_(torch.full(k.shape, float("nan"), dtype=torch.float32, device=DEV).to(elem))
        if dtype == "e4m3":
            self.ks, self.vs = (torch.exp2(torch.from_numpy(rng.integers(*r, (nb, hkv))).float()).to(DEV)
                                for r in ((-8, -5), vscales))
            if any_scales:
                for x in (self.ks, self.vs):
                    x.mul_(torch.from_numpy(rng.uniform(1, 2, (nb, hkv))).float().to(DEV))
        self.kv = []
        for b, t in enumerate(totals):
            vals = []
            for x, s in ((k, self.ks), (v, self.vs)):
                raw = torch.from_numpy(rng.normal(0, 1 if dtype == "bf16" else 90, (t, hkv, dim))).clamp(-448, 448)
                raw = raw.to(elem)
                val = raw.float().double()
                for j in range(0, t, bs):
                    blk = int(self.table[b, j // bs])
                    m = min(bs, t - j)
                    x[blk, :, :m] = raw[j:j + m].transpose(0, 1).to(DEV)
                    if s is not None:
                        val[j:j + m] *= s[blk].cpu().double()[None, :, None]
                vals.append(val.numpy())
            self.kv.append(vals)
        self.k, self.v = k, v
        self.cache = sai.KVCache(k.view(torch.uint8) if dtype == "e4m3" else k,
                                 v.view(torch.uint8) if dtype == "e4m3" else v, self.ks, self.vs)
        self.t_table = torch.from_numpy(self.table).to(DEV)

    def queries(self, rows, hq, sigma=2.0):
        q = torch.from_numpy(self.rng.normal(0, sigma, (rows, hq, self.dim))).to(torch.bfloat16)
        return q.to(DEV), q.float().double().numpy()

    def slot(self, b, t):
        return int(self.table[b, t // self.bs]) * self.bs + t % self.bs


def _check(case, q64, cells, out, lse, sm):
    """cells: for each row the (request, positions) it sees."""
    out, lse = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for i, (b, at) in enumerate(cells):
        k, v = (x[at] for x in case.kv[b]) if len(at) else (np.zeros((0, case.hkv, case.dim)),) * 2
        ref, rl, mag = A.attend(q64[i], k, v, sm)
        if not len(at):
            assert (out[i] == 0).all() and np.isneginf(lse[i]).all(), i
            continue
        grp = q64.shape[1] // case.hkv
        size = np.array([np.abs(k[:, a // grp]).dot(np.abs(q64[i, a])).max() for a in range(q64.shape[1])]) * abs(sm)
        d = (case.dim + 8) * 2.0 ** -23 * size[:, None]
        err = np.abs(out[i] - ref)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 4 * d) * mag
        assert (err <= tol).all(), (i, float((err / tol).max()))
        assert (np.abs(lse[i] - rl) <= 2 * d[:, 0] + 2.0 ** -19 * (1 + np.abs(rl))).all(), i


def _lens(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hkv,group,bs", [(2, 1, 128), (2, 3, 16), (1, 16, 64), (2, 17, 32), (1, 64, 128), (1, 70, 128)])
def test_decode_rows(dtype, dim, hkv, group, bs):
    c = Case(10 + dim + group, LENS, dtype=dtype, hkv=hkv, dim=dim, bs=bs)
    q, q64 = c.queries(len(LENS), hkv * group)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(LENS), max_seq_len=1000, want_lse=True)
    _check(c, q64, [(b, A.seen(n, 0, 0)) for b, n in enumerate(LENS)], out, lse, dim ** -0.5)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 5), (100, 64), (127, 130), (5000, 3)])
def test_decode_window_and_first_tokens(dtype, window, sinks):
    c = Case(30 + window, LENS, dtype=dtype, bs=32)
    q, q64 = c.queries(len(LENS), 8)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(LENS), max_seq_len=1000, window=window, sinks=sinks,
                                   sm_scale=0.11, want_lse=True)
    _check(c, q64, [(b, A.seen(n, window, sinks)) for b, n in enumerate(LENS)], out, lse, 0.11)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_one_long_row_is_split_and_joined(dtype):
    lens = [20011]
    c = Case(40, lens, dtype=dtype, bs=64)
    q, q64 = c.queries(1, 16, sigma=4.0)
    assert sai.paged_attention_workspace(1, 16, c.cache, max_seq_len=20011) > 0
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=20011, want_lse=True)
    _check(c, q64, [(0, np.arange(20011))], out, lse, 128 ** -0.5)
    # a bound far above the row's length leaves most chunks empty
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens([130]), max_seq_len=20011, want_lse=True)
    _check(c, q64, [(0, np.arange(130))], out, lse, 128 ** -0.5)


def test_block_scales_far_apart():
    # weights times scales pass f16's range on both sides unless the running maximum takes the scales in
    lens = [700, 300]
    c = Case(41, lens, dtype="e4m3", bs=16, vscales=(-40, 30))
    q, q64 = c.queries(2, 8)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=700, want_lse=True)
    _check(c, q64, [(b, np.arange(n)) for b, n in enumerate(lens)], out, lse, 128 ** -0.5)


PACKED = [
    # (new rows, total length) of each request
    [(1, 1)],
    [(130, 130)],
    [(5, 700), (64, 64), (1, 300), (200, 333)],
    [(128, 1000), (3, 3)],
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,hkv,group,bs", [(128, 2, 4, 128), (64, 1, 8, 32), (128, 2, 1, 16), (128, 1, 5, 64),
                                              (64, 2, 16, 128), (128, 1, 64, 128)])
@pytest.mark.parametrize("reqs", PACKED)
def test_packed_rows(dtype, dim, hkv, group, bs, reqs):
    _packed(dtype, dim, hkv, group, bs, reqs, 0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 5), (129, 127), (128, 200), (300, 0), (4000, 9)])
@pytest.mark.parametrize("reqs", PACKED[2:])
def test_packed_window_and_first_tokens(dtype, window, sinks, reqs):
    _packed(dtype, 128, 2, 4, 64, reqs, window, sinks)


def _packed(dtype, dim, hkv, group, bs, reqs, window, sinks):
    c = Case(50 + dim + len(reqs), [t for _, t in reqs], dtype=dtype, hkv=hkv, dim=dim, bs=bs)
    lens = [t - n + j + 1 for n, t in reqs for j in range(n)]
    r2b = [b for b, (n, _) in enumerate(reqs) for _ in range(n)]
    q, q64 = c.queries(len(lens), hkv * group)
    kw = dict(max_seq_len=max(lens), row_to_batch=_lens(r2b), window=window, sinks=sinks, want_lse=True)
    cells = [(b, A.seen(n, window, sinks)) for b, n in zip(r2b, lens)]
    # as tiles, as the sizes have it, and row by row
    for packed in (sai.PACKED_TILES, True, False):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), packed=packed, **kw)
        _check(c, q64, cells, out, lse, dim ** -0.5)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_packed_rows_in_any_order_with_padding_rows(dtype):
    """Rows that are neither sorted nor neighbours by request, some of length 0."""
    totals = [300, 40, 513]
    c = Case(60, totals, dtype=dtype, bs=32)
    r2b = [int(x) for x in c.rng.integers(0, 3, 150)]
    lens = [int(c.rng.integers(0, totals[b] + 1)) if i % 7 else 0 for i, b in enumerate(r2b)]
    q, q64 = c.queries(150, 8)
    for packed in (True, False, sai.PACKED_TILES):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=513, row_to_batch=_lens(r2b),
                                       packed=packed, want_lse=True)
        _check(c, q64, [(b, np.arange(n)) for b, n in zip(r2b, lens)], out, lse, 128 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_unseen_nonfinite_cells_do_not_matter(dtype, bad):
    """A token of NaN (inf) keys and values in the middle of a packed request: rows before it and rows whose window
    has left it behind are as if it were not there; rows that see it give NaN."""
    if dtype == "e4m3" and bad == "inf":
        pytest.skip("e4m3 has no infinity")
    n, at = 300, 150
    c = Case(70, [n], dtype=dtype, bs=64)
    blk = int(c.table[0, at // 64])
    val = torch.tensor(float(bad), device=DEV).to(c.k.dtype)
    if dtype == "e4m3":
        c.k.view(torch.uint8)[blk, :, at % 64] = val.view(torch.uint8)
        c.v.view(torch.uint8)[blk, :, at % 64] = val.view(torch.uint8)
    else:
        c.k[blk, :, at % 64] = val
        c.v[blk, :, at % 64] = val
    lens = list(range(1, n + 1))
    q, q64 = c.queries(n, 8)
    for packed in (True, False, sai.PACKED_TILES):
        for window, sinks in ((0, 0), (30, 4)):
            out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=n,
                                           row_to_batch=_lens([0] * n), packed=packed, window=window, sinks=sinks,
                                           want_lse=True)
            sees = np.array([at in A.seen(m, window, sinks) for m in lens])
            clean = [i for i in range(n) if not sees[i]]
            _check(c, q64[clean], [(0, A.seen(lens[i], window, sinks)) for i in clean], out[clean], lse[clean],
                   128 ** -0.5)
            if bad == "nan":
                assert torch.isnan(out[torch.from_numpy(sees).to(DEV)]).all()


@pytest.mark.parametrize("packed", [False, True, 2])
def test_layouts_strides_and_streams(packed):
    """Tokens before heads in the cache, k and v in one array, queries as a slice of a fused projection, and a call on
    another stream than torch's current one."""
    reqs = [(40, 200), (3, 90)]
    c = Case(80, [t for _, t in reqs], dtype="bf16", bs=32, nhd=True)
    both = torch.empty((2,) + tuple(c.k.shape), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    both[:, 0], both[:, 1] = c.k, c.v
    r2b = [0] * 40 + [1] * 3
    lens = list(range(161, 201)) + [88, 89, 90]
    qkv = torch.randn((43, (8 + 4) * 128), device=DEV).to(torch.bfloat16)
    q = qkv[:, :8 * 128].view(43, 8, 128)
    side = torch.cuda.Stream()
    args = dict(max_seq_len=200, row_to_batch=_lens(r2b), packed=packed, want_lse=True)
    ln = _lens(lens)
    torch.cuda.synchronize()
    for cache in (c.cache, sai.KVCache(both[:, 0], both[:, 1])):
        for stream in (None, side, side.cuda_stream):
            out, lse = sai.paged_attention(q, cache, c.t_table, ln, stream=stream, **args)
            side.synchronize()
            _check(c, q.float().cpu().double().numpy(), [(b, np.arange(n)) for b, n in zip(r2b, lens)], out, lse,
                   128 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_offsets_past_32_bits(dtype):
    """Blocks at the far end of a cache of more than 2^32 elements."""
    lens, hkv = [200, 61], 4
    blocks = (1 << 32) // (hkv * 128 * 128) + 1000
    c = Case(90, lens, dtype=dtype, hkv=hkv, blocks=blocks if blocks >= 100000 else None, bs=128)
    if blocks < 100000:  # 128-token blocks: fewer blocks, so the far ones are chosen by hand
        elem = c.k.dtype
        k, v = (torch.empty((blocks, hkv, 128, 128), dtype=elem, device=DEV) for _ in range(2))
        small = c.k.shape[0]
        for x, y in ((k, c.k), (v, c.v)):
            x.view(torch.uint8)[-small:] = y.view(torch.uint8)
        sc = [None, None]
        if dtype == "e4m3":
            sc = [torch.zeros((blocks, hkv), device=DEV) for _ in range(2)]
            for x, y in zip(sc, (c.ks, c.vs)):
                x[-small:] = y
        cache = sai.KVCache(k, v, *sc)
        table = torch.where(c.t_table >= 0, c.t_table + (blocks - small), -1).to(torch.int32)
    q, q64 = c.queries(2, 8)
    cells = [(b, np.arange(n)) for b, n in enumerate(lens)]
    for packed in (False, True, sai.PACKED_TILES):
        out, lse = sai.paged_attention(q, cache, table, _lens(lens), max_seq_len=200, row_to_batch=_lens([0, 1]),
                                       packed=packed, want_lse=True)
        _check(c, q64, cells, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("packed", [False, True, 2])
def test_bad_rows_are_emptied_and_flagged(packed):
    c = Case(100, [300, 200], dtype="bf16", bs=64)
    q, q64 = c.queries(5, 8)
    lens, r2b = [300, -1, 301, 200, 10], [0, 0, 0, 1, 7]
    sai.device_status()
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=300, row_to_batch=_lens(r2b),
                                   packed=packed, want_lse=True)
    assert sai.device_status() == 1
    none = np.arange(0)
    _check(c, q64, [(0, np.arange(300)), (0, none), (0, none), (1, np.arange(200)), (0, none)], out, lse, 128 ** -0.5)
    # a block id outside the cache: its keys are not seen
    table = c.t_table.clone()
    table[0, 1] = c.k.shape[0]
    out, lse = sai.paged_attention(q[:1], c.cache, table, _lens([300]), max_seq_len=300, row_to_batch=_lens([0]),
                                   packed=packed, want_lse=True)
    assert sai.device_status() == 4
    at = np.arange(300)
    _check(c, q64[:1], [(0, at[(at < 64) | (at >= 128)])], out, lse, 128 ** -0.5)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,hkv,group,k", [(128, 2, 4, 512), (64, 2, 3, 100), (128, 1, 64, 512), (128, 1, 20, 1),
                                             (64, 1, 1, 513), (128, 4, 16, 77)])
def test_sparse_rows(dtype, dim, hkv, group, k):
    rows = 9
    c = Case(110 + k, [700, 90], dtype=dtype, hkv=hkv, dim=dim, bs=32)
    q, q64 = c.queries(rows, hkv * group)
    slots, cells = np.full((rows, k), -1, np.int32), []
    for i in range(rows):
        b = i % 2
        n = [k, 1, 0, k // 2, 16, 17, 15, k, k][i]
        at = c.rng.permutation([700, 90][b])[:min(n, k)]
        where = np.sort(c.rng.permutation(k)[:len(at)]) if i == 3 else np.arange(len(at))  # padding in between
        slots[i, where] = [c.slot(b, int(t)) for t in at]
        cells.append((b, at))
    wide = torch.full((rows, k + 3), 10 ** 9, dtype=torch.int32, device=DEV)
    wide[:, :k] = torch.from_numpy(slots).to(DEV)
    for s in (torch.from_numpy(slots).to(DEV), wide[:, :k]):
        out, lse = sai.sparse_attention(q, c.cache, s, want_lse=True)
        _check(c, q64, cells, out, lse, dim ** -0.5)
    assert sai.device_status() == 0


def test_sparse_many_rows_share_a_request():
    rows, n = 700, 900
    c = Case(120, [n], dtype="bf16", hkv=2, bs=128)
    q, q64 = c.queries(rows, 16)
    at = [c.rng.permutation(n)[:512] for _ in range(rows)]
    slots = np.array([[c.slot(0, int(t)) for t in a] for a in at], np.int32)
    out, lse = sai.sparse_attention(q, c.cache, torch.from_numpy(slots).to(DEV), want_lse=True)
    _check(c, q64, [(0, a) for a in at], out, lse, 128 ** -0.5)


def test_sparse_slot_beyond_the_cache_is_flagged():
    c = Case(121, [100], dtype="bf16", bs=16)
    q, q64 = c.queries(1, 4)
    slots = np.array([[c.slot(0, 3), c.k.shape[0] * 16, c.slot(0, 99), -7]], np.int32)
    sai.device_status()
    out, lse = sai.sparse_attention(q, c.cache, torch.from_numpy(slots).to(DEV), want_lse=True)
    assert sai.device_status() == 4
    _check(c, q64, [(0, np.array([3, 99]))], out, lse, 128 ** -0.5)


def test_calls_in_a_graph_and_without_rows():
    c = Case(130, [600, 40], dtype="bf16", bs=64)
    q, q64 = c.queries(2, 8)
    lens = _lens([600, 40])
    out = torch.empty_like(q)
    lse = torch.empty((2, 8), device=DEV)
    ws = torch.empty(sai.paged_attention_workspace(2, 8, c.cache, max_seq_len=600), dtype=torch.uint8, device=DEV)
    sai.paged_attention(q, c.cache, c.t_table, lens, max_seq_len=600)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sai.paged_attention(q, c.cache, c.t_table, lens, max_seq_len=600, out=out, out_lse=lse, workspace=ws)
    for ns in ([600, 40], [33, 0]):
        lens.copy_(_lens(ns))
        g.replay()
        torch.cuda.synchronize()
        _check(c, q64, [(b, np.arange(n)) for b, n in enumerate(ns)], out, lse, 128 ** -0.5)
    assert sai.paged_attention(q[:0], c.cache, c.t_table, lens[:0], max_seq_len=600).shape == (0, 8, 128)
    slots = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    assert sai.sparse_attention(q[:0], c.cache, slots).shape == (0, 8, 128)


def test_refusals():
    c = Case(140, [64], dtype="bf16", bs=64)
    q, _ = c.queries(1, 8)
    lens = _lens([64])

    def paged(**kw):
        a = dict(q=q, cache=c.cache, block_table=c.t_table, seq_lens=lens, max_seq_len=64)
        a.update(kw)
        return sai.paged_attention(**a)

    with pytest.raises(ValueError, match="bfloat16"):
        paged(q=q.float())
    with pytest.raises(ValueError, match="contiguous heads"):
        paged(q=q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="must be"):
        paged(seq_lens=lens.long())
    with pytest.raises(ValueError, match="packed rows"):
        paged(packed=True)
    with pytest.raises(ValueError, match="out must"):
        paged(out=torch.empty((1, 8, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(sai.SaiError, match="size or count"):
        paged(q=q[:, :7].contiguous())  # 7 query heads on 2 kv heads
    with pytest.raises(sai.SaiError, match="size or count"):
        paged(window=-1)
    with pytest.raises(sai.SaiError, match="size or count"):
        paged(sm_scale=float("nan"))
    with pytest.raises(sai.SaiError, match="workspace"):
        paged(max_seq_len=4096, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="slots"):
        sai.sparse_attention(q, c.cache, lens[None].expand(2, 1))
    with pytest.raises(ValueError, match="k and v must both be"):
        sai.KVCache(c.k.float(), c.v.float())
    with pytest.raises(ValueError, match="only with one"):
        sai.KVCache(c.k, c.v, torch.ones((3, 2), device=DEV), torch.ones((3, 2), device=DEV))
    odd = torch.zeros((4, 2, 24, 128), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sai.SaiError, match="unsupported"):
        paged(cache=sai.KVCache(odd, odd))


DEALT = [
    # long keys and few units: the tile kernel deals its tiles out over the SMs and joins the units that are cut
    [(70, 6000)],
    [(3, 9000), (200, 230), (40, 7001)],
    [(300, 5200)],
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,hkv,group,bs", [(128, 1, 8, 128), (64, 2, 4, 32), (128, 2, 3, 16)])
@pytest.mark.parametrize("reqs", DEALT)
def test_packed_rows_dealt_out(dtype, dim, hkv, group, bs, reqs):
    _packed(dtype, dim, hkv, group, bs, reqs, 0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_packed_rows_dealt_out_by_a_far_bound(dtype):
    """A bound far above the lengths, rows of length 0 and windows: shares without tiles, units without keys."""
    totals = [700, 40]
    c = Case(57, totals, dtype=dtype, bs=32)
    lens = [0] * 30 + list(range(600, 701)) + [0, 40, 0]
    r2b = [0] * 131 + [1] * 3
    q, q64 = c.queries(len(lens), 8)
    for window, sinks in ((0, 0), (200, 9)):
        out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=50000, row_to_batch=_lens(r2b),
                                       packed=sai.PACKED_TILES, window=window, sinks=sinks, want_lse=True)
        _check(c, q64, [(b, A.seen(n, window, sinks)) for b, n in zip(r2b, lens)], out, lse, 128 ** -0.5)
    assert sai.device_status() == 0


@pytest.mark.parametrize("packed", [False, True, 2])
@pytest.mark.parametrize("dim,group,bs", [(128, 4, 16), (64, 8, 128), (128, 20, 64)])
def test_scales_that_are_no_powers_of_two(packed, dim, group, bs):
    reqs = [(90, 400), (1, 150), (64, 64)]
    c = Case(58, [t for _, t in reqs], dtype="e4m3", dim=dim, bs=bs, any_scales=True)
    lens = [t - n + j + 1 for n, t in reqs for j in range(n)]
    r2b = [b for b, (n, _) in enumerate(reqs) for _ in range(n)]
    q, q64 = c.queries(len(lens), 2 * group)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=400, row_to_batch=_lens(r2b),
                                   packed=packed, want_lse=True)
    _check(c, q64, [(b, np.arange(n)) for b, n in zip(r2b, lens)], out, lse, dim ** -0.5)


def test_packed_block_scales_far_apart():
    lens = list(range(201, 301))
    c = Case(59, [300], dtype="e4m3", bs=16, vscales=(-40, 30))
    q, q64 = c.queries(100, 8)
    out, lse = sai.paged_attention(q, c.cache, c.t_table, _lens(lens), max_seq_len=300, row_to_batch=_lens([0] * 100),
                                   packed=sai.PACKED_TILES, want_lse=True)
    _check(c, q64, [(0, np.arange(n)) for n in lens], out, lse, 128 ** -0.5)

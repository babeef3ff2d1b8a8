"""GPU parity of the paged append with rotation against the float64 oracle.

bf16 cells and queries: one rounding of an fp32 rotation, |got - ref| <=
2^-8 |ref| + 2^-22 (|x1| + |x2|). e4m3 cells: half a step of the scaled
format, s * max(2^-4 |x / s|, 2^-10), plus the same fp32 term; scales are
powers of two and equal the oracle's. Cells that the call does not touch
stay bit for bit.
"""

import numpy as np
import pytest
import torch

import sparse_attention_indexer_top_gb300 as sai
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _table(rot, max_pos):
    half = max(rot // 2, 1)
    ang = np.arange(max_pos)[:, None] * (10000.0 ** (-np.arange(half) / half))[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Setup:
    def __init__(self, seed, totals, dtype, hkv, dim, bs, nhd=False):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.hkv, self.dim, self.bs = rng, dtype, hkv, dim, bs
        per = [max(1, -(-t // bs)) for t in totals]
        nb = sum(per) + 2
        ids = rng.permutation(nb)[:sum(per)]
        self.table = np.full((len(totals), max(per)), -1, np.int32)
        i = 0
        for b, n in enumerate(per):
            self.table[b, :n] = ids[i:i + n]
            i += n
        elem = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
        shape = (nb, bs, hkv, dim) if nhd else (nb, hkv, bs, dim)
        make = lambda: (torch.from_numpy(rng.normal(0, 90, shape)).clamp(-448, 448).to(elem)
                        .to(DEV).view(torch.uint8 if dtype == "e4m3" else elem))
        self.k, self.v = make(), make()
        if nhd:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.ks = self.vs = None
        if dtype == "e4m3":
            self.ks, self.vs = (torch.exp2(torch.from_numpy(rng.integers(-8, -3, (nb, hkv))).float()).to(DEV)
                                for _ in range(2))
        self.cache = sai.KVCache(self.k, self.v, self.ks, self.vs)

    def values(self):
        """Code values and scales as float64."""
        f = (lambda x: x.float()) if self.dtype == "bf16" else (lambda x: x.view(torch.float8_e4m3fn).float())
        out = [f(self.k.contiguous()).cpu().double().numpy(), f(self.v.contiguous()).cpu().double().numpy()]
        return out + [None if s is None else s.cpu().double().numpy() for s in (self.ks, self.vs)]

    def bits(self):
        return [x.contiguous().view(torch.uint8).cpu().numpy() for x in (self.k, self.v)]


def _run(s, lens, r2b, *, hq, rot, interleaved, sigma=4.0, with_q=True, fused=False):
    rows = len(lens)
    x = s.rng.normal(0, sigma, (rows, hq + 2 * s.hkv, s.dim)) * np.exp2(s.rng.integers(-2, 5, (rows, 1, 1)))
    t = torch.from_numpy(x).to(torch.bfloat16)
    x = t.float().double().numpy()
    t = t.to(DEV)
    parts = [t[:, :hq], t[:, hq:hq + s.hkv], t[:, hq + s.hkv:]]
    if not fused:
        parts = [p.contiguous() for p in parts]
    q, k, v = parts
    cs = _table(rot, 5000) if rot else None
    before, bits = s.values(), s.bits()
    out = sai.append_kv(s.cache, k, v, _i32(s.table.tolist()), _i32(lens),
                        None if cs is None else torch.from_numpy(cs).to(DEV), q=q if with_q else None,
                        row_to_batch=None if r2b is None else _i32(r2b), interleaved=interleaved)
    torch.cuda.synchronize()
    after, bits_after = s.values(), s.bits()
    places, rk, rq = [], [], []
    for i, n in enumerate(lens):
        b = i if r2b is None else r2b[i]
        places.append((int(s.table[b, (n - 1) // s.bs]), (n - 1) % s.bs) if n else None)
        turn = (lambda y: A.rotate(y, n - 1, cs, interleaved)) if rot and n else (lambda y: y)
        rk.append(turn(x[i, hq:hq + s.hkv]))
        rq.append(turn(x[i, :hq]) if n else np.zeros((hq, s.dim)))
    size = np.abs(x).max()
    if with_q:
        rq = np.stack(rq)
        assert (np.abs(out.float().cpu().double().numpy() - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -21 * size).all()
    else:
        assert out is None
    for j, vals in ((0, np.stack(rk)), (1, x[:, hq + s.hkv:])):
        want, scale = before[j].copy(), None if before[2 + j] is None else before[2 + j].copy()
        A.append(vals, want, scale, places)
        got = after[j]
        if scale is None:
            tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size
            assert (np.abs(got - want) <= tol).all()
        else:
            assert np.array_equal(after[2 + j], scale)
            # both sides are e4m3 values of nearly the same number: at most one step apart, and few are
            step = np.maximum(np.abs(want) * 2.0 ** -3, 2.0 ** -9)
            assert (np.abs(got - want) <= step).all()
            assert np.mean(got != want) < 1e-3
        touched = np.zeros(got.shape[:3], bool)
        for at in places:
            if at is not None:
                touched[at[0], :, at[1]] = True
                if scale is not None:
                    touched[at[0], :, :at[1]] |= (scale[at[0]] != before[2 + j][at[0]])[:, None]
        same = (bits_after[j] == bits[j]).reshape(got.shape + (-1,)).all((-1, -2))
        assert same[~touched].all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,hkv,hq,bs,rot,interleaved", [(128, 2, 8, 128, 128, False), (64, 1, 5, 16, 32, True),
                                                           (128, 3, 3, 64, 64, False), (64, 8, 64, 32, 64, True),
                                                           (128, 1, 1, 128, 16, False), (128, 2, 4, 32, 0, False)])
def test_decode_rows(dtype, dim, hkv, hq, bs, rot, interleaved):
    lens = [1, 2, 16, 17, 0, 33, 64, 65, 127, 128, 129, 300]
    s = Setup(1 + dim + hq, lens, dtype, hkv, dim, bs)
    _run(s, lens, None, hq=hq, rot=rot, interleaved=interleaved)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,bs,rot,interleaved", [(128, 128, 128, False), (64, 16, 64, True), (128, 64, 32, True),
                                                    (64, 128, 64, False), (128, 16, 128, False)])
def test_packed_rows(dtype, dim, bs, rot, interleaved):
    # (new rows, total): a long chunk, one that ends a block begun before, a single token, one inside a block
    reqs = [(300, 300), (40, 150), (1, 1), (1, 130), (5, 70), (129, 400), (3, 3)]
    s = Setup(2 + dim, [t for _, t in reqs], dtype, 2, dim, bs)
    lens = [t - n + j + 1 for n, t in reqs for j in range(n)]
    r2b = [b for b, (n, _) in enumerate(reqs) for _ in range(n)]
    _run(s, lens, r2b, hq=4, rot=rot, interleaved=interleaved, fused=True)
    assert sai.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_tokens_one_by_one(dtype):
    """A block filled token by token, whose scale grows on the way: each step against the oracle from the step's start."""
    s = Setup(3, [40], dtype, 2, 64, 32)
    for n in range(1, 41):
        _run(s, [n], None, hq=2, rot=64, interleaved=False, sigma=0.01 * 1.4 ** n, with_q=n % 2 == 0)


def test_layout_with_tokens_before_heads():
    for dtype in ("bf16", "e4m3"):
        s = Setup(4, [90, 20], dtype, 2, 128, 16, nhd=True)
        _run(s, list(range(41, 91)) + [20], [0] * 50 + [1], hq=4, rot=128, interleaved=False)


def test_zero_and_nonfinite_values():
    s = Setup(5, [3], "e4m3", 1, 64, 16)
    k = torch.zeros((3, 1, 64), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    v[0, 0, 0], v[1, 0, 1], v[2, 0, 2] = float("nan"), float("inf"), 100.0
    sai.append_kv(s.cache, k, v, _i32(s.table.tolist()), _i32([1, 2, 3]), row_to_batch=_i32([0, 0, 0]))
    kv = s.values()
    blk = int(s.table[0, 0])
    assert kv[2][blk, 0] == 2.0 ** -64 and (kv[0][blk, 0, :3] == 0).all()
    assert kv[3][blk, 0] == 0.25  # 100 <= 448 / 4
    assert np.isnan(kv[1][blk, 0, 0, 0]) and kv[1][blk, 0, 1, 1] == 448 and kv[1][blk, 0, 2, 2] == 384  # 400 is a tie


def test_bad_rows_are_skipped_and_flagged():
    for dtype in ("bf16", "e4m3"):
        s = Setup(6, [100, 50], dtype, 1, 64, 16)
        before = s.bits()
        x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device=DEV)
        cs = torch.from_numpy(_table(64, 60)).to(DEV)
        sai.device_status()
        # length below 0, past the table, past the angles; a request outside the table
        out = sai.append_kv(s.cache, x, x, _i32(s.table.tolist()), _i32([-3, 113, 61, 5]), cs, q=x,
                            row_to_batch=_i32([0, 0, 0, 2]))
        assert sai.device_status() == 1
        assert (out == 0).all()
        table = s.table.copy()
        table[0, 2] = 99
        sai.append_kv(s.cache, x[:1], x[:1], _i32(table.tolist()), _i32([40]), row_to_batch=_i32([0]))
        assert sai.device_status() == 4
        assert all(np.array_equal(a, b) for a, b in zip(before, s.bits()))


def test_another_stream_and_no_rows():
    s = Setup(7, [10], "bf16", 2, 64, 16)
    x = torch.randn((1, 2, 64), device=DEV).to(torch.bfloat16)
    bt, ln = _i32(s.table.tolist()), _i32([10])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = sai.append_kv(s.cache, x, x, bt, ln, q=x, stream=side)
    side.synchronize()
    assert torch.equal(out, x) and torch.equal(s.k[int(s.table[0, 0]), :, 9], x[0])
    sai.append_kv(s.cache, x[:0], x[:0], bt, ln[:0])


def test_refusals():
    s = Setup(8, [10], "bf16", 2, 64, 16)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=DEV)
    bt, ln = _i32(s.table.tolist()), _i32([10])
    with pytest.raises(ValueError, match="must be"):
        sai.append_kv(s.cache, x[:, :1], x, bt, ln)
    with pytest.raises(ValueError, match="bfloat16"):
        sai.append_kv(s.cache, x.float(), x, bt, ln)
    with pytest.raises(ValueError, match="out_q goes with q"):
        sai.append_kv(s.cache, x, x, bt, ln, out_q=x)
    with pytest.raises(sai.SaiError, match="unsupported"):
        sai.append_kv(s.cache, x, x, bt, ln, torch.zeros((16, 24), device=DEV))
    with pytest.raises(sai.SaiError, match="misaligned"):
        odd = torch.zeros(2 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(1, 2, 64)
        sai.append_kv(s.cache, odd, x, bt, ln)
    with pytest.raises(sai.SaiError, match="size or count"):
        sai.append_kv(s.cache, x.expand(3, 2, 64).contiguous(), x.expand(3, 2, 64).contiguous(), bt, _i32([1, 1, 1]))

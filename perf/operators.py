"""What is measured of the cache and attention operators: appending keys and values to a paged cache, attention over
that cache, and attention over the slots that the indexer picked.

``run`` makes the framework's calls where ``own`` is true, and computes the same in plain 32-bit torch operations where
it is false. The cache is paged: ``[blocks, kv heads, block size, dim]`` of bfloat16 or of e4m3 codes, which then have
one fp32 scale for each block and kv head; ``block_table[request, j]`` names the block of tokens ``[j*bs, (j+1)*bs)``.
"""

import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
MIN_EXP = -64  # the smallest block scale is 2**-64


def listed():
    return [
        # appending one decode token of one request: the smallest call, all latency
        dict(name="append decode 1 row bf16", op="append", dtype="bf16", rows=1, requests=1, packed=False, hq=32, hkv=8,
             dim=128, bs=128, rot=128, interleaved=False, min_len=700, max_len=700, lens=1),
        # a decode step of 64 requests into the 8-bit cache
        dict(name="append decode 64 rows e4m3", op="append", dtype="e4m3", rows=64, requests=64, packed=False, hq=64,
             hkv=8, dim=128, bs=128, rot=128, interleaved=False, min_len=4096, max_len=32768, lens=2),
        # a prefill chunk of five requests of odd lengths, rotation of half the dims
        dict(name="append prefill 8191 rows e4m3", op="append", dtype="e4m3", rows=8191, requests=5, packed=True, hq=64,
             hkv=8, dim=128, bs=128, rot=64, interleaved=True, min_len=1, max_len=4000, lens=3),
        # one short chat turn's decode: the smallest attention call
        dict(name="decode 1 row bf16", op="paged", dtype="bf16", rows=1, requests=1, packed=False, hq=32, hkv=8, dim=128,
             bs=128, window=0, sinks=0, min_len=700, max_len=700, lens=4),
        # the fused decode workload's 64 requests of 4096-32768 keys, 8-bit cache
        dict(name="decode 64 rows e4m3", op="paged", dtype="e4m3", rows=64, requests=64, packed=False, hq=64, hkv=8,
             dim=128, bs=128, window=0, sinks=0, min_len=4096, max_len=32768, lens=5),
        # a sliding-window layer's decode over small pages, odd window, three query heads to a kv head
        dict(name="decode 37 rows window bf16", op="paged", dtype="bf16", rows=37, requests=37, packed=False, hq=24,
             hkv=8, dim=128, bs=16, window=2047, sinks=5, min_len=0, max_len=20000, lens=6),
        # a prefill chunk at the end of a 32768-token request: the largest case
        dict(name="prefill 2048 rows bf16", op="paged", dtype="bf16", rows=2048, requests=1, packed=True, hq=32, hkv=4,
             dim=128, bs=128, window=0, sinks=0, min_len=30720, max_len=30720, lens=7),
        # four requests of odd lengths packed in one call, 8-bit cache
        dict(name="prefill 1849 rows e4m3", op="paged", dtype="e4m3", rows=1849, requests=4, packed=True, hq=64, hkv=8,
             dim=128, bs=64, window=0, sinks=0, min_len=0, max_len=8000, lens=8),
        # a sliding-window layer's prefill
        dict(name="prefill 4096 rows window bf16", op="paged", dtype="bf16", rows=4096, requests=1, packed=True, hq=32,
             hkv=8, dim=128, bs=128, window=1024, sinks=4, min_len=0, max_len=0, lens=9),
        # one decode row on the indexer's 512 slots
        dict(name="sparse 1 row e4m3", op="sparse", dtype="e4m3", rows=1, requests=1, packed=False, hq=32, hkv=8, dim=128,
             bs=128, k=512, min_len=9000, max_len=9000, lens=10),
        # a decode step after the indexer: 64 rows, 512 slots each
        dict(name="sparse 64 rows bf16", op="sparse", dtype="bf16", rows=64, requests=64, packed=False, hq=64, hkv=8,
             dim=128, bs=128, k=512, min_len=4096, max_len=16384, lens=11),
        # the fused prefill workload's 4096 causal rows at the end of 32768 tokens, 512 slots each
        dict(name="sparse 4096 rows bf16", op="sparse", dtype="bf16", rows=4096, requests=1, packed=True, hq=32, hkv=4,
             dim=128, bs=128, k=512, min_len=28672, max_len=28672, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "sparse"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16, 64 // hkv])
    while hkv * group > 64:
        group = rng.choice([1, 2, 4, 8])
    c = dict(op=op, dtype=rng.choice(["bf16", "e4m3"]), hq=hkv * group, hkv=hkv, dim=rng.choice([64, 128, 128]),
             bs=rng.choice([16, 32, 64, 128, 128]), lens=rng.randrange(1, 1 << 20))
    packed = c["packed"] = rng.random() < 0.5
    if op == "append":
        c["rot"] = rng.choice([c["dim"], c["dim"] // 2])
        c["interleaved"] = rng.random() < 0.5
        c["rows"] = _log(rng, 2, 8000) if packed else _log(rng, 1, 256)
        c["requests"] = min(c["rows"], rng.randrange(1, 6)) if packed else c["rows"]
        c["min_len"], c["max_len"] = 1, _log(rng, 1, 4000)
    elif op == "paged":
        c["window"] = rng.choice([0, 0, _log(rng, 1, 5000)])
        c["sinks"] = rng.choice([0, rng.randrange(1, 140)]) if c["window"] else 0
        if packed:
            c["rows"] = _log(rng, 2, 2047)
            c["requests"] = min(c["rows"], rng.choice([1, 1, 2, 3, 4]))
            most = 32 * 2048 * 30720 // (c["requests"] * c["hq"] * c["rows"])
            c["min_len"], c["max_len"] = 0, _log(rng, 1, max(1, min(30000, most - c["rows"])))
        else:
            c["rows"] = _log(rng, 1, 64)
            c["requests"] = c["rows"]
            c["min_len"], c["max_len"] = 0, _log(rng, 1, 32000)
    else:
        c["k"] = rng.choice([512, 512, 512, rng.randrange(1, 512)])
        c["rows"] = _log(rng, 2, 4000 * 4 // max(4, hkv)) if packed else _log(rng, 1, 64)
        c["requests"] = 1 if packed else c["rows"]
        c["min_len"], c["max_len"] = 0, _log(rng, 1, 28000 if packed else 16000)
    return c


def _shape(case):
    """Host-side layout: prefix length and number of new rows of each request (the lengths belong to the case)."""
    r = random.Random(case["lens"])
    pre = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["requests"])]
    if not case["packed"]:
        # a row is a request of its own; its length counts its own token
        return pre, [1] * case["rows"]
    cuts = sorted(r.sample(range(1, case["rows"]), case["requests"] - 1))
    new = [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]
    return pre, new


def _row_lens(case):
    pre, new = _shape(case)
    if not case["packed"]:
        return list(pre)
    return [p + j + 1 for p, n in zip(pre, new) for j in range(n)]


def _codes(shape, g, dtype):
    """Cache contents: bf16 N(0, 1), or e4m3 codes that fill the format's range as a scaled block does."""
    n = math.prod(shape)
    if dtype == "bf16":
        return torch.randn(n, generator=g, device=DEV, dtype=torch.bfloat16).view(shape)
    out = torch.empty(n, device=DEV, dtype=torch.uint8)
    step = 1 << 28
    for a in range(0, n, step):
        m = min(step, n - a)
        x = torch.randn(m, generator=g, device=DEV, dtype=torch.bfloat16).mul_(96).clamp_(-E4M3_MAX, E4M3_MAX)
        out[a:a + m] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out.view(shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    bs, hkv, dim = case["bs"], case["hkv"], case["dim"]
    pre, new = _shape(case)
    lens = _row_lens(case)
    total = [p + n if case["packed"] else p for p, n in zip(pre, new)]
    per = [max(1, -(-t // bs)) for t in total]
    blocks = sum(per) + 3
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    width = max(per)
    first = torch.tensor([sum(per[:b]) for b in range(len(per))], device=DEV)
    table = perm[(first[:, None] + torch.arange(width, device=DEV)[None]).clamp_(max=blocks - 1)].contiguous()
    kc, vc = (_codes((blocks, hkv, bs, dim), g, case["dtype"]) for _ in range(2))
    ks = vs = None
    if case["dtype"] == "e4m3":
        ks, vs = (torch.exp2(torch.randint(-8, -5, (blocks, hkv), generator=g, device=DEV).float()) for _ in range(2))
    s = dict(case=case, table=table, kc=kc, vc=vc, ks=ks, vs=vs, max_len=max(max(lens), 1), requests=case["requests"],
             max_rows=max(new), lens=torch.tensor(lens, dtype=torch.int32, device=DEV), row_to_batch=None)
    if case["packed"]:
        s["row_to_batch"] = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(DEV, torch.int32)
    rows, hq = case["rows"], case["hq"]
    # scores of unit-variance heads: a few keys carry most of a softmax, as trained heads have it
    s["q"] = torch.randn((rows, hq, dim), generator=g, device=DEV, dtype=torch.bfloat16).mul_(2.0)
    if case["op"] == "append":
        s["k"], s["v"] = (torch.randn((rows, hkv, dim), generator=g, device=DEV, dtype=torch.bfloat16).mul_(4.0)
                          for _ in range(2))
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        ang = torch.arange(s["max_len"], device=DEV, dtype=torch.float64)[:, None] * freq[None]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    else:
        _poison(s, total, bs)
    if case["op"] == "sparse":
        s["slots"] = _slots(s, case["k"], g)
    if own:  # the handle that a serving program keeps for each layer's cache
        import sparse_attention_indexer_top_gb300 as sai

        s["cache"] = sai.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


def _poison(s, total, bs):
    """Cells past a request's last token hold whatever the block's last owner left there: here NaN."""
    nan = float("nan") if s["ks"] is None else 0x7F
    for b, t in enumerate(total):
        if t % bs:
            blk = s["table"][b, t // bs].long()
            s["kc"][blk, :, t % bs:] = nan
            s["vc"][blk, :, t % bs:] = nan


def _slots(s, k, g):
    """Slots of k distinct earlier tokens of each row, in no order of position, -1 padded."""
    bs, rows = s["case"]["bs"], s["lens"].shape[0]
    out = torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
    b = torch.arange(rows, device=DEV) if s["row_to_batch"] is None else s["row_to_batch"].long()
    for a in range(0, rows, 1024):
        n = s["lens"][a:a + 1024].long()
        x = torch.rand((n.shape[0], s["max_len"]), generator=g, device=DEV)
        x.masked_fill_(torch.arange(s["max_len"], device=DEV)[None] >= n[:, None], -1.0)
        top = x.topk(min(k, s["max_len"]), dim=1)
        t = top.indices
        slot = torch.gather(s["table"][b[a:a + 1024]].long(), 1, t // bs) * bs + t % bs
        out[a:a + 1024, :t.shape[1]] = torch.where(top.values >= 0, slot, -1).to(torch.int32)
    return out


# ------------------------------------------------------------------ plain forms (32 bits, elementary operations)


def _rope32(x, pos, cos_sin, rot, interleaved):
    x = x.float()
    half = rot // 2
    c, sn = cos_sin[pos][:, None, :half], cos_sin[pos][:, None, half:]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y1, y2 = a * c - b * sn, b * c + a * sn
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _put32(x, cache, scale, blk, off, firsts, bs):
    """x [rows, heads, dim] (fp32) into the paged cache at (blk, :, off)."""
    if scale is None:
        cache[blk, :, off] = x.to(torch.bfloat16)
        return cache, None
    heads = torch.arange(x.shape[1], device=x.device)
    amax = x.abs().amax(-1)
    top = torch.zeros_like(scale).index_reduce_(0, blk, amax, "amax")
    start = torch.full((scale.shape[0],), bs, device=x.device).index_reduce_(0, blk, off, "amin")
    # the least power of two with top <= 448 * 2**e, 448 being 0.875 * 2**9
    man, ex = torch.frexp(top)
    e = torch.where(top > 0, ex - 9 + (man > 0.875), MIN_EXP).clamp(min=MIN_EXP).float()
    need = torch.exp2(e)
    new = torch.where((start == 0)[:, None], need, torch.maximum(scale, need))
    # older tokens of a block that was begun before go to the new scale
    fb = blk[firsts]
    old = cache[fb].view(torch.float8_e4m3fn).float() * (scale[fb] / new[fb])[..., None, None]
    old = old.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = torch.arange(bs, device=x.device)[None, None, :, None] < start[fb][:, None, None, None]
    cache[fb] = torch.where(keep, old, cache[fb])
    code = (x / new[blk[:, None], heads[None]][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    cache[blk, :, off] = code.view(torch.uint8)
    scale[fb] = new[fb]
    return cache, scale


def _append32(s):
    c = s["case"]
    bs, rows = c["bs"], c["rows"]
    pos = s["lens"].long() - 1
    b = torch.arange(rows, device=DEV) if s["row_to_batch"] is None else s["row_to_batch"].long()
    blk, off = s["table"][b, pos // bs].long(), pos % bs
    # one row of each block that the call touches, the others of the list being repeats
    begins = torch.ones(rows, dtype=torch.bool, device=DEV)
    begins[1:] = blk[1:] != blk[:-1]
    firsts = torch.argsort(~begins, stable=True)[:min(rows, rows // bs + 2 * c["requests"])]
    k = _rope32(s["k"], pos, s["cos_sin"], c["rot"], c["interleaved"])
    q = _rope32(s["q"], pos, s["cos_sin"], c["rot"], c["interleaved"]).to(torch.bfloat16)
    _put32(k, s["kc"], s["ks"], blk, off, firsts, bs)
    _put32(s["v"].float(), s["vc"], s["vs"], blk, off, firsts, bs)
    return q


def _values32(cache, scale, blk, off):
    """fp32 values [..., heads, dim] of the cache cells (blk, off)."""
    if scale is None:
        return cache[blk, :, off].float()
    return cache[blk, :, off].view(torch.float8_e4m3fn).float() * scale[blk][..., None]


def _softmax32(sc):
    """exp weights, their sum and the log-sum-exp along the last axis; a row of -inf alone has weight 0."""
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc.sub_(m))
    total = p.sum(-1, keepdim=True)
    return p, total, (m + torch.log(total))[..., 0]


def _paged32(s):
    c = s["case"]
    bs, hkv, dim, rows, nb, mr = c["bs"], c["hkv"], c["dim"], c["rows"], s["requests"], s["max_rows"]
    lens, grp = s["lens"].long(), c["hq"] // c["hkv"]
    if s["row_to_batch"] is None:
        b, j = torch.arange(rows, device=DEV), torch.zeros(rows, dtype=torch.long, device=DEV)
    else:
        b = s["row_to_batch"].long()
        j = torch.arange(rows, device=DEV) - torch.searchsorted(b, torch.arange(nb, device=DEV))[b]
    t = torch.arange(s["max_len"], device=DEV)
    n = torch.zeros((nb, mr), dtype=torch.long, device=DEV)
    n[b, j] = lens
    q = torch.zeros((nb, mr, c["hq"], dim), device=DEV)
    q[b, j] = s["q"].float()
    live = t[None] < n.amax(1)[:, None]
    blk = s["table"][:, t // bs].long()
    off = (t % bs)[None].expand_as(blk)
    k = torch.where(live[..., None, None], _values32(s["kc"], s["ks"], blk, off), 0.0)
    q = q.view(nb, mr, hkv, grp, dim).permute(0, 2, 3, 1, 4).reshape(nb, hkv, grp * mr, dim)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)).view(nb, hkv, grp, mr, -1)
    del k
    sc.mul_(dim ** -0.5)
    see = t[None, None] < n[..., None]
    if c["window"]:
        see &= (t >= n[..., None] - c["window"]) | (t < c["sinks"])
    sc.masked_fill_(~see[:, None, None], -math.inf)
    p, total, lse = _softmax32(sc)
    v = torch.where(live[..., None, None], _values32(s["vc"], s["vs"], blk, off), 0.0)
    o = torch.matmul(p.view(nb, hkv, grp * mr, -1), v.transpose(1, 2)).view(nb, hkv, grp, mr, dim)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(nb, mr, c["hq"], dim)[b, j]
    return o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(nb, mr, c["hq"])[b, j]


def _sparse32(s):
    c = s["case"]
    bs, hkv, dim, rows = c["bs"], c["hkv"], c["dim"], c["rows"]
    slots = s["slots"].long()
    live = slots >= 0
    blk, off = slots.clamp(min=0) // bs, slots.clamp(min=0) % bs
    k = torch.where(live[..., None, None], _values32(s["kc"], s["ks"], blk, off), 0.0)
    q = s["q"].float().view(rows, hkv, -1, dim)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(dim ** -0.5)
    del k
    sc.masked_fill_(~live[:, None, None], -math.inf)
    p, total, lse = _softmax32(sc)
    v = torch.where(live[..., None, None], _values32(s["vc"], s["vs"], blk, off), 0.0)
    o = torch.matmul(p, v.transpose(1, 2))
    o = torch.where(total > 0, o / total, 0.0)
    return o.reshape(rows, c["hq"], dim).to(torch.bfloat16), lse.reshape(rows, c["hq"])


def _cache_out(s, q):
    out = dict(q=q)
    for name, cache, scale in (("k", s["kc"], s["ks"]), ("v", s["vc"], s["vs"])):
        out[name] = cache if scale is None else cache.view(torch.float8_e4m3fn)
        if scale is not None:
            out[name + "_scale"] = scale
    return out


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "append":
            return _cache_out(s, _append32(s))
        out, lse = (_paged32 if c["op"] == "paged" else _sparse32)(s)
        return dict(out=out, lse=lse)
    import sparse_attention_indexer_top_gb300 as sai

    if c["op"] == "append":
        q = sai.append_kv(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cos_sin"], q=s["q"],
                          row_to_batch=s["row_to_batch"], interleaved=c["interleaved"])
        return _cache_out(s, q)
    if c["op"] == "paged":
        out, lse = sai.paged_attention(s["q"], s["cache"], s["table"], s["lens"], max_seq_len=s["max_len"],
                                       row_to_batch=s["row_to_batch"], packed=c["packed"], window=c["window"],
                                       sinks=c["sinks"], want_lse=True)
    else:
        out, lse = sai.sparse_attention(s["q"], s["cache"], s["slots"], want_lse=True)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ what a pass cannot do without


def _seen(n, c):
    """Keys that a row of length n sees."""
    if not c["window"] or n <= c["window"]:
        return n
    return c["window"] + min(c["sinks"], n - c["window"])


def work(case):
    elem = 2 if case["dtype"] == "bf16" else 1
    rows, hq, hkv, dim, bs = (case[x] for x in ("rows", "hq", "hkv", "dim", "bs"))
    pre, new = _shape(case)
    lens = _row_lens(case)
    if case["op"] == "append":
        read = rows * (hq + 2 * hkv) * dim * 2 + rows * 12 + len(set(lens)) * case["rot"] * 4
        write = rows * (hq * 2 + 2 * hkv * elem) * dim
        scales = 0 if elem == 2 else 2 * 4 * hkv * sum((p + n - 1) // bs - p // bs + 1 for p, n in zip(pre, new))
        return dict(bytes=read + write + 2 * scales, flops=rows * (hq + hkv) * case["rot"] * 3)
    if case["op"] == "paged":
        pairs = sum(_seen(n, case) for n in lens)
        if case["packed"]:
            # the union of what a request's rows see: all but what lies before the first row's window
            tokens = 0
            for p, n in zip(pre, new):
                low = max(0, p + 1 - case["window"]) if case["window"] else 0
                tokens += p + n - low + min(low, case["sinks"])
        else:
            tokens = pairs
        meta = rows * 8 + 4 * (tokens // bs + len(pre))
    else:
        pairs = sum(min(n, case["k"]) for n in lens)
        tokens = min(pairs, sum(p + n if case["packed"] else p for p, n in zip(pre, new)))
        meta = rows * case["k"] * 4
    scales = 0 if elem == 2 else 8 * hkv * (tokens // bs + 1)
    return dict(bytes=tokens * hkv * dim * 2 * elem + rows * hq * (dim * 4 + 4) + meta + scales,
                flops=4 * pairs * hq * dim)


# ------------------------------------------------------------------ the definitions, in 64 bits


def _e4m3_round(x):
    """x (float64, |x| <= 448) at the nearest e4m3 value, ties to even."""
    mag = x.abs()
    _, e = torch.frexp(mag)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    return torch.sign(x) * torch.round(mag / step) * step


def _exact_rope(x, lens, cos_sin, rot, interleaved):
    y = x.double().clone()
    half = rot // 2
    cs = cos_sin.double()[lens.long() - 1]
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, sn = cs[:, None, i], cs[:, None, half + i]
        y[..., lo] = x[..., lo].double() * c - x[..., hi].double() * sn
        y[..., hi] = x[..., hi].double() * c + x[..., lo].double() * sn
    return y


def _exact_put(x, cache, scale, case, table, pre, new, packed):
    """Request by request, block by block, on float64 values (codes for an 8-bit cache)."""
    bs = case["bs"]
    out = cache.double() if scale is None else cache.view(torch.float8_e4m3fn).double()
    so = None if scale is None else scale.double().clone()
    row = 0
    for b, (p, n) in enumerate(zip(pre, new)):
        pos = p if packed else p - 1
        while n:
            o = pos % bs
            m = min(bs - o, n)
            blk = int(table[b, pos // bs])
            part = x[row:row + m].transpose(0, 1)
            if so is not None:
                amax = part.abs().amax((1, 2))
                need = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(min=MIN_EXP))
                if o:
                    was = so[blk].clone()
                    so[blk] = torch.maximum(was, need)
                    out[blk, :, :o] = _e4m3_round(out[blk, :, :o] * (was / so[blk])[:, None, None])
                else:
                    so[blk] = need
                part = _e4m3_round(part / so[blk][:, None, None])
            out[blk, :, o:o + m] = part
            row, pos, n = row + m, pos + m, n - m
    return out, so


def _cells(cache, scale, blk, off):
    x = cache[blk, :, off]
    if scale is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * scale[blk].double()[..., None]


def _attend64(q, k, v, see, dim):
    """q [m, hkv, g, dim], k and v [n, hkv, dim], see [m, n]: outputs [m, hq, dim] and log-sum-exps [m, hq]."""
    m, hkv, g, _ = q.shape
    sc = torch.einsum("mhgd,nhd->mhgn", q.double(), k) / math.sqrt(dim)
    sc = sc.masked_fill(~see[:, None, None], -math.inf)
    lse = torch.logsumexp(sc, -1)
    w = torch.exp(sc - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    return torch.einsum("mhgn,nhd->mhgd", w, v).reshape(m, hkv * g, dim), lse.reshape(m, hkv * g)


def exact(case, seed):
    s = prepare(case, seed)
    pre, new = _shape(case)
    rows, hq, hkv, dim, bs = (case[x] for x in ("rows", "hq", "hkv", "dim", "bs"))
    if case["op"] == "append":
        k = _exact_rope(s["k"], s["lens"], s["cos_sin"], case["rot"], case["interleaved"])
        out = dict(q=_exact_rope(s["q"], s["lens"], s["cos_sin"], case["rot"], case["interleaved"]))
        for name, x, cache, scale in (("k", k, s["kc"], s["ks"]), ("v", s["v"].double(), s["vc"], s["vs"])):
            out[name], so = _exact_put(x, cache, scale, case, s["table"], pre, new, case["packed"])
            if so is not None:
                out[name + "_scale"] = so
        return out
    out = torch.zeros((rows, hq, dim), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=DEV)
    q = s["q"].view(rows, hkv, hq // hkv, dim)
    if case["op"] == "sparse":
        slots = s["slots"].long()
        for i in range(0, rows, 256):
            at = slots[i:i + 256]
            see = at >= 0
            blk, off = at.clamp(min=0) // bs, at.clamp(min=0) % bs
            k, v = (_cells(c, z, blk, off).masked_fill(~see[..., None, None], 0.0)
                    for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            sc = torch.einsum("mhgd,mnhd->mhgn", q[i:i + 256].double(), k) / math.sqrt(dim)
            sc = sc.masked_fill(~see[:, None, None], -math.inf)
            l = torch.logsumexp(sc, -1)
            w = torch.exp(sc - l.masked_fill(l == -math.inf, 0.0)[..., None])
            out[i:i + 256] = torch.einsum("mhgn,mnhd->mhgd", w, v).reshape(-1, hq, dim)
            lse[i:i + 256] = l.reshape(-1, hq)
        return dict(out=out, lse=lse)
    lens, row = _row_lens(case), 0
    for b, n in enumerate(new):
        top = lens[row + n - 1]
        t = torch.arange(top, device=DEV)
        if top:
            blk, off = s["table"][b].long()[t // bs], t % bs
            k, v = _cells(s["kc"], s["ks"], blk, off), _cells(s["vc"], s["vs"], blk, off)
            step = max(1, (1 << 28) // (top * hq))
            for i in range(row, row + n, step):
                e = min(i + step, row + n)
                ln = s["lens"][i:e].long()[:, None]
                see = t[None] < ln
                if case["window"]:
                    see = see & ((t[None] >= ln - case["window"]) | (t[None] < case["sinks"]))
                out[i:e], lse[i:e] = _attend64(q[i:e], k, v, see, dim)
        row += n
    return dict(out=out, lse=lse)

"""What is measured of the attention with changed scores and masks, and of the operators on a cache's pages: copying
them, forking requests, growing, shrinking and ending them, and compacting the pool.

``run`` makes the framework's calls where ``own`` is true, and computes the same in plain torch operations where it is
false. The caches are paged: ``[blocks, kv heads, block size, dim]`` (or tokens before heads) of bfloat16 or of e4m3
codes, which then have one fp32 scale for each block and kv head; ``block_table[request, j]`` names the block of tokens
``[j*bs, (j+1)*bs)``, and ``refs[block]`` counts the requests that hold a block, 0 being free.
"""

import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    paged = dict(op="attention", kind="paged", window=0, sinks=0, softcap=0.0, slopes=False, docs=0, prefix=0)
    pages = dict(layout="hnd", index=False, share=1, dim=128)
    return [
        # one short chat turn's decode with capped scores: the smallest attention call, all latency
        dict(paged, name="decode 1 row softcap bf16", dtype="bf16", rows=1, requests=1, packed=False, hq=32, hkv=8, dim=128,
             bs=128, min_len=700, max_len=700, softcap=50.0, lens=1),
        # a decode step of 64 requests of 4096-32768 keys, biased by distance, 8-bit cache
        dict(paged, name="decode 64 rows slopes e4m3", dtype="e4m3", rows=64, requests=64, packed=False, hq=64, hkv=8,
             dim=128, bs=128, min_len=4096, max_len=32768, slopes=True, lens=2),
        # a prefill chunk with capped scores at the end of a 32768-token request: the largest case
        dict(paged, name="prefill 2048 rows softcap bf16", dtype="bf16", rows=2048, requests=1, packed=True, hq=32, hkv=4,
             dim=128, bs=128, min_len=30720, max_len=30720, softcap=50.0, lens=3),
        # documents packed into one sequence, each with a prefix that all its tokens see, biased by distance
        dict(paged, name="prefill 3001 rows documents e4m3", dtype="e4m3", rows=3001, requests=1, packed=True, hq=64, hkv=8,
             dim=128, bs=64, min_len=0, max_len=0, slopes=True, docs=700, prefix=100, lens=4),
        # a request's prompt handed to another place of the pool: the smallest copy
        dict(pages, name="copy 3 pages bf16", op="copy", dtype="bf16", layers=1, hkv=8, bs=128, blocks=64, pairs=3, lens=5),
        # pages of four layers and their index keys on their way out of or into a window of the pool
        dict(pages, name="copy 500 pages 4 layers e4m3", op="copy", dtype="e4m3", layers=4, hkv=8, bs=128, blocks=1024,
             pairs=500, index=True, lens=6),
        # one step of a beam search over one prompt
        dict(name="fork 8 beams", op="fork", requests=8, share=8, min_len=1000, max_len=1000, tail=40, width=16, bs=128,
             blocks=1024, children=8, lens=7),
        # samples of many prompts taken up, dropped and doubled at once
        dict(name="fork 512 requests", op="fork", requests=512, share=2, min_len=10000, max_len=60000, tail=3000, width=512,
             bs=128, blocks=131072, children=600, lens=8),
        # a decode step of four beams each of four prompts, which still share their last pages
        dict(pages, name="resize 16 beams 4 layers bf16", op="resize", dtype="bf16", layers=4, hkv=4, bs=128, blocks=256,
             requests=16, share=4, tail=0, min_len=300, max_len=3000, spare=64, mix=False, lens=9, width=32),
        # a server's step: requests end, are rolled back, decode, or get a prompt
        dict(pages, name="resize 160 requests e4m3", op="resize", dtype="e4m3", layers=2, hkv=4, bs=64, blocks=6144,
             requests=160, share=2, tail=500, min_len=100, max_len=4000, spare=2000, mix=True, lens=10, width=96),
        # a small pool after a few requests ended
        dict(pages, name="compact 200 pages bf16", op="compact", dtype="bf16", layers=1, hkv=2, bs=16, blocks=512, requests=7,
             share=1, tail=0, min_len=1, max_len=700, width=64, lens=11, dim=64),
        # a pool of four layers half of whose pages have become free
        dict(pages, name="compact 4096 pages 4 layers e4m3", op="compact", dtype="e4m3", layers=4, hkv=4, bs=64, blocks=4096,
             requests=40, share=2, tail=700, min_len=1000, max_len=6000, width=128, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "copy", "fork", "resize", "resize", "compact"])
    c = dict(op=op, lens=rng.randrange(1, 1 << 20))
    if op == "attention":
        return _draw_attention(rng, c)
    if op == "fork":
        c.update(requests=_log(rng, 1, 512), share=rng.choice([1, 1, 2, 4, 8]), bs=rng.choice([16, 32, 64, 128]))
        c["tail"] = rng.choice([0, _log(rng, 1, 100)])
        c["max_len"] = _log(rng, 1, min(20000, 512 * c["bs"] - 100))
        c["min_len"] = c["max_len"] // 2
        c["width"] = -(-(c["max_len"] + c["tail"]) // c["bs"]) + rng.randrange(0, 9)
        c["blocks"] = c["requests"] * c["width"] + rng.randrange(1, 1000)
        c["children"] = _log(rng, 1, 600)
        return c
    c.update(dtype=rng.choice(["bf16", "e4m3"]), layers=rng.choice([1, 1, 2, 3, 4]), hkv=rng.choice([1, 2, 4, 8]),
             bs=rng.choice([16, 32, 64, 128]), dim=rng.choice([64, 128, 128]), layout=rng.choice(["hnd", "nhd"]),
             index=rng.random() < 0.3, share=rng.choice([1, 2, 4]))
    page = c["layers"] * c["hkv"] * c["bs"] * c["dim"]  # keys' elements of a page
    c["blocks"] = _log(rng, 16, max(17, min(20000, (1 << 29) // page)))
    if op == "copy":
        c["pairs"] = _log(rng, 1, c["blocks"] // 2)
        return c
    c["requests"] = min(200, _log(rng, 1, max(1, c["blocks"] // 8)))
    most = max(1, c["blocks"] * c["bs"] // (2 * c["requests"]) - c["bs"])
    c["tail"] = rng.choice([0, _log(rng, 1, most)])
    c["max_len"] = _log(rng, 1, most)
    c["min_len"] = c["max_len"] // 3
    c["width"] = -(-2 * (c["max_len"] + c["tail"]) // c["bs"]) + 2
    if op == "resize":
        c["mix"] = rng.random() < 0.6
        c["spare"] = rng.randrange(0, c["blocks"] // 2 + 1)
        if rng.random() < 0.3:  # a pool that runs out
            c["spare"] = 0
            c["blocks"] = max(16, len(_held(c)[2]) + rng.randrange(0, c["requests"] + 1))
    return c


def _draw_attention(rng, c):
    kind = c["kind"] = rng.choice(["paged", "paged", "paged", "sparse"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16, 64 // hkv) if g * hkv <= 64])
    packed = c["packed"] = kind == "paged" and rng.random() < 0.6
    c.update(dtype=rng.choice(["bf16", "e4m3"]), hq=hkv * group, hkv=hkv, dim=rng.choice([64, 128, 128]),
             bs=rng.choice([16, 32, 64, 128, 128]), window=0, sinks=0, slopes=False, docs=0, prefix=0,
             softcap=rng.choice([0.0, 20.0, 50.0, rng.uniform(5, 200)]))
    if kind == "sparse":
        c.update(softcap=c["softcap"] or 30.0, k=rng.choice([512, rng.randrange(1, 512)]), rows=_log(rng, 1, 64))
        c["requests"], c["min_len"], c["max_len"] = c["rows"], 0, _log(rng, 1, 16000)
        return c
    c["slopes"] = rng.random() < 0.5 or c["softcap"] == 0.0
    c["window"] = rng.choice([0, 0, _log(rng, 1, 5000)])
    c["sinks"] = rng.choice([0, rng.randrange(1, 140)]) if c["window"] else 0
    c["docs"] = rng.choice([0, _log(rng, 1, 3000)])
    c["prefix"] = rng.choice([0, _log(rng, 1, 600)]) if packed else 0
    if packed:
        c["rows"] = _log(rng, 2, 2047)
        c["requests"] = min(c["rows"], rng.choice([1, 1, 2, 3, 4]))
        most = 32 * 2048 * 30720 // (c["requests"] * c["hq"] * c["rows"])
        c["min_len"], c["max_len"] = 0, _log(rng, 1, max(1, min(30000, most - c["rows"])))
    else:
        c["rows"] = c["requests"] = _log(rng, 1, 64)
        c["min_len"], c["max_len"] = 0, _log(rng, 1, 32000)
    return c


# ------------------------------------------------------------------ the cases' layouts, on the host


def _shape(case):
    """Attention: length before, and number of new rows, of each request (the lengths belong to the case)."""
    r = random.Random(case["lens"])
    pre = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["requests"])]
    if not case["packed"]:
        return pre, [1] * case["rows"]  # a row is a request of its own; its length counts its own token
    cuts = sorted(r.sample(range(1, case["rows"]), case["requests"] - 1))
    return pre, [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]


def _rows(case):
    """Attention: (lengths, first tokens of the rows' documents, ends of their prefixes), one for each row."""
    r = random.Random(case["lens"] + 1)
    pre, new = _shape(case)
    if not case["packed"]:
        starts = [r.randint(max(0, n - case["docs"]), n) for n in pre] if case.get("docs") else [0] * len(pre)
        return pre, starts, [0] * len(pre)
    lens, starts, ends = [], [], []
    for p, n in zip(pre, new):
        at = 0
        cut = p + n if not case["docs"] else 0  # end of the document at work
        for t in range(p + n):
            if t == cut or t == 0:
                at = t
                cut = min(p + n, t + r.randint(1, 2 * case["docs"])) if case["docs"] else p + n
            if t >= p:
                lens.append(t + 1)
                starts.append(at)
                ends.append(min(cut, at + case["prefix"]))
    return lens, starts, ends


def _held(case):
    """Pages: the requests' pages by number, their lengths, and how many hold each page. Groups of ``share`` requests
    continue one prompt, whose whole pages they share, and its last one too while none has gone on."""
    r = random.Random(case["lens"])
    bs, cap = case["bs"], case["blocks"]
    rows, lens, refs = [], [], []

    def page():
        refs.append(0)
        return len(refs) - 1

    for g in range(0, case["requests"], case["share"]):
        prompt = r.randint(case["min_len"], case["max_len"])
        n = min(case["share"], case["requests"] - g)
        tails = [r.randint(0, case["tail"]) for _ in range(n)]
        need = -(-prompt // bs) + sum(-(-t // bs) + 1 for t in tails)
        if len(refs) + need > cap - case.get("spare", 0) or max(prompt + max(tails), 1) > case["width"] * bs:
            prompt, tails = 0, [0] * n  # no room: requests that have not begun
        whole = [page() for _ in range(prompt // bs)]
        last = page() if prompt % bs and 0 in tails else None
        for t in tails:
            row = list(whole)
            if t == 0 and last is not None:
                row.append(last)
            while len(row) * bs < prompt + t:
                row.append(page())
            for x in row:
                refs[x] += 1
            rows.append(row)
            lens.append(prompt + t)
    return rows, lens, refs


def _new_lens(case, lens):
    r = random.Random(case["lens"] + 2)
    top = case["width"] * case["bs"]
    if not case["mix"]:
        return [min(top, n + 1) for n in lens]
    out = []
    for n in lens:
        k = r.random()
        out.append(0 if k < 0.15 else r.randint(0, n) if k < 0.3 else min(top, n + 1) if k < 0.8
                   else min(top, n + r.randint(1, max(1, case["max_len"]))))
    return out


def _parents(case):
    r = random.Random(case["lens"] + 3)
    return [r.randrange(case["requests"]) if r.random() < 0.9 else -1 for _ in range(case["children"])]


# ------------------------------------------------------------------ inputs


def _codes(shape, g, dtype):
    """Cache contents: bf16 N(0, 1), or e4m3 codes that fill the format's range as a scaled block does."""
    n = math.prod(shape)
    if dtype == "bf16":
        return torch.randn(n, generator=g, device=DEV, dtype=torch.bfloat16).view(shape)
    out = torch.empty(n, device=DEV, dtype=torch.uint8)
    step = 1 << 28
    for a in range(0, n, step):
        m = min(step, n - a)
        x = torch.randn(m, generator=g, device=DEV, dtype=torch.bfloat16).mul_(96).clamp_(-448, 448)
        out[a:a + m] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out.view(shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return _prepare_attention(case, g) if case["op"] == "attention" else _prepare_pages(case, g)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _prepare_attention(case, g):
    bs, hkv, dim = case["bs"], case["hkv"], case["dim"]
    pre, new = _shape(case)
    lens, starts, ends = _rows(case)
    total = [p + n if case["packed"] else p for p, n in zip(pre, new)]
    per = [max(1, -(-t // bs)) for t in total]
    blocks = sum(per) + 3
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(per[:b]) for b in range(len(per))], device=DEV)
    table = perm[(first[:, None] + torch.arange(max(per), device=DEV)[None]).clamp_(max=blocks - 1)].contiguous()
    kc, vc = (_codes((blocks, hkv, bs, dim), g, case["dtype"]) for _ in range(2))
    ks = vs = None
    if case["dtype"] == "e4m3":
        ks, vs = (torch.exp2(torch.randint(-8, -5, (blocks, hkv), generator=g, device=DEV).float()) for _ in range(2))
    s = dict(case=case, table=table, kc=kc, vc=vc, ks=ks, vs=vs, max_len=max(max(lens), max(ends), 1),
             requests=case["requests"], max_rows=max(new), lens=_ints(lens), row_to_batch=None, slopes=None, starts=None,
             ends=None)
    if case["packed"]:
        s["row_to_batch"] = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(DEV, torch.int32)
    if case["docs"]:
        s["starts"] = _ints(starts)
    if case["prefix"]:
        s["ends"] = _ints(ends)
    if case["slopes"]:  # the geometric slopes that such models have
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["hq"] + 1, device=DEV, dtype=torch.float64) / case["hq"]).float()
    # scores of a few units, as trained heads have them; capped ones reach the cap's bend
    s["q"] = torch.randn((case["rows"], case["hq"], dim), generator=g, device=DEV, dtype=torch.bfloat16).mul_(2.0)
    nan = float("nan") if ks is None else 0x7F
    for b, t in enumerate(total):  # cells past a request's last token hold whatever the block's last owner left: here NaN
        if t % bs:
            blk = table[b, t // bs].long()
            kc[blk, :, t % bs:] = nan
            vc[blk, :, t % bs:] = nan
    if case["kind"] == "sparse":
        s["slots"] = _slots(s, case["k"], g)
    if own:  # the handle that a serving program keeps for each layer's cache
        import sparse_attention_indexer_top_gb300 as sai

        s["cache"] = sai.KVCache(kc, vc, ks, vs)
    return s


def _slots(s, k, g):
    """Slots of k distinct earlier tokens of each row, in no order of position, -1 padded."""
    bs, n = s["case"]["bs"], s["lens"].long()
    out = torch.full((n.shape[0], k), -1, dtype=torch.int32, device=DEV)
    x = torch.rand((n.shape[0], s["max_len"]), generator=g, device=DEV)
    x.masked_fill_(torch.arange(s["max_len"], device=DEV)[None] >= n[:, None], -1.0)
    top = x.topk(min(k, s["max_len"]), dim=1)
    slot = torch.gather(s["table"].long(), 1, top.indices // bs) * bs + top.indices % bs
    out[:, :top.indices.shape[1]] = torch.where(top.values >= 0, slot, -1).to(torch.int32)
    return out


def _prepare_pages(case, g):
    nb, bs = case["blocks"], case["bs"]
    s = dict(case=case)
    perm = torch.randperm(nb, generator=g, device=DEV)
    if case["op"] == "copy":
        s["src"], s["dst"] = perm[:case["pairs"]].to(torch.int32), perm[-case["pairs"]:].to(torch.int32)
    else:
        rows, lens, refs = _held(case)
        flat = torch.tensor([x for r in rows for x in r + [-1] * (case["width"] - len(r))], device=DEV)
        s["table"] = torch.where(flat >= 0, perm[flat.clamp(min=0)], -1).to(torch.int32).view(len(rows), case["width"])
        s["lens"] = _ints(lens)
        s["refs"] = torch.zeros(nb, dtype=torch.int32, device=DEV)
        s["refs"][perm[:len(refs)]] = _ints(refs)
        if case["op"] == "fork":
            shift = int(torch.randint(0, case["requests"], (1,), generator=g, device=DEV))
            s["parents"] = _ints([-1 if p < 0 else (p + shift) % case["requests"] for p in _parents(case)])
            return s
        if case["op"] == "resize":
            s["new_lens"] = _ints(_new_lens(case, lens))
    h, d = case["hkv"], case["dim"]
    inner = (h, bs, d) if case["layout"] == "hnd" else (bs, h, d)
    s["kv"] = _codes((case["layers"], 2, nb) + inner, g, case["dtype"])
    if case["dtype"] == "e4m3":
        s["scale"] = torch.exp2(torch.randint(-8, -5, (case["layers"], 2, nb, h), generator=g, device=DEV).float())
    if case["index"]:  # the indexer's keys of the same blocks
        s["index_k"] = _codes((case["layers"], nb, bs, 128), g, "e4m3")
        s["index_scale"] = torch.rand((case["layers"], nb, bs), generator=g, device=DEV)
    if own:  # the handle of a server's pool
        import sparse_attention_indexer_top_gb300 as sai

        view = (lambda x: x) if case["layout"] == "hnd" else (lambda x: x.transpose(1, 2))
        caches = [sai.KVCache(view(s["kv"][i, 0]), view(s["kv"][i, 1]),
                              *((s["scale"][i, 0], s["scale"][i, 1]) if "scale" in s else ()))
                  for i in range(case["layers"])]
        s["pages"] = sai.PageSet(caches, [x for n in ("index_k", "index_scale") if n in s for x in s[n].unbind(0)])
    return s


# ------------------------------------------------------------------ plain forms


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


def _cap32(sc, cap):
    return sc.div_(cap).tanh_().mul_(cap) if cap else sc


def _paged32(s):
    c = s["case"]
    bs, hkv, dim, rows, nb, mr = c["bs"], c["hkv"], c["dim"], c["rows"], s["requests"], s["max_rows"]
    grp = c["hq"] // c["hkv"]
    if s["row_to_batch"] is None:
        b, j = torch.arange(rows, device=DEV), torch.zeros(rows, dtype=torch.long, device=DEV)
    else:
        b = s["row_to_batch"].long()
        j = torch.arange(rows, device=DEV) - torch.searchsorted(b, torch.arange(nb, device=DEV))[b]
    t = torch.arange(s["max_len"], device=DEV)
    n, lo, hi = (torch.zeros((nb, mr, 1), dtype=torch.long, device=DEV) for _ in range(3))
    n[b, j, 0] = s["lens"].long()
    if s["starts"] is not None:
        lo[b, j, 0] = s["starts"].long()
    if s["ends"] is not None:
        hi[b, j, 0] = s["ends"].long()
    hi = torch.where(n > 0, torch.maximum(n, hi), 0)
    q = torch.zeros((nb, mr, c["hq"], dim), device=DEV)
    q[b, j] = s["q"].float()
    live = t[None] < hi.amax((1, 2))[:, None]
    blk = s["table"][:, t // bs].long()
    off = (t % bs)[None].expand_as(blk)
    k = torch.where(live[..., None, None], _values32(s["kc"], s["ks"], blk, off), 0.0)
    q = q.view(nb, mr, hkv, grp, dim).permute(0, 2, 3, 1, 4).reshape(nb, hkv, grp * mr, dim)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)).view(nb, hkv, grp, mr, -1)
    del k
    sc = _cap32(sc.mul_(dim ** -0.5), c["softcap"])
    if s["slopes"] is not None:
        sc -= s["slopes"].view(hkv, grp)[None, :, :, None, None] * (n - 1 - t).abs().float()[:, None, None]
    see = (t < hi) & (t >= lo)
    if c["window"]:
        see &= (t >= n - c["window"]) | (t < lo + c["sinks"])
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
    sc = _cap32(torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(dim ** -0.5), c["softcap"])
    sc.masked_fill_(~live[:, None, None], -math.inf)
    p, total, lse = _softmax32(sc)
    v = torch.where(live[..., None, None], _values32(s["vc"], s["vs"], blk, off), 0.0)
    o = torch.matmul(p, v.transpose(1, 2))
    o = torch.where(total > 0, o / total, 0.0)
    return o.reshape(rows, c["hq"], dim).to(torch.bfloat16), lse.reshape(rows, c["hq"])


def _move(s, src, dst, cells=None):
    """Pages src to dst of every array; of keys and values the first ``cells`` tokens of each."""
    part = s["kv"][:, :, src]
    if cells is not None:
        tok = torch.arange(s["case"]["bs"], device=DEV)
        keep = tok[None] < cells[:, None]
        keep = keep[:, None, :, None] if s["case"]["layout"] == "hnd" else keep[:, :, None, None]
        part = torch.where(keep, part, s["kv"][:, :, dst])
    s["kv"][:, :, dst] = part
    if "scale" in s:
        s["scale"][:, :, dst] = s["scale"][:, :, src]
    if "index_k" in s:
        s["index_k"][:, dst] = s["index_k"][:, src]
        s["index_scale"][:, dst] = s["index_scale"][:, src]


def _fork(s):
    table, lens, refs, parents = s["table"], s["lens"], s["refs"], s["parents"].long()
    on, at = parents >= 0, parents.clamp(min=0)
    children = torch.zeros_like(lens).index_add_(0, at, on.to(torch.int32))
    col = torch.arange(table.shape[1], device=DEV)
    held = col[None] < (-(-lens // s["case"]["bs"]))[:, None]
    more = torch.where(held, (children - 1)[:, None], 0)
    refs = refs.index_add(0, torch.where(held, table, 0).flatten().long(), more.flatten().to(torch.int32))
    return torch.where(on[:, None], table[at], -1), torch.where(on, lens[at], 0), refs


def _resize(s):
    table, lens, new, refs, bs = s["table"], s["lens"].long(), s["new_lens"].long(), s["refs"], s["case"]["bs"]
    free = (refs <= 0).nonzero()[:, 0]
    req, col = torch.arange(lens.shape[0], device=DEV), torch.arange(table.shape[1], device=DEV)[None]
    have, want = -(-lens // bs), -(-new // bs)
    last = table[req, (lens // bs).clamp(max=table.shape[1] - 1)].long()
    shared = (new > lens) & (lens % bs > 0)
    shared &= refs[last.clamp(min=0)] > 1
    # the last of a page's holders keeps it where all of them go on
    same = (last[:, None] == last[None]) & shared[:, None] & shared[None]
    keeps = shared & (same.sum(1) == refs[last.clamp(min=0)]) & ~(same & (req[None] > req[:, None])).any(1)
    copies = shared & ~keeps
    need = copies.long() + (want - have).clamp(min=0)
    upto = need.cumsum(0)
    served = (upto <= free.shape[0]) | ((need == 0) & ~keeps)
    first = (upto - need)[:, None]
    grown = served[:, None] & (col >= have[:, None]) & (col < want[:, None])
    fresh = served[:, None] & copies[:, None] & (col == (lens // bs)[:, None])
    rank = torch.where(fresh, first, first + copies[:, None] + col - have[:, None])
    pages = torch.cat([free, free.new_zeros(1)])[rank.clamp(0, free.shape[0])].to(torch.int32)
    gone = served[:, None] & (col >= want[:, None]) & (col < have[:, None])
    takes = grown | fresh
    refs = refs.clone()
    refs[pages[takes].long()] = 1
    refs.index_add_(0, table[gone | fresh].long(), torch.full((1,), -1, dtype=torch.int32, device=DEV).expand(
        int((gone | fresh).sum())))
    _move(s, table[fresh].long(), pages[fresh].long(), (lens % bs)[fresh.any(1)])
    return torch.where(takes, pages, torch.where(gone, -1, table)), torch.where(served, new, lens).to(torch.int32), refs


def _compact(s):
    table, refs = s["table"], s["refs"]
    ids = torch.arange(refs.shape[0], device=DEV)
    on = refs > 0
    count = on.sum()
    src, dst = (on & (ids >= count)).nonzero()[:, 0], (~on & (ids < count)).nonzero()[:, 0]
    moves = torch.where(on, ids, -1).to(torch.int32)
    moves[src] = dst.to(torch.int32)
    refs = refs.clone()
    refs[dst] = refs[src]
    refs[src] = 0
    held = torch.arange(table.shape[1], device=DEV)[None] < (-(-s["lens"] // s["case"]["bs"]))[:, None]
    table = torch.where(held, moves[torch.where(held, table, 0).long()], table)
    _move(s, src, dst)
    return table, refs, moves


def _arrays(s):
    """The pool's contents, 8-bit codes as the values they stand for."""
    f8 = torch.float8_e4m3fn
    out = dict(kv=s["kv"] if s["case"]["dtype"] == "bf16" else s["kv"].view(f8))
    if "scale" in s:
        out["scale"] = s["scale"]
    if "index_k" in s:
        out.update(index_k=s["index_k"].view(f8), index_scale=s["index_scale"])
    return out


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import sparse_attention_indexer_top_gb300 as sai

    if op == "attention":
        if not own:
            out, lse = (_paged32 if c["kind"] == "paged" else _sparse32)(s)
        elif c["kind"] == "paged":
            out, lse = sai.paged_attention(s["q"], s["cache"], s["table"], s["lens"], max_seq_len=s["max_len"],
                                           row_to_batch=s["row_to_batch"], packed=c["packed"], window=c["window"],
                                           sinks=c["sinks"], want_lse=True, softcap=c["softcap"], slopes=s["slopes"],
                                           row_starts=s["starts"], prefix_lens=s["ends"])
        else:
            out, lse = sai.sparse_attention(s["q"], s["cache"], s["slots"], want_lse=True, softcap=c["softcap"])
        return dict(out=out, lse=lse)
    if op == "copy":
        if own:
            sai.copy_pages(s["pages"], s["src"], s["dst"])
        else:
            _move(s, s["src"].long(), s["dst"].long())
        return _arrays(s)
    if op == "fork":
        if own:
            table, lens, refs = sai.fork_pages(s["table"], s["lens"], s["refs"], s["parents"], block_size=c["bs"])
        else:
            table, lens, refs = _fork(s)
        return dict(table=table, lens=lens, refs=refs)
    if op == "resize":
        if own:
            table, lens, refs = sai.resize_pages(s["pages"], s["table"], s["lens"], s["new_lens"], s["refs"])
        else:
            table, lens, refs = _resize(s)
        return dict(_arrays(s), table=table, lens=lens, refs=refs)
    if own:
        table, refs, moves = sai.compact_pages(s["pages"], s["table"], s["lens"], s["refs"])
    else:
        table, refs, moves = _compact(s)
    return dict(_arrays(s), table=table, refs=refs, moves=moves)


# ------------------------------------------------------------------ what a pass cannot do without


def _sees(n, lo, hi, window, sinks):
    """Numbers of keys that a row sees: of its first tokens, and from its window on."""
    hi = max(n, hi) if n else 0
    first = max(lo, n - window) if window else lo
    return max(0, min(lo + sinks, first, hi) - lo), max(0, hi - first)


def work(case):
    if case["op"] != "attention":
        return _work_pages(case)
    elem = 2 if case["dtype"] == "bf16" else 1
    rows, hq, hkv, dim, bs = (case[x] for x in ("rows", "hq", "hkv", "dim", "bs"))
    if case["kind"] == "sparse":
        pairs = tokens = sum(min(n, case["k"]) for n in _shape(case)[0])
        meta = rows * case["k"] * 4
    else:
        pre, new = _shape(case)
        lens, starts, ends = _rows(case)
        seen = [_sees(*x, case["window"], case["sinks"]) for x in zip(lens, starts, ends)]
        pairs = sum(a + b for a, b in seen)
        tokens, at = 0, 0
        for n in new:  # the union of what a request's rows see, as the span of their windows (and its first tokens)
            if case["packed"]:
                part = [i for i in range(at, at + n) if sum(seen[i])]
                if part:
                    low = min(max(starts[i], lens[i] - case["window"]) if case["window"] else starts[i] for i in part)
                    tokens += max(max(lens[i], ends[i]) for i in part) - low
            else:
                tokens += sum(seen[at])
            at += n
        meta = rows * 4 * (2 + bool(case["docs"]) + bool(case["prefix"])) + 4 * (tokens // bs + len(pre))
    scales = 0 if elem == 2 else 8 * hkv * (tokens // bs + 1)
    return dict(bytes=tokens * hkv * dim * 2 * elem + rows * hq * (dim * 4 + 4) + meta + scales,
                flops=4 * pairs * hq * dim)


def _work_pages(case):
    if case["op"] == "fork":
        cells = (case["requests"] + case["children"]) * case["width"]
        return dict(bytes=4 * (cells + 2 * case["blocks"] + 2 * case["children"] + case["requests"]), flops=0)
    elem = 2 if case["dtype"] == "bf16" else 1
    cell = case["layers"] * case["hkv"] * case["dim"] * 2 * elem
    rest = case["layers"] * ((8 * case["hkv"] if elem == 1 else 0) + (132 * case["bs"] if case["index"] else 0))
    if case["op"] == "copy":
        return dict(bytes=2 * case["pairs"] * (cell * case["bs"] + rest + 4), flops=0)
    rows, lens, refs = _held(case)
    meta = 8 * (case["blocks"] + len(rows) * case["width"]) + 8 * len(rows)
    if case["op"] == "compact":
        count = len(refs)  # where they lie is the seed's: as many as on average
        moved = round(count * (1 - count / case["blocks"]))
        return dict(bytes=meta + 4 * case["blocks"] + 2 * moved * (cell * case["bs"] + rest), flops=0)
    refs = refs + [0] * (case["blocks"] - len(refs))
    *_, copied = _resize_host(rows, lens, _new_lens(case, lens), refs, case["bs"])
    return dict(bytes=meta + 2 * sum(c * cell + rest for _, _, c in copied), flops=0)


# ------------------------------------------------------------------ the definitions: 64 bits, and page by page


def _cells(cache, scale, blk, off):
    x = cache[blk, :, off]
    if scale is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * scale[blk].double()[..., None]


def _exact_attention(case, s):
    rows, hq, hkv, dim, bs = (case[x] for x in ("rows", "hq", "hkv", "dim", "bs"))
    out = torch.zeros((rows, hq, dim), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=DEV)
    q = s["q"].view(rows, hkv, hq // hkv, dim)
    cap = case["softcap"]

    def attend(i, e, k, v, see, dist):
        """Rows i to e on keys k, v [n, ...] (shared) or [rows, n, ...]."""
        each = "mnhd" if k.dim() == 4 else "nhd"
        sc = torch.einsum(f"mhgd,{each}->mhgn", q[i:e].double(), k) / math.sqrt(dim)
        if cap:
            sc = torch.tanh(sc / cap) * cap
        if dist is not None:
            sc = sc - dist[:, None, None] * s["slopes"].double().view(hkv, -1)[None, :, :, None]
        sc = sc.masked_fill(~see[:, None, None], -math.inf)
        l = torch.logsumexp(sc, -1)
        w = torch.exp(sc - l.masked_fill(l == -math.inf, 0.0)[..., None])
        out[i:e] = torch.einsum(f"mhgn,{each}->mhgd", w, v).reshape(e - i, hq, dim)
        lse[i:e] = l.reshape(e - i, hq)

    if case["kind"] == "sparse":
        for i in range(0, rows, 64):
            at = s["slots"][i:i + 64].long()
            see = at >= 0
            blk, off = at.clamp(min=0) // bs, at.clamp(min=0) % bs
            k, v = (_cells(c, z, blk, off).masked_fill(~see[..., None, None], 0.0)
                    for c, z in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            attend(i, i + at.shape[0], k, v, see, None)
        return dict(out=out, lse=lse)
    lens, starts, ends = _rows(case)
    row = 0
    for b, n in enumerate(_shape(case)[1]):
        tops = [max(lens[i], ends[i]) if lens[i] else 0 for i in range(row, row + n)]
        if max(tops):
            t = torch.arange(max(tops), device=DEV)
            blk, off = s["table"][b].long()[t // bs], t % bs
            k, v = _cells(s["kc"], s["ks"], blk, off), _cells(s["vc"], s["vs"], blk, off)
            step = max(1, (1 << 28) // (max(tops) * hq))
            for i in range(row, row + n, step):
                e = min(i + step, row + n)
                ln, lo, hi = (torch.tensor(x, device=DEV)[:, None] for x in (lens[i:e], starts[i:e], tops[i - row:e - row]))
                see = (t[None] >= lo) & (t[None] < hi)
                if case["window"]:
                    see &= (t[None] + case["window"] >= ln) | (t[None] - case["sinks"] < lo)
                attend(i, e, k, v, see, (t[None] + 1 - ln).abs().double() if case["slopes"] else None)
        row += n
    return dict(out=out, lse=lse)


def _resize_host(rows, lens, new, refs, bs):
    """Request by request: (rows, lengths, refs, copies (from, to, cells)) after the step; pages taken lowest first."""
    free = [p for p, r in enumerate(refs) if r <= 0]
    now, rows, lens, was = list(refs), [list(r) for r in rows], list(lens), list(lens)
    wants = {}  # growing requests of each shared last page
    for i, n in enumerate(was):
        if new[i] > n and n % bs and refs[rows[i][n // bs]] > 1:
            wants.setdefault(rows[i][n // bs], []).append(i)
    used, copied = 0, []
    for i, n in enumerate(was):
        have, want = -(-n // bs), -(-new[i] // bs)
        page = rows[i][n // bs] if n % bs else None
        sharers = wants.get(page, []) if new[i] > n else []
        keeps = bool(sharers) and len(sharers) == refs[page] and sharers[-1] == i
        copy = bool(sharers) and not keeps
        need = copy + max(0, want - have)
        if (need or keeps) and used + need > len(free):
            used += need
            continue
        got, used = free[used:used + need], used + need
        lens[i] = new[i]
        if copy:
            rows[i][n // bs] = got[0]
            copied.append((page, got[0], n % bs))
            now[page] -= 1
        for p in rows[i][want:have]:
            now[p] -= 1
        rows[i] = rows[i][:want] + got[copy:]
        for p in got:
            now[p] = 1
    return rows, lens, now, copied


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "fork":
        return None  # whole numbers alone
    if case["op"] == "copy":
        copied = [(a, b, case["bs"]) for a, b in zip(s["src"].tolist(), s["dst"].tolist())]
    else:
        lens, refs, bs = s["lens"].tolist(), s["refs"].tolist(), case["bs"]
        rows = [r[:-(-n // bs)] for r, n in zip(s["table"].tolist(), lens)]
        if case["op"] == "resize":
            *_, copied = _resize_host(rows, lens, s["new_lens"].tolist(), refs, bs)
        else:
            top = sum(r > 0 for r in refs)
            holes = iter([p for p in range(top) if refs[p] <= 0])
            copied = [(p, next(holes), bs) for p in range(top, len(refs)) if refs[p] > 0]
    f8 = torch.float8_e4m3fn
    out = dict(kv=(s["kv"] if case["dtype"] == "bf16" else s["kv"].view(f8)).double())
    if "scale" in s:
        out["scale"] = s["scale"].double()
    if "index_k" in s:
        out.update(index_k=s["index_k"].view(f8).double(), index_scale=s["index_scale"].double())
    for a, b, n in copied:
        if case["layout"] == "hnd":
            out["kv"][:, :, b, :, :n] = out["kv"][:, :, a, :, :n]
        else:
            out["kv"][:, :, b, :n] = out["kv"][:, :, a, :n]
        for name in ("index_k", "index_scale"):
            if name in out:
                out[name][:, b] = out[name][:, a]
        if "scale" in out:
            out["scale"][:, :, b] = out["scale"][:, :, a]
    return out

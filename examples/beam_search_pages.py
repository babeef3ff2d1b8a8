"""Beam search over one prompt on a paged cache: beams share pages, and pages are moved by the device alone.

    python examples/beam_search_pages.py [--cache bf16|e4m3] [--prompt 300] [--beams 4] [--steps 20] [--softcap 30]

The prompt is prefilled once for all beams. Every step the beams fork (``fork_pages``: a beam continues one of the old
ones, all its pages shared), get room for one token (``resize_pages``: a page that others hold too is copied first), the
token's keys and values are appended (``append_kv``), and the layer attends with capped scores and a bias by distance
(``paged_attention`` with ``softcap`` and ``slopes``). Every few steps the pool is compacted (``compact_pages``).
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_indexer_top_gb300 as sai  # noqa: E402

DEV = "cuda"


class Beams:
    def __init__(self, cache_type: str, beams: int, max_len: int, *, q_heads: int = 8, kv_heads: int = 2, dim: int = 64, bs: int = 16):
        blocks = -(-max_len // bs) * (beams + 1) + beams
        shape, f8 = (blocks, kv_heads, bs, dim), cache_type == "e4m3"
        zeros = lambda: torch.zeros(shape, dtype=torch.uint8 if f8 else torch.bfloat16, device=DEV)
        ones = lambda: (torch.ones((blocks, kv_heads), device=DEV),) if f8 else (None,)
        self.cache = sai.KVCache(zeros(), zeros(), *ones(), *ones())
        self.pages = sai.PageSet([self.cache])
        self.table = torch.full((beams, -(-max_len // bs)), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(beams, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(blocks, dtype=torch.int32, device=DEV)
        self.slopes = torch.exp2(-8.0 * torch.arange(1, q_heads + 1, device=DEV) / q_heads)
        self.q_heads, self.kv_heads, self.dim, self.bs, self.max_len = q_heads, kv_heads, dim, bs, max_len

    def tokens(self, rows: int):
        x = torch.randn((rows, self.q_heads + 2 * self.kv_heads, self.dim), device=DEV).to(torch.bfloat16)
        return x.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def grow(self, new_lens):
        self.table, self.lens, self.refs = sai.resize_pages(self.pages, self.table, self.lens, new_lens, self.refs)

    def fork(self, parents):
        self.table, self.lens, self.refs = sai.fork_pages(self.table, self.lens, self.refs, parents, block_size=self.bs)

    def compact(self):
        self.table, self.refs, _ = sai.compact_pages(self.pages, self.table, self.lens, self.refs)

    def prefill(self, n: int):
        """A prompt of n tokens for the first beam, which the others then continue."""
        new = torch.zeros_like(self.lens)
        new[0] = n
        self.grow(new)
        q, k, v = self.tokens(n)
        rows = torch.arange(1, n + 1, dtype=torch.int32, device=DEV)
        sai.append_kv(self.cache, k, v, self.table, rows, row_to_batch=torch.zeros_like(rows))
        self.fork(torch.zeros_like(self.lens))
        return k, v

    def step(self, parents, softcap: float):
        """One token for each beam; returns its queries, keys, values and outputs."""
        self.fork(parents)
        self.grow(self.lens + 1)
        q, k, v = self.tokens(parents.shape[0])
        sai.append_kv(self.cache, k, v, self.table, self.lens)
        out = sai.paged_attention(q, self.cache, self.table, self.lens, max_seq_len=self.max_len, softcap=softcap,
                                  slopes=self.slopes)
        return q, k, v, out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--softcap", type=float, default=30.0)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    beams = Beams(a.cache, a.beams, a.prompt + a.steps)
    history = [beams.prefill(a.prompt)]
    print(f"prompt: {a.prompt} tokens in {int((beams.refs > 0).sum())} pages for {a.beams} beams")
    for step in range(a.steps):
        parents = torch.randint(0, a.beams, (a.beams,), device=DEV, dtype=torch.int32)
        q, k, v, out = beams.step(parents, a.softcap)
        history.append((parents, q, k, v, out))
        if step % 8 == 7:
            beams.compact()
    held = int((beams.refs > 0).sum())
    print(f"{a.steps} steps: {held} pages held, {int((beams.refs > 1).sum())} of them by several beams, |out| {out.float().norm():.3f}")
    bits = sai.device_status()
    if bits:
        raise SystemExit(f"device status {bits}")
    return beams, history


if __name__ == "__main__":
    main()

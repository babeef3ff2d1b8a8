"""One layer's prefill chunk and a decode step behind the sparse-attention indexer, on random weights' outputs.

    python examples/sparse_layer_step.py [--cache bf16|e4m3] [--requests 3] [--prompt 3000] [--steps 4]

Prefill: the chunk's keys and values go into the paged cache, rotated on the way (``append_kv``), and all rows attend
densely in one packed call (``paged_attention``). Decode, step by step: the new token's keys and values are appended, the
indexer scores the paged index keys and picks 512 slots (``index_score_topk``), and the layer attends over them
(``sparse_attention``); a second, windowed layer on the same cache attends over its last tokens and the first few
(``paged_attention`` with ``window`` and ``sinks``). The slots come out as cells of the same blocks, since the
index cache and the key/value cache share one block table.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_indexer_top_gb300 as sai  # noqa: E402

DEV = "cuda"
BS, DIM, INDEX_HEADS = 128, 128, 64


def rotary_table(max_pos: int, dim: int) -> torch.Tensor:
    half = dim // 2
    freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * freq[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def index_keys(x: torch.Tensor):
    """e4m3 codes of index keys [n, 128] and their scales [n]."""
    scale = (x.float().abs().amax(1) / 448).clamp_min(1e-8)
    return (x.float() / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


class Layer:
    def __init__(self, cache_type: str, requests: int, max_len: int, q_heads: int = 16, kv_heads: int = 2):
        per = -(-max_len // BS)
        blocks = requests * per
        self.table = torch.randperm(blocks, device=DEV).to(torch.int32).view(requests, per)
        shape = (blocks, kv_heads, BS, DIM)
        if cache_type == "e4m3":
            self.cache = sai.KVCache(torch.zeros(shape, dtype=torch.uint8, device=DEV),
                                     torch.zeros(shape, dtype=torch.uint8, device=DEV),
                                     torch.ones((blocks, kv_heads), device=DEV), torch.ones((blocks, kv_heads), device=DEV))
        else:
            self.cache = sai.KVCache(torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                                     torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        self.index_k = torch.zeros((blocks, BS, DIM), dtype=torch.uint8, device=DEV)
        self.index_scale = torch.zeros((blocks, BS), device=DEV)
        self.cos_sin = rotary_table(max_len, DIM)
        self.q_heads, self.kv_heads, self.max_len = q_heads, kv_heads, max_len

    def qkv(self, rows: int):
        """Queries, keys and values as slices of one fused projection's output."""
        x = torch.randn((rows, (self.q_heads + 2 * self.kv_heads) * DIM), device=DEV).to(torch.bfloat16)
        q, k, v = x.split([self.q_heads * DIM, self.kv_heads * DIM, self.kv_heads * DIM], 1)
        return q.unflatten(1, (-1, DIM)), k.unflatten(1, (-1, DIM)), v.unflatten(1, (-1, DIM))

    def append(self, lens, row_to_batch=None):
        q, k, v = self.qkv(lens.shape[0])
        q = sai.append_kv(self.cache, k, v, self.table, lens, self.cos_sin, q=q, row_to_batch=row_to_batch)
        pos = lens.long() - 1
        b = torch.arange(lens.shape[0], device=DEV) if row_to_batch is None else row_to_batch.long()
        blk = self.table[b, pos // BS].long()
        codes, scale = index_keys(torch.randn((lens.shape[0], DIM), device=DEV))
        self.index_k[blk, pos % BS], self.index_scale[blk, pos % BS] = codes, scale
        return q

    def prefill(self, prompts):
        lens = torch.cat([torch.arange(1, n + 1) for n in prompts]).to(DEV, torch.int32)
        r2b = torch.repeat_interleave(torch.arange(len(prompts)), torch.tensor(prompts)).to(DEV, torch.int32)
        q = self.append(lens, r2b)
        return sai.paged_attention(q, self.cache, self.table, lens, max_seq_len=self.max_len, row_to_batch=r2b, packed=True)

    def decode(self, lens):
        """One token for each request, whose length now is lens."""
        q = self.append(lens)
        rows = lens.shape[0]
        iq = index_keys(torch.randn((rows * INDEX_HEADS, DIM), device=DEV))[0].view(rows, INDEX_HEADS, DIM)
        w = torch.rand((rows, INDEX_HEADS), device=DEV) / 8
        slots, _, _ = sai.index_score_topk(iq, w, self.index_k, self.index_scale, self.table, lens, max_seq_len=self.max_len)
        sparse = sai.sparse_attention(q, self.cache, slots)
        windowed = sai.paged_attention(q, self.cache, self.table, lens, max_seq_len=self.max_len, window=1024, sinks=4)
        return sparse, windowed, slots


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="e4m3")
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=3000)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    prompts = [max(1, a.prompt - 700 * i) for i in range(a.requests)]
    layer = Layer(a.cache, a.requests, max(prompts) + a.steps)
    out = layer.prefill(prompts)
    print(f"prefill: {sum(prompts)} rows of {a.requests} requests -> {list(out.shape)}")
    lens = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    for step in range(a.steps):
        lens = lens + 1
        sparse, windowed, slots = layer.decode(lens)
        picked = (slots >= 0).sum(1).tolist()
        print(f"decode {step}: lengths {lens.tolist()}, slots {picked}, |sparse| {sparse.float().norm():.3f}, "
              f"|windowed| {windowed.float().norm():.3f}")
    bits = sai.device_status()
    if bits:
        raise SystemExit(f"device status {bits}")
    return layer, out, sparse, windowed, slots


if __name__ == "__main__":
    main()

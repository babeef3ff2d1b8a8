"""The layer example runs, and its last decode step agrees with the oracle on the cache it left behind."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_sparse_layer_step(cache, monkeypatch):
    spec = importlib.util.spec_from_file_location("sparse_layer_step", os.path.join(ROOT, "examples", "sparse_layer_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    seen = {}
    real = ex.sai.sparse_attention

    def keep(q, cache, slots, **kw):
        seen["q"] = q
        return real(q, cache, slots, **kw)

    monkeypatch.setattr(ex.sai, "sparse_attention", keep)
    layer, out, sparse, windowed, slots = ex.main(["--cache", cache, "--prompt", "1500", "--steps", "2"])
    assert out.shape == (1500 + 800 + 100, 16, 128) and torch.isfinite(out.float()).all()
    c = layer.cache
    dec = (lambda x, s: x.float().double()) if cache == "bf16" else \
        (lambda x, s: x.view(torch.float8_e4m3fn).float().double() * s.double()[:, :, None, None])
    k, v = (dec(x, s).cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, c.heads, c.dim)
            for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    q = seen["q"].float().double().cpu().numpy()
    lens = [1502, 802, 102]
    for i, n in enumerate(lens):
        at = slots[i].cpu().numpy()
        at = at[at >= 0]
        assert len(at) == min(n, 512) and len(set(at.tolist())) == len(at)
        t = A.seen(n, 1024, 4)
        cells = layer.table[i].cpu().numpy()[t // 128] * 128 + t % 128
        for got, idx in ((sparse, at), (windowed, cells)):
            ref, _, mag = A.attend(q[i], k[idx], v[idx], c.dim ** -0.5)
            err = np.abs(got[i].float().cpu().double().numpy() - ref)
            # bf16 result and weights, 2^-9 each, doubled; fp32 scores of 128 products of size < 64
            assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_beam_search_pages(cache):
    """Every beam's output at every step is the attention over its own history of tokens, whatever pages it was in."""
    spec = importlib.util.spec_from_file_location("beam_search_pages", os.path.join(ROOT, "examples", "beam_search_pages.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    prompt, n, cap = 77, 5, 6.0
    beams, history = ex.main(["--cache", cache, "--prompt", str(prompt), "--beams", str(n), "--steps", "40", "--softcap", str(cap)])
    f = lambda x: x.float().cpu().double().numpy()
    past = [tuple(f(x) for x in history[0])] * n
    slopes = f(beams.slopes)
    for parents, q, k, v, out in history[1:]:
        q, k, v, out = (f(x) for x in (q, k, v, out))
        past = [tuple(np.concatenate([old, new[i:i + 1]]) for old, new in zip(past[p], (k, v))) for i, p in enumerate(parents.tolist())]
        for i in range(n):
            kk, vv = past[i]
            dist = np.arange(len(kk) - 1, -1, -1.0)
            ref, _, mag = A.attend_changed(q[i], kk, vv, beams.dim ** -0.5, cap, slopes, dist)
            # bf16: the result and the weights, 2^-9 each, doubled. e4m3: codes are off by 2^-4 of themselves at most
            # (below the least normal one by 2^-10 of a scale of |x| / 224 or less, which is less), twice where a
            # page's scale grew: values by 2^-3 of sum w|v|, scores by d = 2^-3 sum|q k| / 8, weights by 2 d of it
            if cache == "bf16":
                tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag
            else:
                d = np.array([np.abs(kk[:, a // 4]).dot(np.abs(q[i, a])).max() for a in range(8)])[:, None] * 2.0 ** -6
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -3 + 2.0 ** -6) * mag + np.expm1(2 * d) * (np.abs(ref) + mag)
            assert (np.abs(out[i] - ref) <= tol).all()
    # the counts are those of the table's holders
    held = torch.zeros_like(beams.refs)
    for row, length in zip(beams.table.tolist(), beams.lens.tolist()):
        for page in row[:-(-length // beams.bs)]:
            held[page] += 1
    assert torch.equal(held, beams.refs) and beams.lens.tolist() == [prompt + 40] * n

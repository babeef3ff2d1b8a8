"""Oracle of the paged cache and the attention over it (numpy, float64).

The definitions, one row at a time: rotation by position, the append with a
power-of-two scale for each block and head, and softmax attention over a
list of cells. No code is shared with the CUDA path.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_EXP = -64


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even), saturating at +-448; NaN stays."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), E4M3_MAX)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(mag)  # mag = m * 2**e, 0.5 <= m < 1
        step = np.exp2(np.maximum(e - 1, -6) - 3.0)
        return np.where(np.isnan(x), np.nan, np.copysign(np.rint(mag / step) * step, x))


def rotate(x: np.ndarray, pos: int, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [heads, dim] rotated by the position's angles."""
    y = np.array(x, np.float64)
    rot = cos_sin.shape[1]
    half = rot // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = float(cos_sin[pos, j]), float(cos_sin[pos, half + j])
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


def needed_scale(amax: float) -> float:
    """Least 2**e, e >= MIN_EXP, with amax <= 448 * 2**e."""
    e = MIN_EXP
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(values: np.ndarray, cache: np.ndarray, scale, places) -> None:
    """values [rows, heads, dim] into cache [blocks, heads, block_size, dim] in
    place (code values for an 8-bit cache, whose scale [blocks, heads] moves
    with it). places: (block, cell) of each row or None."""
    if scale is None:
        for x, at in zip(values, places):
            if at is not None:
                cache[at[0], :, at[1]] = x
        return
    groups = {}
    for i, at in enumerate(places):
        if at is not None:
            groups.setdefault(at[0], []).append((at[1], i))
    for blk, cells in groups.items():
        first = min(c for c, _ in cells)
        for h in range(values.shape[1]):
            new = np.stack([values[i, h] for _, i in cells])
            s = needed_scale(float(np.max(np.abs(new[np.isfinite(new)]), initial=0.0)))
            if first:
                s = max(s, float(scale[blk, h]))
                cache[blk, h, :first] = e4m3_round(cache[blk, h, :first] * (float(scale[blk, h]) / s))
            scale[blk, h] = s
            for (c, _), x in zip(cells, new):
                cache[blk, h, c] = e4m3_round(x / s)


def seen(n: int, window: int, sinks: int) -> np.ndarray:
    """Positions that a row of length n sees."""
    t = np.arange(n)
    return t[(t >= n - window) | (t < sinks)] if window else t


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, sm_scale: float):
    """q [q_heads, dim], k and v [n, heads, dim]: (out [q_heads, dim], lse
    [q_heads], weight [q_heads, dim]) with weight = sum_t w_t |v_t|, the size
    that rounding errors of the weights are measured against."""
    hq, dim = q.shape
    out, lse, mag = np.zeros((hq, dim)), np.full(hq, -np.inf), np.zeros((hq, dim))
    if len(k) == 0:
        return out, lse, mag
    group = hq // k.shape[1]
    for a in range(hq):
        s = k[:, a // group] @ q[a] * sm_scale
        m = s.max()
        w = np.exp(s - m)
        total = w.sum()
        out[a] = w @ v[:, a // group] / total
        mag[a] = w @ np.abs(v[:, a // group]) / total
        lse[a] = m + np.log(total)
    return out, lse, mag

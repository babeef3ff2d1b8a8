"""Pins of the cache and attention oracle (CPU): e4m3 rounding against torch's
conversion, scales against their inequality, the rotation's invariants, and
the attention against closed forms."""

import numpy as np
import torch

from oracle import attention as A


def test_e4m3_rounding_matches_torch():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(0, 1, 4000) * np.exp2(rng.integers(-14, 9, 4000)), np.arange(-448, 449, 0.5),
                        np.exp2(np.arange(-12.0, 9)), 3 * np.exp2(np.arange(-12.0, 7)), [0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(A.e4m3_round(x), ref.astype(np.float64))
    assert A.e4m3_round(np.array([np.inf, -1e9]))[0] == 448 and np.isnan(A.e4m3_round(np.array([np.nan]))[0])


def test_needed_scale_is_least():
    for amax in (1e-30, 1e-6, 0.5, 447.9, 448.0, 448.1, 896.0, 3e4):
        s = A.needed_scale(amax)
        assert amax <= 448 * s and (s == 2.0 ** A.MIN_EXP or amax > 448 * s / 2)
    assert A.needed_scale(0.0) == 2.0 ** A.MIN_EXP


def test_rotation_keeps_norms_and_relative_angles():
    rng = np.random.default_rng(2)
    half = 8
    ang = np.arange(40)[:, None] * (10000.0 ** (-np.arange(half) / half))[None]
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = rng.normal(size=(1, 16)), rng.normal(size=(1, 16))
    for inter in (False, True):
        dots = [float((A.rotate(q, p + 5, cs, inter) * A.rotate(k, p, cs, inter)).sum()) for p in (0, 3, 20)]
        assert np.allclose(dots, dots[0])
        assert np.isclose(np.linalg.norm(A.rotate(q, 7, cs, inter)), np.linalg.norm(q))
        assert np.array_equal(A.rotate(q, 0, cs, inter), q)


def test_append_grows_a_block_scale_and_keeps_its_values():
    cache, scale = np.zeros((1, 1, 16, 4)), np.zeros((1, 1))
    A.append(np.array([[[1.0, -2.0, 0.5, 448.0]]]), cache, scale, [(0, 0)])
    assert scale[0, 0] == 1.0
    A.append(np.array([[[896.0, 0, 0, 0]]]), cache, scale, [(0, 1)])
    assert scale[0, 0] == 2.0
    assert np.array_equal(cache[0, 0, 0] * 2, [1.0, -2.0, 0.5, 448.0])
    A.append(np.array([[[1.0, 0, 0, 0]]]), cache, scale, [(0, 0)])  # the block starts anew
    assert scale[0, 0] == 2.0 ** -8 and cache[0, 0, 0, 0] == 256


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    k, v = rng.normal(size=(7, 2, 4)), rng.normal(size=(7, 2, 4))
    out, lse, _ = A.attend(np.zeros((4, 4)), k, v, 1.0)
    assert np.allclose(out[:2], v[:, 0].mean(0)) and np.allclose(out[2:], v[:, 1].mean(0))
    assert np.allclose(lse, np.log(7))
    q = rng.normal(size=(4, 4))
    out, lse, _ = A.attend(q, k[:1], v[:1], 0.5)
    assert np.allclose(out[0], v[0, 0]) and np.isclose(lse[3], 0.5 * q[3] @ k[0, 1])
    out, lse, _ = A.attend(q, k[:0], v[:0], 0.5)
    assert (out == 0).all() and np.isneginf(lse).all()
    assert list(A.seen(6, 2, 1)) == [0, 4, 5] and list(A.seen(2, 5, 1)) == [0, 1] and list(A.seen(3, 0, 0)) == [0, 1, 2]

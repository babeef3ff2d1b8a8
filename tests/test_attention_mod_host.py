"""Host-side argument checks of the attention with changed scores and masks (CPU)."""

import ctypes

import numpy as np
import pytest

from oracle import attention as A
from test_attention_host import P, _desc, lib  # noqa: F401


def _mod(softcap=0.0, slopes=None, row_starts=None, prefix_lens=None):
    from sparse_attention_indexer_top_gb300._lib import ScoreMod

    return ScoreMod(softcap, slopes, row_starts, prefix_lens)


def _paged(lib, m, q=P):  # noqa: F811
    d = _desc()
    return lib.sai_paged_attention_mod(q, 8 * 128, 8, ctypes.addressof(d), P, 4, 8, None, P, 4, 1024, 0, 0, 0.1, 0,
                                       None if m is None else ctypes.addressof(m), P, None, None, 0, None)


def _sparse(lib, m, q=P):  # noqa: F811
    d = _desc()
    return lib.sai_sparse_attention_mod(q, 8 * 128, 8, ctypes.addressof(d), P, 512, 512, 4, 0.1,
                                        None if m is None else ctypes.addressof(m), P, None, None, 0, None)


@pytest.mark.parametrize("call", [_paged, _sparse])
def test_caps(lib, call):  # noqa: F811
    for cap in (-1.0, float("inf"), float("nan"), 1e-38, 1e35):
        assert call(lib, _mod(cap)) == -2
    # these get past the modifiers and stop at the missing queries
    for m in (None, _mod(), _mod(30.0), _mod(1e-30), _mod(1e30)):
        assert call(lib, m, q=None) == -1


def test_arrays(lib):  # noqa: F811
    for name in ("slopes", "row_starts", "prefix_lens"):
        assert _paged(lib, _mod(**{name: P + 2})) == -7
        assert _paged(lib, _mod(**{name: P}), q=None) == -1
        assert _sparse(lib, _mod(**{name: P})) == -3  # slots have no positions


def test_oracle_without_changes_is_the_plain_one():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(4, 64)), rng.normal(size=(50, 2, 64)), rng.normal(size=(50, 2, 64))
    for a, b in zip(A.attend(q, k, v, 0.1), A.attend_changed(q, k, v, 0.1)):
        assert np.array_equal(a, b)
    far = A.attend_changed(q, k, v, 0.1, softcap=1e9)
    assert np.allclose(A.attend(q, k, v, 0.1)[0], far[0], atol=1e-12)
    for n, w, s in ((0, 0, 0), (40, 0, 0), (40, 10, 3), (40, 50, 3)):
        assert np.array_equal(A.seen(n, w, s), A.span(n, w, s))
    assert A.span(5, 0, 0, 5).size == 0 and A.span(5, 0, 0, 9).size == 0
    assert A.span(5, 2, 1, 1, 8).tolist() == [1, 3, 4, 5, 6, 7]

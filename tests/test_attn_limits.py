"""The softmax-attention layers' reference, refusals and build at their limits, without a GPU."""
import numpy as np
import pytest

from oracle import attn as oa


def test_reference_window_counts_back_from_a_length_behind_the_table():
    """Eight rows of table, pages of 4: a length of 11 with a window of 5 sees tokens 6 and 7 of its 6 .. 10."""
    r = np.random.default_rng(2)
    kc, vc = r.standard_normal((2, 4, 1, 4)), r.standard_normal((2, 4, 1, 4))
    q, table = r.standard_normal((1, 1, 4)), np.array([[1, 0]])
    o, lse = oa.attn_decode(q, kc, vc, table, [11], window=5)
    s = kc[0, 2:4, 0] @ q[0, 0] / 2.0
    assert np.allclose(o[0, 0], np.exp(s) @ vc[0, 2:4, 0] / np.exp(s).sum()) and np.isclose(lse[0, 0], np.log(np.exp(s).sum()))
    for told, window in ((13, 5), (2 ** 31 - 1, 7)):  # the whole window lies behind
        o, lse = oa.attn_decode(q, kc, vc, table, [told], window=window)
        assert (o == 0).all() and np.isneginf(lse).all()
    o, _ = oa.attn_decode(q, kc, vc, table, [12], window=5)
    assert np.allclose(o[0, 0], vc[0, 3, 0])
    assert np.array_equal(oa.attn_decode(q, kc, vc, table, [99])[0], oa.attn_decode(q, kc, vc, table, [8])[0])

"""CPU: the attention oracle on rows whose scores are not finite."""
import numpy as np

import oracle as O


def test_a_row_that_sees_a_nan_is_nan_and_one_that_sees_nothing_is_zero():
    r = np.random.default_rng(3)
    q, k, v = (r.standard_normal((6, 1, 4)) for _ in range(3))
    k[2] = np.nan
    out, spread, _ = O.viewed_attention(q, k, v, np.arange(6) - 1, 0.5, left=0, right=0)
    assert not out[0].any() and np.isnan(out[3]).all() and np.isnan(spread[3]).all()
    assert np.array_equal(out[[1, 2, 4, 5]], v[[0, 1, 3, 4]])
    k[2] = 0.0
    k[2, 0, 1] = np.inf
    q[:, 0, 1] = [1, -1, 1, -1, 1, -1]
    with np.errstate(invalid="ignore"):
        out, _, _ = O.viewed_attention(q, k, v, np.arange(6), 0.5)
        assert np.isnan(out[0::2]).all()
        ref, _, _ = O.viewed_attention(q[1::2], np.delete(k, 2, 0), np.delete(v, 2, 0), np.arange(3), 0.5)
        assert np.allclose(out[1::2], ref, rtol=1e-12)
        out, _, _ = O.viewed_attention(q, k, v, np.arange(6), 0.5, cap=3.0)
    assert np.isfinite(out).all()

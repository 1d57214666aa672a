"""GPU: capped scores of the packed attention where the cap's arithmetic can go wrong: caps at the ends of their range, scores
at the ends of the polynomial's, tiles that mix both."""
import numpy as np
import pytest

from test_gpu_attention_views import b, check, engines, np64, packed_reference, rows, run_packed, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def against_reference(engines, dt, q, k, v, lens, view, D):  # noqa: F811
    T = sum(lens)
    out = run_packed(engines[dt], q, k, v, lens, view, D)
    b.sf_check(engines[dt])
    ref, spread, big = packed_reference(np64(q[:T]), np64(k[:T]), np64(v[:T]), lens, dict(view, cap=float(np.float32(view["cap"]))), D,
                                        q.shape[1])
    check(np64(out[:T]), ref, spread, big, "packed", dt, D, view, 0)
    return out


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [50.0, 1e3, 1e5, 1e8])
@pytest.mark.parametrize("view", [{}, dict(right=0)])
def test_a_large_score_beside_small_ones(engines, dt, cap, view):  # noqa: F811
    """Rows behind the sequence that are far beyond the cap, and one row of large scores in the sequence: the other rows,
    which share tiles with them, keep the accuracy of their small scores."""
    H, KV, D, n = 4, 2, 64, 232
    q, k, v = (rows(230 + i, n + 30, h, D, dt) for i, h in enumerate((H, KV, KV)))
    k[n:] *= 3e4 * cap
    q[100] *= 0.5 * cap
    against_reference(engines, dt, q, k, v, [n], dict(view, cap=cap), D)

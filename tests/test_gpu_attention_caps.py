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


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap,scale", [(1e-6, 0.125), (1e-6, 1e3), (1e-5, 1.0), (1e-4, 10.0), (1e-3, 0.125), (1e6, 1e-6)])
@pytest.mark.parametrize("which", ["q", "k"])
def test_zeros_under_every_cap(engines, dt, cap, scale, which):  # noqa: F811
    """Silence: queries or keys of zeros have scores of zero, and every row the mean of its values."""
    H, D, n = 2, 64, 150
    q, k, v = (rows(240 + i, n, H, D, dt) for i in range(3))
    (q if which == "q" else k).zero_()
    out = torch.full_like(q, 7.0)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    b.sf_attention_packed(engines[dt], q, k, v, cu, out, b.attn_params(H, H, D, cap=cap, scale=scale))
    b.sf_check(engines[dt])
    # equal weights are 1 before their rounding, so exact; fp32 sums of n values, one division, one rounding
    mean, size = np64(v).mean(0), np.abs(np64(v)).mean(0)
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    assert (np.abs(np64(out) - mean) <= half * np.abs(mean) + (n + 3) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [64.0, 2e3, 1e4, 1e5])
def test_equal_scores_of_different_tiles_under_large_caps(engines, dt, cap):  # noqa: F811
    """Scores of 0.7 cap in a tile that lies in the polynomial's range and in one that does not (its last score is -0.9
    cap) are the same score: the mean of their values."""
    H, D, n = 2, 64, 128
    q, k, v = (torch.zeros(n, H, D, device="cuda", dtype=rows(0, 1, 1, D, dt).dtype) for _ in range(3))
    q[:, :, 0] = 8.0
    k[:, :, 0] = 0.7 * cap
    k[n - 1, :, 0] = -0.9 * cap
    v[:64], v[64:] = 1.0, -1.0
    against_reference(engines, dt, q, k, v, [n], dict(cap=cap), D)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [1e-5, 0.02, 30.0, 700.0, 3e4])
@pytest.mark.parametrize("view", [{}, dict(right=3), dict(left=50, right=70)])
def test_scores_around_the_end_of_the_polynomial(engines, dt, cap, view):  # noqa: F811
    """Scores spread over 0 .. 1.5 caps in either sign."""
    H, D, n = 2, 64, 333
    g = torch.Generator(device="cuda").manual_seed(250)
    q, k, v = rows(251, n, H, D, dt, 1e-3 * min(cap, 1.0)), rows(252, n, H, D, dt, 1e-3 * min(cap, 1.0)), rows(253, n, H, D, dt)
    q[:, :, 0] = torch.rand(n, H, generator=g, device="cuda") * 12 * cap ** 0.5
    k[:, :, 0] = (torch.rand(n, H, generator=g, device="cuda") * 2 - 1) * cap ** 0.5
    against_reference(engines, dt, q, k, v, [n], dict(view, cap=cap), D)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [20.0, 53.0, 60.0, 64.0])
def test_scores_far_below_zero(engines, dt, cap):  # noqa: F811
    """A tile of scores of -0.73 cap, then thousands further down: their small weights add up and are not lost."""
    H, D, n = 1, 64, 4096
    q, k, v = (torch.zeros(n, H, D, device="cuda", dtype=rows(0, 1, 1, D, dt).dtype) for _ in range(3))
    q[:, :, 0] = 8.0
    k[:64, :, 0], k[64:, :, 0] = -0.73 * cap, -cap
    v[:64], v[64:] = 1.0, -1.0
    against_reference(engines, dt, q, k, v, [n], dict(cap=cap), D)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [20.0, 50.0, 64.0, 300.0])
@pytest.mark.parametrize("lift", [False, True])
def test_small_values_under_scores_far_below_zero(engines, dt, cap, lift):  # noqa: F811
    """Values of 1e-18 under scores of -0.7 cap (lift: but for one in each tile): their products with the weights stay in
    range.  The results are rounded from 2^-100 and more: relative to them as ever."""
    H, D, n = 2, 64, 256
    q, k, v = (rows(260 + i, n, H, D, dt, 1e-2 if i < 2 else 1.0) for i in range(3))
    q[:, :, 0] = 8.0
    k[:, :, 0] = -0.7 * cap
    if lift:
        k[5::64, :, 0] = -0.6 * cap
    out = run_packed(engines[dt], q, k, (v.float() * 1e-18).to(v.dtype), [n], dict(cap=cap), D)
    b.sf_check(engines[dt])
    v = np64((v.float() * 1e-18).to(v.dtype)) * 1e18
    ref, spread, big = packed_reference(np64(q), np64(k), v, [n], dict(cap=cap), D, H)
    check(np64(out) * 1e18, ref, spread, big, "packed", dt, D, cap, 0)

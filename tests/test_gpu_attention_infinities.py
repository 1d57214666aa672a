"""GPU: infinite queries and keys in the limited-view attention, by the scores they make."""
import numpy as np
import pytest

import oracle as O
from test_gpu_attention_views import (b, cached_reference, check, engines, make_cache, make_table, np64,  # noqa: F401
                                      rows, run_cached, run_packed, torch)

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0, 500.0, 1e5])
@pytest.mark.parametrize("view", [{}, dict(right=0), dict(left=40, right=12)])
@pytest.mark.parametrize("which", ["query", "key", "both"])
def test_packed(engines, dt, D, cap, view, which):  # noqa: F811
    """An infinite element of a query or of a key makes scores of +inf and -inf: NaN rows, weights of 0 and, under a cap, scores
    of cap and -cap.  Rows that do not see it are what they are without it."""
    H, n = 2, 200
    q, k, v = (rows(270 + i, n, H, D, dt) for i in range(3))
    _, _, big = O.viewed_attention(np64(q), np64(k), np64(v), np.arange(n), D ** -0.5, cap, view.get("left", -1), view.get("right", -1))
    if which != "key":
        q[70, 0, 5] = INF
    if which != "query":
        k[90, :, 7] = -INF
    with np.errstate(invalid="ignore"):
        ref, spread, _ = O.viewed_attention(np64(q), np64(k), np64(v), np.arange(n), float(np.float32(D ** -0.5)), cap,
                                            view.get("left", -1), view.get("right", -1))
    out = np64(run_packed(engines[dt], q, k, v, [n], dict(view, cap=cap), D))
    b.sf_check(engines[dt])
    lost = np.isnan(ref).all(-1)
    assert (np.isnan(ref).any(-1) == lost).all() and (np.isnan(out).all(-1) == lost).all() and np.isfinite(out[~lost]).all()
    if cap == 0.0 and which == "key":
        assert lost.any() and not lost.all()
    zero = np.where(lost[..., None], 0.0, 1.0)
    check(np.nan_to_num(out) * zero, np.nan_to_num(ref) * zero, np.nan_to_num(spread) * zero, np.maximum(big, cap), "packed", dt, D, view, 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_packed_row_of_minus_infinity(engines, dt, cap):  # noqa: F811
    """Every score of a row -inf: zeros, and the mean of the values under a cap."""
    H, D, n = 1, 64, 130
    q, k, v = (rows(280 + i, n, H, D, dt).abs() for i in range(3))
    q[3, 0, 9] = -INF
    out = np64(run_packed(engines[dt], q, k, v, [n], dict(cap=cap), D))[3, 0]
    mean = np64(v)[:, 0].mean(0)
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    # equal weights of one size: half a step in each weight (1 before a rescaling), the sums, the result
    assert (np.abs(out - (mean if cap else 0.0)) <= (2 * half * mean + (n + 8) * 2.0 ** -24 * mean if cap else 0.0)).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
def test_cached_query(engines, dt, cap, D):  # noqa: F811
    """A row whose query is infinite or NaN is NaN in that head; the rows beside it in its tile are not touched."""
    H, KV, page, held, new = 4, 2, 16, 100, 7
    table, pages = make_table(285, [held], page)
    cache = make_cache(286, pages, KV, page, D)
    q = rows(287, new, H, D, dt)
    q[2, 1, 3], q[5, 2, 60], q[6, 0, 0] = INF, -INF, float("nan")
    out = np64(run_cached(engines[dt], q, cache, table, [held], [new], dict(cap=cap, right=0), D))
    b.sf_check(engines[dt])
    lost = np.zeros((new, H), bool)
    lost[2, 1] = lost[5, 2] = lost[6, 0] = True
    assert np.isnan(out[lost]).all() and np.isfinite(out[~lost]).all()
    fine = torch.nan_to_num(q, nan=0.0, posinf=0.0, neginf=0.0)
    ref, spread, big = cached_reference(np64(fine), cache, table, [held], [new], dict(cap=cap, right=0), D, H)
    out[lost], ref[lost] = 0.0, 0.0
    check(out, ref, spread, big, "cached", dt, D, cap, 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 64), (128, 16), (128, 32)])
@pytest.mark.parametrize("view", [dict(right=0), dict(left=40, right=0), dict(left=9, right=5, prefix=[20]), {}])
@pytest.mark.parametrize("which", ["k", "v"])
def test_cached_nan_codes(engines, dt, D, page, view, which):  # noqa: F811
    """NaN codes among a sequence's cached rows (a caller's: sf_kv_append writes none): the rows that see them are NaN in that
    head, at least in that dim of a value; the others are what they are without them."""
    H, KV, held, new = 4, 2, 150, 23
    table, pages = make_table(288, [held], page)
    cache = make_cache(289, pages, KV, page, D)
    q = rows(290, new, H, D, dt)
    spots = [(5, 0, 3), (70, 1, 60), (131, 0, 17), (140, 0, 18), (149, 1, 40)]
    codes = getattr(cache, which).view(torch.uint8)
    for j, g, d in spots:
        codes[table[0, j // page], g, j % page, d] = 0
    ref, spread, big = cached_reference(np64(q), cache, table, [held], [new], view, D, H)
    for n, (j, g, d) in enumerate(spots):
        codes[table[0, j // page], g, j % page, d] = 0x7f if n % 2 else 0xff
    out = np64(run_cached(engines[dt], q, cache, table, [held], [new], view, D))
    b.sf_check(engines[dt])
    i = np.arange(held - new, held)
    pre, left, right = view.get("prefix", [0])[0], view.get("left", -1), view.get("right", -1)
    lost = np.zeros((new, H), bool)
    for j, g, d in spots:
        sees = (j < pre) | (((left < 0) | (i - j <= left)) & ((right < 0) | (j - i <= right)))
        lost[np.ix_(sees, range(2 * g, 2 * g + 2))] = True
        assert np.isnan(out[sees][:, 2 * g:2 * g + 2, d] if which == "v" else out[sees][:, 2 * g:2 * g + 2]).all()
    assert np.isfinite(out[~lost]).all()
    if view.get("left", -1) >= 0:
        assert lost.any() and not lost.all()
    out[lost], ref[lost] = 0.0, 0.0
    check(out, ref, spread, big, "cached", dt, D, view, 0)

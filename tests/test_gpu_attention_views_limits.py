"""GPU: the limited-view attention at the ends of its documented ranges."""
import numpy as np
import pytest

from test_gpu_attention_views import (b, cached_reference, check, dev, engines, make_cache, make_table, np64,  # noqa: F401
                                      packed_reference, rows, run_cached, run_packed, torch)

pytestmark = pytest.mark.gpu


def test_one_sequence_of_more_rows_than_tiles_of_16_count(engines):  # noqa: F811
    """2^25 + 128 rows x heads in one sequence, in 8-row tiles (fp32, heads of 128): every row is written.  All but the
    last 64 new rows come out before position 0."""
    H, KV, D, page, held = 8, 1, 128, 64, 64
    T = 2 ** 22 + 16
    table, pages = make_table(210, [held], page)
    cache = make_cache(211, pages, KV, page, D)
    q, out = (torch.zeros(T, H, D, device="cuda") for _ in range(2))
    q[-held:] = rows(212, held, H, D, "f32")
    out.fill_(7.0)
    run_cached(engines["f32"], q, cache, table, [held], [T], dict(right=0), D, out=out)
    b.sf_check(engines["f32"])
    assert not out[:-held].any()
    ref, spread, big = cached_reference(np64(q[-held:]), cache, table, [held], [held], dict(right=0), D, H)
    check(np64(out[-held:]), ref, spread, big, "cached", "f32", D, "limits", 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cu", [[0, 200, 100, 300], [0, 90, 80, 300], [0, 200, 200, 190]])
def test_offsets_out_of_order_are_reported(engines, dt, cu):  # noqa: F811
    """Offsets that fall back, also where the sequence between them owns no slot: SF_EDEVICE, then all is well."""
    KV, D, page, T, eng = 2, 64, 16, 300, engines[dt]
    x, p = rows(220, T, KV, D, dt), b.attn_params(KV, KV, D)
    cache, held = make_cache(221, 60, KV, page, D), dev([300, 300, 300])
    table = dev(np.arange(60).reshape(3, 20))
    calls = [lambda at: b.sf_attention_packed(eng, x, x, x, at, torch.empty_like(x), p),
             lambda at: b.sf_kv_append(eng, x, x, at, held, table, cache),
             lambda at: b.sf_attention_cached(eng, x, at, held, table, cache, torch.empty_like(x), p)]
    for call in calls:
        call(dev(cu))
        with pytest.raises(b.SFError, match="SF_EDEVICE"):
            b.sf_check(eng)
        call(dev(sorted(cu)))
        b.sf_check(eng)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scales_and_caps_at_the_ends_of_fp32(engines, dt):  # noqa: F811
    """Scales and caps whose products leave fp32's normal range are refused; those just inside give finite results."""
    eng, D, n = engines[dt], 64, 70
    x, cu = rows(225, n, 2, D, dt), dev([0, n])
    cache, held, table = make_cache(226, 5, 2, 16, D), dev([n]), dev([[0, 1, 2, 3, 4]])
    for kw in (dict(scale=1e-39), dict(scale=2e30), dict(scale=-1.0), dict(cap=3e38), dict(cap=1.1e30), dict(cap=1e30, scale=1e-9),
               dict(scale=float("nan")), dict(cap=float("inf"))):
        p = b.attn_params(2, 2, D, **kw)
        for call in (lambda: b.sf_attention_packed(eng, x, x, x, cu, torch.empty_like(x), p),
                     lambda: b.sf_attention_cached(eng, x, cu, held, table, cache, torch.empty_like(x), p)):
            with pytest.raises(b.SFError, match="SF_EINVAL"):
                call()
    for kw in (dict(scale=1.2e-38), dict(cap=1e30, scale=2e-8), dict(cap=1e30), dict(cap=1e-6, scale=1e30)):
        p, out = b.attn_params(2, 2, D, **kw), [torch.empty_like(x) for _ in range(2)]
        b.sf_attention_packed(eng, x, x, x, cu, out[0], p)
        b.sf_attention_cached(eng, x, cu, held, table, cache, out[1], p)
        assert all(torch.isfinite(o).all() for o in out)
    b.sf_check(eng)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("scales", [(2.0 ** -70, 2.0 ** -70), (2.0 ** -75, 2.0 ** -62), (2.0 ** -62, 2.0 ** -75), (2.0 ** -90, 0.0),
                                    (0.0, 0.0), (2.0 ** -100, 1.0), (1.0, 2.0 ** -100), (2.0 ** 24, 2.0 ** -100), (2.0 ** 24, 0.0),
                                    (0.0, 2.0 ** 24), (2.0 ** 60, 2.0 ** -20), (2.0 ** 110, 2.0 ** 90)])
def test_values_of_every_size(engines, dt, page, scales):  # noqa: F811
    """Value scales far below and above 1.  Under 2^-60 the weights in the outputs carry the rest: they are off by half a step
    of fp16's least, 2^-25, beside a largest weight of 2^14 or more, so by 2^-39 of 448 x 2^-60 for each key."""
    H, KV, D, held = 4, 2, 64, 2 * page
    cache, table = make_cache(227, 2, KV, page, D), np.array([[1, 0]])
    cache.v_scale[1], cache.v_scale[0] = scales
    q = rows(228, 9, H, D, dt)
    out = np64(run_cached(engines[dt], q, cache, table, [held], [9], {}, D))
    b.sf_check(engines[dt])
    ref, spread, big = cached_reference(np64(q), cache, table, [held], [9], {}, D, H)
    unit = max(max(scales), 2.0 ** -60)   # compared in units that the bound's own floor does not reach
    low = held * 448 * 2.0 ** -39 * 2.0 ** -60 / unit
    half = 2.0 ** -11 if dt == "bf16" else 2.0 ** -22
    check(out / unit, ref / unit, spread / unit + low / half, big, "cached", dt, D, scales, 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H", [([1], 2), ([63], 2), ([200, 321], 8), ([1500], 2), ([2309], 2), ([322] * 40, 16)])
@pytest.mark.parametrize("view", [{}, dict(right=0), dict(left=60, right=3, prefix=[130] * 40)])
def test_what_lies_behind_a_sequence_changes_no_bit(engines, dt, D, lens, H, view):  # noqa: F811
    """Keys and values behind the last sequence, and a sequence's neighbour's, that are not finite: the results of zeros there,
    to the bit (a row computed again from its own keys alone would differ in its roundings, and cost a hundred times as much)."""
    T = sum(lens)
    q, k, v = (rows(290 + i, T + 70, H, D, dt) for i in range(3))
    outs = []
    for x in (0.0, float("nan"), float("inf")):
        for t in (k, v):
            t[T:] = x
        if len(lens) > 2:
            for t in (k, v):
                t[lens[0]:2 * lens[0]] = x   # the second sequence
        outs.append(run_packed(engines[dt], q, k, v, lens, view, D))
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    if len(lens) > 2:
        keep[lens[0]:2 * lens[0]] = False
    assert all(torch.equal(o[:T][keep], outs[0][:T][keep]) for o in outs[1:]) and torch.isfinite(outs[0][:T]).all()
    b.sf_check(engines[dt])

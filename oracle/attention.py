"""Attention with capped, biased and limited scores, and the 8-bit paged
key/value cache: the formulas of sf.h's sf_attention_packed, sf_kv_append and
sf_attention_cached, one sequence at a time in float64.

    s(i, j)    = scale q_i . k_j, then cap tanh(s / cap) where cap > 0,
                 then s - slope_head |i - j|
    seen(i, j) = (i - left <= j <= i + right) or j < prefix      (-1: no limit)
    out_i      = sum over seen j of softmax_j(s(i, .)) v_j, zeros where none is

e4m3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits, largest 448,
smallest step 2^-9 ("FP8 Formats for Deep Learning", E4M3)."""
import numpy as np

E4M3_MAX = 448.0


def viewed_attention(q, k, v, pos_q, scale, cap=0.0, left=-1, right=-1, prefix=0, slopes=None):
    """q [n, H, D] at positions pos_q, k and v [L, KV, D] at 0 .. L - 1.

    Returns (out [n, H, D], spread [n, H, D], s_err [n, H]) where spread is
    sum_j p_j |v_j| (what a relative error of the weights scales) and s_err a
    bound's ingredient: the largest sum_d |q_d k_d| scale over seen keys."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, D = q.shape
    L, KV, _ = k.shape
    j = np.arange(L)[None]
    i = np.asarray(pos_q)[:, None]
    seen = np.ones((n, L), bool)
    if left >= 0:
        seen &= j >= i - left
    if right >= 0:
        seen &= j <= i + right
    seen |= j < prefix
    seen &= i >= 0
    out, spread, big = np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros((n, H))
    for h in range(H):
        kk, vv = k[:, h // (H // KV)], v[:, h // (H // KV)]
        s = scale * (q[:, h] @ kk.T)
        if cap > 0:
            s = cap * np.tanh(s / cap)
        if slopes is not None:
            s = s - float(slopes[h]) * np.abs(i - j)
        s = np.where(seen, s, -np.inf)
        m = s.max(axis=1, keepdims=True, initial=-np.inf)
        p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        t = p.sum(axis=1, keepdims=True)
        p = np.divide(p, t, out=np.zeros_like(p), where=t != 0)   # (a NaN sum stays one)
        out[:, h], spread[:, h] = p @ vv, p @ np.abs(vv)
        big[:, h] = np.where(seen, scale * (np.abs(q[:, h]) @ np.abs(kk).T), 0.0).max(axis=1, initial=0.0)
    return out, spread, big


def e4m3_round(x):
    """The nearest e4m3 value, ties to the even mantissa, saturating."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.abs(x))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.round(x / step) * step, -E4M3_MAX, E4M3_MAX)


def kv_append(codes, scales, rows, first, table, page):
    """One sequence's new rows [n, KV, D] at positions first .. into codes
    [pages, KV, page, D] (as values) and scales [pages, KV], in place.  The
    quotients and scales are rounded to float32 as the formula's are."""
    f = np.float32
    n = len(rows)
    t = first
    while t < first + n:
        p, off = int(table[t // page]), t % page
        m = min(page - off, first + n - t)
        new = np.asarray(rows[t - first:t - first + m], f).transpose(1, 0, 2)
        had = scales[p].astype(f) if off else np.zeros(new.shape[0], f)
        now = np.maximum(had, np.abs(new).max(axis=(1, 2)) / f(E4M3_MAX))
        by = np.where(now > 0, now, f(1))[:, None, None]
        if off:
            moved = e4m3_round(codes[p, :, :off].astype(f) * (had[:, None, None] / by))
            codes[p, :, :off] = np.where((now > had)[:, None, None], moved, codes[p, :, :off])
        codes[p, :, off:off + m] = e4m3_round(new / by)
        scales[p] = now
        t += m

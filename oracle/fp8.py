"""Scored routing and the block-scaled FP8 (OCP E4M3) operators, in float64 (test
infrastructure; see the package docstring).

E4M3 is decoded from its bit fields; a value is rounded to it by looking up the two
neighbouring values of the format's table.  Every step follows the definition in
include/moe_mxfp4.h (moe_route_scored) and include/moe_fp8.h."""
from __future__ import annotations

import numpy as np

__all__ = ["E4M3", "decode_e4m3", "round_e4m3", "quantize_fp8", "expand_rows", "expand_weights",
           "gemm_fp8", "route_scored", "ffn_fp8"]

BLOCK = 128
# The FP8 matrix instruction cuts each product of a group of 16 at 2^-13 of the power of two of
# the group's largest (which is exact): at most this share of the sum of magnitudes.
MFMA_CUT = 15 * 2.0 ** -13


def _table() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 0x7F) == 0x7F else sign * mag
    return v


E4M3 = _table()


def decode_e4m3(codes) -> np.ndarray:
    return E4M3[np.asarray(codes, np.uint8)]


def round_e4m3(v) -> np.ndarray:
    """Codes of the nearest E4M3 values, ties to the even code; magnitudes are at most 448."""
    v = np.asarray(v, np.float64)
    mag = np.abs(v)
    grid = E4M3[:0x7F]                                   # 0 .. 448, ascending
    hi = np.clip(np.searchsorted(grid, mag), 1, 0x7E)
    lo = hi - 1
    below, above = mag - grid[lo], grid[hi] - mag
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def quantize_fp8(x):
    """Codes uint8 [rows, K] and scales float32 [rows, ceil(K/128)] of x [rows, K]; the quotient
    448 x / a is taken in float64 (its 11-bit by 8-bit numerators and denominators, for bf16 x,
    make a quotient off a border differ from it by far more than float64's rounding)."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    nb = -(-K // BLOCK)
    codes, scale = np.empty((rows, K), np.uint8), np.empty((rows, nb), np.float32)
    for b in range(nb):
        cut = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        part = x[:, cut]
        ok = np.isfinite(part).all(1)
        a = np.maximum(np.where(ok, np.abs(np.where(np.isfinite(part), part, 0)).max(1), 1.0), 2.0 ** -100)
        q = round_e4m3(np.where(ok[:, None], part, 0.0) * 448.0 / a[:, None])
        codes[:, cut] = np.where(ok[:, None], q, 0x7F)
        scale[:, b] = np.where(ok, (a / 448.0).astype(np.float32), np.float32(np.nan))
    return codes, scale


def expand_rows(scale, K) -> np.ndarray:
    return np.repeat(np.asarray(scale, np.float64), BLOCK, axis=1)[:, :K]


def expand_weights(scale, n, K) -> np.ndarray:
    return expand_rows(np.repeat(np.asarray(scale, np.float64), BLOCK, axis=0)[:n], K)


def gemm_fp8(xq, xs, w, ws):
    """(y, sum of magnitudes) in float64: the second bounds what rounding the sums can do."""
    K = xq.shape[1]
    x = decode_e4m3(xq) * expand_rows(xs, K)
    m = decode_e4m3(w) * expand_weights(ws, w.shape[0], K)
    return x @ m.T, np.abs(x) @ np.abs(m).T


def route_scored(logits, k, *, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2,
                 renormalize=True, scale=1.0):
    """ids int32 [T, k] and weights float64 [T, k], token by token."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    per = E // groups
    ids, weights = np.empty((T, k), np.int32), np.empty((T, k))
    for t in range(T):
        live = l[t] > -np.inf                            # not -inf, not NaN
        s = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[live] = 1.0 / (1.0 + np.exp(-l[t][live]))
        elif live.any():
            m = l[t][live].max()
            with np.errstate(invalid="ignore"):
                z = np.where(l[t][live] == m, 1.0, np.exp(l[t][live] - m))
            s[live] = z / z.sum()
        # without a bias, experts are ordered by their logits
        key = np.where(live, l[t] if bias is None else s + b, -np.inf)
        def group_key(g):
            of = [e for e in range(g * per, (g + 1) * per) if live[e]]
            if not of:
                return -np.inf
            if group_top == 1:
                return max(key[e] for e in of)
            best = sorted(of, key=lambda e: (-key[e], e))[:2]
            return sum((s[e] + b[e]) for e in best)
        order = sorted(range(groups), key=lambda g: (-group_key(g), g))[:topk_groups] if groups > 1 else [0]
        pool = [e for g in order for e in range(g * per, (g + 1) * per)]
        chosen = sorted(pool, key=lambda e: (-key[e], e))[:k]
        w = s[chosen]
        if renormalize:
            if score == "softmax" and live[chosen].any():   # the same ratio, without underflow
                top = l[t][chosen][live[chosen]].max()
                with np.errstate(invalid="ignore"):
                    w = np.where(live[chosen], np.where(l[t][chosen] == top, 1.0, np.exp(l[t][chosen] - top)), 0.0)
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        ids[t], weights[t] = chosen, w * scale
    return ids, weights


def _h_of(g, u, limit):
    if limit is not None and np.isfinite(limit) and limit > 0:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def ffn_fp8(x, gather, offsets, k, w1, w1s, w2, w2s, limit):
    """(y, slack) float64 [T*k, H]: y by the definition, and how far fp32 arithmetic may move it.

    Slack.  u = 2^-24.  A product's sum of n runs is off by at most (n + 130) 2u + MFMA_CUT times
    the sum of its terms' magnitudes (128 products within a run, n scaled sums, and the cut).  SiLU(g) u has slopes at
    most 1.1 |u| in g and |SiLU(g)| in u, and the fp32 exponential and reciprocal add 2^-20 of
    it.  An element of h whose quotient may cross a border of E4M3 moves by one step; its run's
    scale moves relatively as far as the largest of the run does.  Rounding y to bf16 is not in it.
    """
    u24 = 2.0 ** -24
    E, I, H = w1.shape[0], w1.shape[1] // 2, w1.shape[2]
    xq, xs = quantize_fp8(x)
    slots = gather.size
    y, slack = np.zeros((slots, H)), np.zeros((slots, H))
    for e in range(E):
        p = slice(int(offsets[e]), int(offsets[e + 1]))
        if p.start == p.stop:
            continue
        rows = gather[p] // k
        gu, mag = gemm_fp8(xq[rows], xs[rows], w1[e], w1s[e])
        off = ((H // BLOCK + 130) * 2 * u24 + MFMA_CUT) * mag
        g, up = gu[:, :I], gu[:, I:]
        h = _h_of(g, up, limit)
        lim = limit if limit and limit > 0 and np.isfinite(limit) else np.inf
        silu = np.abs(_h_of(g, np.ones_like(g), limit if np.isfinite(lim) else None))
        dh = 1.1 * np.minimum(np.abs(up), lim) * off[:, :I] + silu * off[:, I:] + 2.0 ** -20 * np.abs(h)
        hq, hs = quantize_fp8(h)
        step = np.zeros_like(h)
        rel = np.zeros_like(h)
        for b in range(I // BLOCK):
            cut = slice(b * BLOCK, (b + 1) * BLOCK)
            a = np.maximum(np.abs(h[:, cut]).max(1, keepdims=True), 2.0 ** -100)
            da = dh[:, cut].max(1, keepdims=True) / a + 4 * u24
            z = np.abs(h[:, cut]) * 448.0 / a
            dz = dh[:, cut] * 448.0 / a + z * (da + 4 * u24)
            lo, hi = round_e4m3(np.maximum(z - dz, 0.0)), round_e4m3(np.minimum(z + dz, 448.0))
            step[:, cut] = E4M3[hi] - E4M3[lo]
            rel[:, cut] = da
        hd = decode_e4m3(hq) * expand_rows(hs, I)
        moved = step * expand_rows(hs, I) + rel * np.abs(hd)
        m2 = decode_e4m3(w2[e]) * expand_weights(w2s[e], H, I)
        y[p] = hd @ m2.T
        slack[p] = moved @ np.abs(m2).T + ((I // BLOCK + 130) * 2 * u24 + MFMA_CUT) * (np.abs(hd) @ np.abs(m2).T)
    return y, slack

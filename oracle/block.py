"""The operators around the routed layer in float64 (numpy): RMS norm and its gradient, the balance
loss and its gradient, low-rank adapters.  Written from their definitions; test infrastructure."""
from __future__ import annotations

import numpy as np


def round_bf16(v):
    """Nearest bf16 value of a float64 array, ties to even (infinities and NaN stay)."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(np.where(np.isfinite(v), v, 0.0))
    step = np.ldexp(1.0, np.maximum(ex - 8, -133))
    r = np.where(np.isfinite(v), np.round(np.where(np.isfinite(v), v, 0.0) / step) * step, v)
    return np.where(np.abs(r) > 3.3895313892515355e38, np.copysign(np.inf, r), r)


def rms_norm(x, residual, w, eps):
    """(s, y) in float64; s is rounded to bf16 where there is a residual."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = round_bf16(s + residual)
    with np.errstate(all="ignore"):
        y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * w
    return s, y


def rms_norm_grad(s, w, eps, dy, dsum=None):
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    r = 1.0 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    u, z = s * r, dy * w
    dx = r * (z - u * np.mean(z * u, axis=1, keepdims=True))
    return dx if dsum is None else dx + dsum, np.sum(dy * u, axis=0)


def shares(logits, score):
    """p [T, E]: the scores divided by their sum; 0 for excluded experts (-inf, NaN)."""
    l = np.asarray(logits, np.float64)
    out = ~(l > -np.inf)
    a = np.where(out, -np.inf, l)
    if score == "sigmoid":
        with np.errstate(all="ignore"):
            a = np.where(out, -np.inf, -np.logaddexp(0.0, -np.where(out, 0.0, a)))
    m = a.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        e = np.where(out, 0.0, np.where(a == m, 1.0, np.exp(a - m)))
        t = e.sum(axis=1, keepdims=True)
        return np.where(t > 0, e / np.where(t > 0, t, 1.0), 0.0)


def sequences(T, seq_offsets):
    return [(0, T)] if seq_offsets is None else list(zip(seq_offsets[:-1], seq_offsets[1:]))


def balance_loss(logits, ids, score, seq_offsets=None):
    T, E = logits.shape
    k = ids.shape[1]
    p = shares(logits, score)
    loss, counts = [], []
    for t0, t1 in sequences(T, seq_offsets):
        flat = ids[t0:t1].reshape(-1)
        c = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        n = t1 - t0
        counts.append(c)
        loss.append(float(E / (k * n) * (c * p[t0:t1].mean(axis=0)).sum()) if n else 0.0)
    return np.array(loss), np.array(counts, np.int32)


def balance_loss_grad(logits, k, counts, dloss, score, seq_offsets=None, add_to=None):
    T, E = logits.shape
    p = shares(logits, score)
    d = np.zeros((T, E)) if add_to is None else np.array(add_to, np.float64)
    with np.errstate(all="ignore"):
        slope = np.where(logits > -np.inf, 1.0 / (1.0 + np.exp(np.asarray(logits, np.float64))), 0.0)
    for s, (t0, t1) in enumerate(sequences(T, seq_offsets)):
        n = t1 - t0
        if n == 0:
            continue
        c, q = counts[s].astype(np.float64), p[t0:t1]
        c = c - c.mean() * (q.sum(axis=1, keepdims=True) > 0)   # sum p = 1: the same difference
        g = float(dloss[s]) * E / (k * n * n) * q * (c - (q * c).sum(axis=1, keepdims=True))
        d[t0:t1] += g * slope[t0:t1] if score == "sigmoid" else g
    return d


def lora_group(ids, L):
    ids = np.asarray(ids)
    key = np.where((ids >= 0) & (ids < L), ids, L)
    rows = np.argsort(key, kind="stable")
    return np.r_[0, np.cumsum(np.bincount(key, minlength=L + 1)[:L])].astype(np.int32), rows.astype(np.int32)


def lora_add(x, a, b, scaling, ids, base):
    """y in float64, and a bound's ingredients: sum_r |B| |v| and sum_r |B| sum_i |x A|, scaled."""
    M, N = x.shape[0], b.shape[1]
    y = np.zeros((M, N)) if base is None else np.array(base, np.float64)
    split, inner = np.zeros((M, N)), np.zeros((M, N))
    for l in range(a.shape[0]):
        at = np.nonzero(np.asarray(ids) == l)[0]
        if at.size == 0:
            continue
        s = 1.0 if scaling is None else float(scaling[l])
        v = x[at] @ a[l].T
        y[at] += s * (v @ b[l].T)
        split[at] = abs(s) * (np.abs(v) @ np.abs(b[l]).T)
        inner[at] = abs(s) * ((np.abs(x[at]) @ np.abs(a[l]).T) @ np.abs(b[l]).T)
    return y, split, inner

"""Pins of the float64 oracle of the operators around the routed layer: closed forms, brute force
on tiny inputs, and gradients against differences."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import block


def rng(seed=0):
    return np.random.default_rng(seed)


def test_round_bf16_keeps_eight_bits_and_goes_to_even():
    v = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -30, -3.0, 2.0 ** -133, 2.0 ** -134,
                  3 * 2.0 ** -134, 3.4e38, np.inf])
    want = [1.0, 1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -3.0, 2.0 ** -133, 0.0, 2.0 ** -132, np.inf, np.inf]
    assert np.array_equal(block.round_bf16(v), want)


def test_norm_of_a_constant_row_is_its_weight():
    w = rng().normal(size=24)
    s, y = block.rms_norm(np.full((3, 24), -2.5), None, w, 0.0)
    assert np.allclose(y, -w, rtol=1e-15)
    s, y = block.rms_norm(np.full((1, 24), 3.0), np.full((1, 24), -3.0), w, 1e-6)
    assert not s.any() and not y.any()


def test_norm_does_not_change_with_its_row_scale():
    x, w = rng(1).normal(size=(4, 40)), rng(2).normal(size=40)
    a, b = block.rms_norm(x, None, w, 0.0)[1], block.rms_norm(64.0 * x, None, w, 0.0)[1]
    assert np.allclose(a, b, rtol=1e-14)


@pytest.mark.parametrize("beside", [False, True])
def test_norm_gradient_against_differences(beside):
    r = rng(3)
    s, w, dy = r.normal(size=(3, 16)), r.normal(size=16), r.normal(size=(3, 16))
    dsum = r.normal(size=(3, 16)) if beside else None

    def f(s, w):
        return (block.rms_norm(s, None, w, 0.1)[1] * dy).sum() + (0.0 if dsum is None else (s * dsum).sum())

    dx, dw = block.rms_norm_grad(s, w, 0.1, dy, dsum)
    h = 1e-6
    for i, j in ((0, 0), (1, 7), (2, 15)):
        e = np.zeros_like(s)
        e[i, j] = h
        assert abs((f(s + e, w) - f(s - e, w)) / (2 * h) - dx[i, j]) < 1e-8
    for j in (0, 9):
        e = np.zeros_like(w)
        e[j] = h
        assert abs((f(s, w + e) - f(s, w - e)) / (2 * h) - dw[j]) < 1e-8


def test_even_load_costs_one_and_has_no_gradient():
    T, E, k = 12, 6, 2
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    l = rng(4).normal(size=(T, E))
    for score in ("softmax", "sigmoid"):
        loss, counts = block.balance_loss(l, ids, score)
        assert np.array_equal(counts, [[4] * 6]) and abs(loss[0] - 1.0) < 1e-14
        assert np.abs(block.balance_loss_grad(l, k, counts, [1.0], score)).max() < 1e-16


def test_all_on_one_expert_costs_e_times_its_share():
    l = rng(5).normal(size=(5, 4))
    loss, _ = block.balance_loss(l, np.full((5, 1), 2), "softmax")
    p = np.exp(l) / np.exp(l).sum(1, keepdims=True)
    assert abs(loss[0] - 4 * p[:, 2].mean()) < 1e-14


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    r = rng(6)
    T, E, k, offsets = 11, 7, 3, [0, 4, 4, 9]
    l, ids, dloss = r.normal(size=(T, E)), r.integers(0, E, size=(T, k)), np.array([0.5, 2.0, -1.0])
    add = r.normal(size=(T, E))
    counts = block.balance_loss(l, ids, score, offsets)[1]
    g = block.balance_loss_grad(l, k, counts, dloss, score, offsets, add)

    def f(l):
        return (block.balance_loss(l, ids, score, offsets)[0] * dloss).sum() + (l * add).sum()

    for i, j in ((0, 0), (3, 6), (8, 2), (10, 1)):
        e = np.zeros_like(l)
        e[i, j] = 1e-6
        assert abs((f(l + e) - f(l - e)) / 2e-6 - g[i, j]) < 1e-8
    assert np.array_equal(g[9:], add[9:])


def test_excluded_experts_and_extreme_logits():
    l = np.array([[-np.inf, 1.0, 1.0], [np.nan, -np.inf, -np.inf], [-1000.0, -1001.0, -2000.0], [np.inf, 0.0, np.inf]])
    for score in ("softmax", "sigmoid"):
        p = block.shares(l, score)
        assert np.allclose(p[0], [0, 0.5, 0.5]) and not p[1].any()
        assert np.allclose(p[2], [1 / (1 + np.exp(-1)), 1 - 1 / (1 + np.exp(-1)), 0])
    assert np.allclose(block.shares(l, "softmax")[3], [0.5, 0, 0.5])
    assert np.allclose(block.shares(l, "sigmoid")[3], [0.4, 0.2, 0.4])


def test_lora_group_and_add_by_brute_force():
    r = rng(7)
    ids = np.array([2, -1, 0, 2, 5, 0, 1, -7])
    offsets, rows = block.lora_group(ids, 3)
    assert np.array_equal(offsets, [0, 2, 3, 5]) and np.array_equal(rows, [2, 5, 6, 0, 3, 1, 4, 7])
    x, a, b = r.normal(size=(8, 5)), r.normal(size=(3, 2, 5)), r.normal(size=(3, 4, 2))
    base, scaling = r.normal(size=(8, 4)), np.array([0.5, 1.0, 2.0])
    y = block.lora_add(x, a, b, scaling, ids, base)[0]
    for m in range(8):
        want = base[m].copy()
        if 0 <= ids[m] < 3:
            for n in range(4):
                want[n] += scaling[ids[m]] * sum(b[ids[m], n, q] * sum(x[m, i] * a[ids[m], q, i] for i in range(5))
                                                 for q in range(2))
        assert np.allclose(y[m], want, rtol=1e-13)

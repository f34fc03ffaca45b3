"""Pins of the float64 oracle of the FP8 operators and scored routing (CPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8


def test_decode_matches_the_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(fp8.E4M3, t.astype(np.float64), equal_nan=True)
    assert fp8.E4M3[0x7E] == 448.0 and np.isnan(fp8.E4M3[[0x7F, 0xFF]]).all()


def test_rounding_is_nearest_even():
    rng = np.random.default_rng(0)
    v = np.concatenate([fp8.E4M3[:0x7F], (fp8.E4M3[:0x7E] + fp8.E4M3[1:0x7F]) / 2,
                        rng.uniform(0, 448, 4000), rng.uniform(0, 0.05, 4000)]).astype(np.float32)
    v = np.concatenate([v, -v])
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.round_e4m3(v), ref)


def test_quantize_definition():
    x = np.zeros((3, 144))
    x[0, 3], x[0, 7] = -7.0, 3.5
    x[1, 140] = np.inf
    q, s = fp8.quantize_fp8(x)
    assert s[0, 0] == np.float32(7 / 448) and fp8.E4M3[q[0, 3]] == -448 and fp8.E4M3[q[0, 7]] == 224
    assert (q[2] == 0).all() and s[2, 0] == np.float32(2.0 ** -100 / 448)
    assert np.isnan(s[1, 1]) and (q[1, 128:] == 0x7F).all() and s[1, 0] == s[2, 0]


@pytest.mark.parametrize("renormalize", [True, False])
def test_scored_softmax_without_bias_is_plain_routing(renormalize):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((50, 24)).astype(np.float32)
    l[:, 5] = l[:, 9]                                    # ties
    ids, w = fp8.route_scored(l, 4, renormalize=renormalize)
    ref_ids, ref_w = oracle.route(l, 4)
    assert np.array_equal(ids, ref_ids)
    if renormalize:
        assert np.allclose(w, ref_w, rtol=1e-6)
    else:
        p = np.exp(l.astype(np.float64))
        p /= p.sum(1, keepdims=True)
        assert np.allclose(w, np.take_along_axis(p, ids, 1), rtol=1e-12)


def test_scored_groups_and_bias_by_hand():
    l = np.array([[0.0, 1.0, 3.0, -9.0, 2.0, 2.0]])
    s = 1 / (1 + np.exp(-l[0]))
    # groups {0,1} {2,3} {4,5}: sums of two: .5+.73, .95+~0, .88+.88 -> groups 2 and 0
    ids, w = fp8.route_scored(l, 3, score="sigmoid", groups=3, topk_groups=2, group_top=2, scale=2.0)
    assert ids.tolist() == [[4, 5, 1]] and np.allclose(w[0], 2 * s[[4, 5, 1]] / s[[4, 5, 1]].sum())
    ids, _ = fp8.route_scored(l, 2, score="sigmoid", groups=3, topk_groups=1, group_top=1)
    assert ids.tolist() == [[2, 3]]
    bias = np.array([0, 0, -1, 0, 0, 0.5])
    ids, w = fp8.route_scored(l, 2, score="sigmoid", bias=bias, renormalize=False)
    assert ids.tolist() == [[5, 4]] and np.allclose(w[0], s[[5, 4]])


def test_scored_excluded_experts():
    inf, nan = np.inf, np.nan
    l = np.array([[-inf, 1.0, nan, 0.5], [-inf, -inf, nan, -inf], [inf, 0.0, inf, 1.0]])
    for bias in (None, np.array([5.0, 0, 5.0, 0])):
        ids, w = fp8.route_scored(l[:2], 3, bias=bias)
        assert ids.tolist() == [[1, 3, 0], [0, 1, 2]]
        assert np.allclose(w[0], [1 / (1 + np.exp(-.5)), 1 - 1 / (1 + np.exp(-.5)), 0]) and (w[1] == 0).all()
    ids, w = fp8.route_scored(l[2:], 3, renormalize=False)
    assert ids.tolist() == [[0, 2, 3]] and w.tolist() == [[0.5, 0.5, 0.0]]


def test_ffn_bounds_catch_a_wrong_scale_and_a_dropped_run():
    rng = np.random.default_rng(2)
    T, E, k, H, I = 9, 3, 2, 256, 256
    x = torch.from_numpy(rng.standard_normal((T, H))).bfloat16().float().numpy()
    ids = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :k]
    _, offsets, gather, _ = oracle.expert_offsets(ids, E)
    w1 = rng.integers(0, 0x7F, (E, 2 * I, H)).astype(np.uint8) | (rng.integers(0, 2, (E, 2 * I, H)) * 128).astype(np.uint8)
    w2 = rng.integers(0, 0x7F, (E, H, I)).astype(np.uint8) | (rng.integers(0, 2, (E, H, I)) * 128).astype(np.uint8)
    w1s = (rng.uniform(0.5, 1.5, (E, 2 * I // 128, H // 128)) / 2000).astype(np.float32)
    w2s = (rng.uniform(0.5, 1.5, (E, H // 128, I // 128)) / 2000).astype(np.float32)
    y, slack = fp8.ffn_fp8(x, gather, offsets, k, w1, w1s, w2, w2s, 10.0)
    assert (slack < 0.3 * np.abs(y).max()).all()
    # a wrong block scale or a dropped run is far outside the 2-norm bound of the GPU tests
    y2, _ = fp8.ffn_fp8(x, gather, offsets, k, w1, w1s[:, :, ::-1].copy(), w2, w2s, 10.0)
    assert np.linalg.norm(y - y2) > 4 * 2.0 ** -7 * np.linalg.norm(y)
    w2[:, :, 240:] = 0
    y3, _ = fp8.ffn_fp8(x, gather, offsets, k, w1, w1s, w2, w2s, 10.0)
    assert np.linalg.norm(y - y3) > 4 * 2.0 ** -7 * np.linalg.norm(y)

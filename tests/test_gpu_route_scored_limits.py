"""Scored routing where fp32 arithmetic runs out, on the GPU against the float64 oracle: group
keys whose two terms cancel, and scores below fp32's range.  Ids equal, weights within 2^-20
relative (fp32 exponential and quotient: 14 u at most, u = 2^-24, and one rounding)."""
from __future__ import annotations

import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_routed_expert_route_amd import binding
    binding.load()


def check(logits, k, bias=None, **how):
    from mxfp4_routed_expert_route_amd import binding
    print(f"[route_scored limits] {logits.shape} k={k} {how} bias={bias is not None}", file=sys.stderr, flush=True)
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    binding.moe_route_scored(torch.from_numpy(logits).cuda(), k, ids, w,
                             bias=None if bias is None else torch.from_numpy(bias).cuda(), **how)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    ref_ids, ref_w = fp8.route_scored(logits, k, bias=bias, **how)
    wrong = (ids != ref_ids).any(1)
    assert not wrong.any(), (int(wrong.sum()), np.argwhere(wrong)[:5].ravel().tolist())
    assert (np.abs(w - ref_w) <= 2.0 ** -20 * np.abs(ref_w) + 1e-38).all()


def close_pairs(rng, T, score, spread):
    """Logits [T, 4] of two groups of two experts whose sums of scores lie 1e-7 to `spread` apart."""
    gap = np.exp(rng.uniform(np.log(1e-7), np.log(spread), T)) * rng.choice([-1, 1], T)
    if score == "softmax":
        a, r, q = (1 + gap) / 2, rng.uniform(0.1, 0.9, T), rng.uniform(0.1, 0.9, T)
        p = np.stack([a * r, a * (1 - r), (1 - a) * q, (1 - a) * (1 - q)], 1)
        return np.log(p).astype(np.float32)
    s = np.stack([rng.uniform(0.3, 0.7, T) for _ in range(3)], 1)
    last = s[:, 0] + s[:, 1] + gap * 0.2 - s[:, 2]
    s = np.concatenate([s, np.clip(last, 0.02, 0.98)[:, None]], 1)
    return np.log(s / (1 - s)).astype(np.float32)


# ------------------------------------------------------------ group keys that cancel

def test_group_sums_of_opposite_biases_by_hand():
    # scores 0.370160 + 0.541073 against 0.481108 + 0.430145: in fp32, with the biases, the other way round
    logits = np.array([[-0.53151953, 0.1646726, -0.07560388, -0.2812635]], np.float32)
    check(logits, 2, np.array([1000, -1000, 1000, -1000], np.float32), score="sigmoid", groups=2, topk_groups=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [4.0, 64.0, 1000.0, 3e4, 1e7])
def test_group_sums_of_opposite_biases(score, size):
    rng = np.random.default_rng(int(size))
    logits = close_pairs(rng, 600, score, min(0.3, size * 2.0 ** -23))
    bias = np.array([size, -size, size, -size], np.float32)
    for k in (1, 2):
        check(logits, k, bias, score=score, groups=2, topk_groups=1, group_top=2)
    # the same pairs as groups of three, the third expert never among a group's two largest
    three = np.insert(logits, [2, 4], -30.0, axis=1)
    check(three, 2, np.insert(bias, [2, 4], -2 * size).astype(np.float32), score=score, groups=2, topk_groups=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("keep", [1, 2, 3])
def test_a_group_of_large_keys_among_small_ones(score, keep):
    # the group whose sum fp32 does not resolve is not the one at the border
    rng = np.random.default_rng(keep)
    logits = rng.standard_normal((500, 8)).astype(np.float32)
    for at in (0, 1, 3):
        bias = np.zeros(8, np.float32)
        bias[2 * at:2 * at + 2] = 1e7, -1e7
        check(logits, 2, bias, score=score, groups=4, topk_groups=keep, group_top=2)


def test_group_sums_past_the_range_of_fp32():
    logits = np.zeros((3, 6), np.float32)
    bias = np.array([3.0e38, 3.0e38, 3.2e38, 3.0e38, -3.1e38, -3.1e38], np.float32)
    for keep in (1, 2):
        check(logits, 2, bias, score="sigmoid", groups=3, topk_groups=keep, group_top=2)
    check(logits, 2, -bias, score="sigmoid", groups=3, topk_groups=2, group_top=2)


# ------------------------------------------------------------ scores below the range of fp32

@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 8, 2)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_sigmoid_scores_below_fp32(groups, keep, top, renormalize):
    rng = np.random.default_rng(groups)
    at = np.array([-59, -61, -70, -86, -88, -100, -103, -120, -170, -226, -230, -241, -242, -250, -300, -500, -700], np.float32)
    logits = (at[:, None] + rng.permutation(16)[None] * 0.5).astype(np.float32)
    # a large score among small ones: quotients of scores that fp32 holds as denormals or not at all
    wide = rng.uniform(-200, -40, (60, 16)).astype(np.float32)
    bias = (rng.standard_normal(16) * 0.1).astype(np.float32)
    for l in (logits, wide):
        for k in (1, 4):
            check(l, k, score="sigmoid", groups=groups, topk_groups=keep, group_top=top, renormalize=renormalize)
    check(logits[5:], 4, bias, score="sigmoid", groups=groups, topk_groups=keep, group_top=top,
          renormalize=renormalize, scale=2.5)

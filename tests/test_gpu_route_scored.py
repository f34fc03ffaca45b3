"""Scored routing on the GPU against the float64 oracle: ids equal, weights within 2^-20
relative (fp32 exponential and quotient: 14 u at most, u = 2^-24, and one rounding)."""
from __future__ import annotations

import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mxfp4_routed_expert_route_amd import binding
    binding.load()


def gpu_route(logits, k, **how):
    from mxfp4_routed_expert_route_amd import binding
    T = logits.shape[0]
    bias = how.pop("bias", None)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    binding.moe_route_scored(logits, k, ids, w, bias=None if bias is None else torch.from_numpy(bias).cuda(), **how)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


def check(logits, k, **how):
    """logits: a CPU tensor, fp32 or bf16."""
    print(f"[route_scored] {tuple(logits.shape)} {logits.dtype} k={k} "
          f"{ {n: v for n, v in how.items() if n != 'bias'} } bias={how.get('bias') is not None}", file=sys.stderr, flush=True)
    ids, w = gpu_route(logits.cuda(), k, **how)
    ref_ids, ref_w = fp8.route_scored(logits.float().numpy(), k, **how)
    assert np.array_equal(ids, ref_ids), np.argwhere(ids != ref_ids)[:5]
    assert (np.abs(w - ref_w) <= 2.0 ** -20 * np.abs(ref_w) + 1e-38).all()


SHAPES = [   # T, E, k, groups, topk_groups
    (1, 1, 1, 1, 1), (1, 8, 8, 1, 1), (3, 256, 6, 8, 4), (64, 256, 6, 1, 1), (65, 64, 8, 4, 2), (200, 256, 8, 8, 3),
    (33, 38, 7, 2, 1), (50, 99, 3, 33, 5), (50, 300, 6, 3, 2), (20, 1000, 8, 1, 1), (20, 1024, 8, 8, 2),
    (40, 64, 4, 64, 9), (16, 640, 5, 5, 5), (30, 1023, 8, 33, 7), (7, 512, 1, 64, 1), (9, 130, 2, 13, 1),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_matches_the_oracle(shape, score, with_bias):
    T, E, k, groups, topk_groups = shape
    rng = np.random.default_rng(T * 1009 + E * 7 + k)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32) * 2)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
    for n, (top, renorm, scale, dtype) in enumerate([(1, True, 1.0, torch.float32), (2, False, 2.5, torch.float32),
                                                     (2, True, 2.5, torch.bfloat16)]):
        check(logits.to(dtype), k, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_top=top,
              renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_keys_that_fp32_cannot_tell_apart(score, groups):
    # biases that lift every expert's key to nearly the same value: fp32 keys collide, and the
    # order is decided in 64 bits (gaps of about 1e-8, against fp64's 1e-16)
    rng = np.random.default_rng(5)
    E, T = 64, 60
    l = rng.standard_normal((1, E)).astype(np.float32)
    s = 1 / (1 + np.exp(-l[0].astype(np.float64))) if score == "sigmoid" else np.exp(l[0].astype(np.float64)) / np.exp(l[0].astype(np.float64)).sum()
    bias = (1.0 - s).astype(np.float32)
    logits = np.repeat(l, T, 0)
    logits[1:] += (rng.standard_normal((T - 1, 1)) * 1e-6).astype(np.float32)
    check(torch.from_numpy(logits), 8, score=score, bias=bias, groups=groups, topk_groups=max(1, groups // 2))


def test_equal_keys_go_to_the_lower_index():
    l = torch.zeros(5, 96)
    l[1] = -3.0
    l[2, ::2] = 1.0
    l[3, 50:] = 2.0
    l[4] = torch.tensor([0.0, -0.0]).repeat(48)
    for bias in (None, np.zeros(96, np.float32)):
        for groups, keep in ((1, 1), (6, 2), (48, 10)):
            for score in ("softmax", "sigmoid"):
                check(l, 6, score=score, bias=bias, groups=groups, topk_groups=keep)


def test_excluded_and_extreme_logits():
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rng = np.random.default_rng(9)
    l = torch.from_numpy(rng.standard_normal((14, 32)).astype(np.float32))
    l[0] = -inf
    l[1] = nan
    l[2] = low
    l[3, 1:] = -inf
    l[4, ::3] = nan
    l[5, 8:] = low
    l[6, 5] = inf
    l[7, [3, 20]] = inf
    l[8] = 80.0 + 0.1 * torch.arange(32)
    l[9] = -80.0 - 0.1 * torch.arange(32)
    l[10, 16:] = -inf
    l[11] = torch.linspace(-200, 200, 32)
    l[12, :30] = -inf
    l[13] = 3e38
    bias = (rng.standard_normal(32) * 0.1).astype(np.float32)
    for b in (None, bias):
        for score in ("softmax", "sigmoid"):
            for groups, keep, top in ((1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 3, 2)):
                for renorm in (True, False):
                    rows = list(range(14))
                    if score == "sigmoid" and (b is not None or groups > 1 and top == 2):
                        rows.remove(8)   # saturated scores: their order is not resolved by 64 bits
                        rows.remove(11)
                        rows.remove(9)
                    if score == "softmax" and (b is not None or groups > 1 and top == 2):
                        rows.remove(11)   # scores below 1e-16 of the bias
                    check(l[rows], 6, score=score, bias=b, groups=groups, topk_groups=keep, group_top=top,
                          renormalize=renorm)


def test_nan_bias_leaves_ids_valid_and_distinct():
    bias = np.full(40, np.nan, np.float32)
    bias[3] = -np.float32(np.nan)
    ids, w = gpu_route(torch.randn(9, 40, device="cuda"), 8, score="sigmoid", bias=bias)
    assert all(sorted(set(r)) == sorted(r) and min(r) >= 0 and max(r) < 40 for r in ids.tolist())


@pytest.mark.parametrize("T,E,k,groups", [(0, 16, 2, 1), (1, 256, 6, 8), (64, 256, 8, 8), (65, 256, 6, 4), (64, 1024, 8, 1),
                                          (700, 96, 5, 3), (1300, 256, 6, 1), (12, 1023, 8, 33), (60, 512, 8, 1)])
def test_and_group_equals_the_separate_calls(T, E, k, groups):
    from mxfp4_routed_expert_route_amd import binding, layer
    rng = np.random.default_rng(T + E)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    bias = torch.from_numpy((rng.standard_normal(E) * 0.1).astype(np.float32)).cuda()
    how = dict(score="sigmoid", bias=bias, groups=groups, topk_groups=(groups + 1) // 2, group_top=2, scale=1.5)
    a, b = (layer.LayerBuffers.allocate(T, E, k, 128, 128) for _ in range(2))
    names = ("topk_ids", "topk_weights", "bitmatrix", "counts", "offsets", "gather", "scatter")
    for buf in (a, b):
        for n in names:
            getattr(buf, n).view(torch.int32).fill_(-3)
    binding.moe_route_scored(logits, k, a.topk_ids, a.topk_weights, **how)
    binding.moe_build_bitmatrix(a.topk_ids, E, a.bitmatrix)
    binding.moe_expert_offsets(a.bitmatrix, a.topk_ids, E, a.counts, a.offsets, a.gather, a.scatter, a.ws)
    binding.moe_route_scored_and_group(logits, k, b.topk_ids, b.topk_weights, b.bitmatrix, b.counts, b.offsets,
                                       b.gather, b.scatter, b.ws, **how)
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(getattr(a, n).view(torch.int32), getattr(b, n).view(torch.int32)), n
    if T:
        counts, offsets, gather, scatter = oracle.expert_offsets(b.topk_ids.cpu().numpy(), E)
        assert np.array_equal(b.gather.cpu().numpy(), gather) and np.array_equal(b.counts.cpu().numpy(), counts)
    else:
        assert (b.counts == 0).all() and (b.offsets == 0).all()


def test_more_tokens_than_one_launch_takes():
    # 2^22 tokens go into a launch; the tokens' experts repeat with period 7
    from mxfp4_routed_expert_route_amd import binding, layer
    T, E, k = (1 << 22) + 3, 7, 2
    print(f"[route_scored] T={T}", file=sys.stderr, flush=True)
    rows = torch.tensor([[1.0 if (t + 1) % 7 == e else 2.0 if t == e else -e for e in range(7)] for t in range(7)])
    logits = rows.bfloat16().repeat(T // 7 + 1, 1)[:T].cuda().contiguous()
    t7 = (torch.arange(T, device="cuda") % 7).int()
    want = torch.stack([t7, (t7 + 1) % 7], 1).int()
    b = layer.LayerBuffers.allocate(T, E, k, 128, 128)
    binding.moe_route_scored_and_group(logits, k, b.topk_ids, b.topk_weights, b.bitmatrix, b.counts, b.offsets,
                                       b.gather, b.scatter, b.ws, renormalize=True)
    torch.cuda.synchronize()
    assert torch.equal(b.topk_ids, want)
    bits = (1 << want.long()).sum(1)
    assert torch.equal(b.bitmatrix.view(torch.int32).view(T, -1)[:, 0].long(), bits)
    assert torch.equal(b.counts.long(), torch.bincount(want.flatten().long(), minlength=E))
    p = 1 / (1 + np.exp(-1.0))
    assert (b.topk_weights.double() - torch.tensor([p, 1 - p], dtype=torch.float64, device="cuda")).abs().max() < 1e-6


@pytest.mark.parametrize("T,E,k,groups", [(1, 256, 6, 8), (16, 64, 4, 1), (64, 32, 6, 4), (200, 16, 3, 4), (600, 16, 2, 1)])
def test_scored_routing_in_front_of_the_mxfp4_experts(T, E, k, groups):
    """Scored routing in moe_route's place: the MXFP4 FFN and the combine take its outputs."""
    from mxfp4_routed_expert_route_amd import binding, layer
    from tests.test_gpu_parity import ffn_close, tiny
    H, I = 256, 128
    print(f"[route_scored] mxfp4 T={T} E={E} k={k} groups={groups}", file=sys.stderr, flush=True)
    inp = tiny(T, E, k, H, I, 70 + T)
    dev = layer.to_device(inp)
    b = layer.LayerBuffers.allocate(T, E, k, H, I)
    b.ws.fill_(0x5A)
    bias = (np.random.default_rng(T).standard_normal(E) * 0.1).astype(np.float32)
    how = dict(score="sigmoid", groups=groups, topk_groups=(groups + 1) // 2, scale=2.5)
    binding.moe_route_scored_and_group(dev["logits"], k, b.topk_ids, b.topk_weights, b.bitmatrix, b.counts, b.offsets,
                                       b.gather, b.scatter, b.ws, bias=torch.from_numpy(bias).cuda(), **how)
    layer.run_ffn(dev, b, 10.0)
    torch.cuda.synchronize()
    ids, w = fp8.route_scored(inp["logits"], k, bias=bias, **how)
    assert np.array_equal(b.topk_ids.cpu().numpy(), ids)
    counts, offsets, gather, scatter = oracle.expert_offsets(ids, E)
    assert np.array_equal(b.gather.cpu().numpy(), gather) and np.array_equal(b.scatter.cpu().numpy(), scatter)
    ys = oracle.ffn(inp["x"], gather, offsets, k, inp["w1"], inp["w1_s"], inp["w2"], inp["w2_s"], 10.0)
    ffn_close(layer.bf16_tensor_to_f32(b.y_sorted), ys)
    ffn_close(layer.bf16_tensor_to_f32(b.y), oracle.combine(ys, w.astype(np.float32), scatter, T, k))


@pytest.mark.parametrize("T,E,groups", [(24, 256, 8), (25, 256, 1), (24, 40, 1), (25, 40, 5), (8, 512, 1), (9, 512, 1),
                                        (8, 300, 3), (9, 300, 3), (24, 512, 64), (24, 65, 13)])
def test_and_group_on_both_sides_of_the_one_launch_rule(T, E, groups):
    test_and_group_equals_the_separate_calls(T, E, 6 if E // groups > 5 else 2, groups)

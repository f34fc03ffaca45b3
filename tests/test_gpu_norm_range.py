"""The norm and its gradient where fp32 products leave their range on the way to results within it.

Tolerances as in test_gpu_block.py: bf16 results half a step, NORM for the fp32 in front of them.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from mxfp4_routed_expert_route_amd import binding
from oracle import block
from tests.test_gpu_block import DEV, HALF, NORM, U, check_norm_grad, close, f64, gen, norm, norm_grad, randn

pytestmark = pytest.mark.gpu


def check(x, w, eps, out):
    """y, and the FP8 output by what it stands for: runs of small values are quantised from y."""
    _, y = block.rms_norm(f64(x), None, f64(w), eps)
    H = x.shape[1]
    close(out["y"], y, np.abs(y) * (HALF + NORM) + 2.0 ** -133, "y")
    amax = np.maximum.reduceat(np.abs(y), np.arange(0, H, 128), axis=1)
    scale = np.maximum(amax, 2.0 ** -100) / 448.0
    close(out["scale"], scale, scale * (NORM + 2 * U), "scale")
    each = np.repeat(scale, 128, axis=1)[:, :H]
    back = f64(out["q"].float()) * np.repeat(f64(out["scale"]), 128, axis=1)[:, :H]
    # half a step of E4M3 relative, half its smallest step below 2^-6 of the scale's unit
    close(back, y, np.abs(y) * (2.0 ** -4 + 2 * NORM) + each * 2.0 ** -10 * 1.01, "q")


SIZES = [64, 208, 400, 1024, 4096, 16400, 65536]   # every number of lanes and chunks of a row


@pytest.mark.parametrize("H", SIZES)
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
def test_norm_of_one_huge_element_among_small_ones(H, wtype):
    """A row whose squares leave fp32, with elements whose products are below it until they meet 1 / rms."""
    g = gen(H)
    x = torch.rand(5, H, generator=g) + 1.0
    for i, (huge, small) in enumerate([(52, -45), (52, -50), (127, 30), (60, -40), (100, -20)]):
        x[i] *= 2.0 ** small
        x[i, (7 * i) % H] = 2.0 ** huge
    x = x.bfloat16().to(DEV)
    w = randn(g, H, dtype=wtype)
    for eps in (0.0, 1e-6):
        check(x, w, eps, norm(x, w, eps, None, y=True, q=True))


@pytest.mark.parametrize("H", SIZES)
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
def test_norm_of_large_rows_by_large_weights(H, wtype):
    """s w is past fp32's largest value, s w / rms is not; beside runs where neither is."""
    g = gen(H + 1)
    x = torch.randn(3, H, generator=g)
    for i, size in enumerate([45, 40, 0]):
        x[i] *= 2.0 ** size
    x = x.bfloat16().to(DEV)
    w = torch.randn(H, generator=g)
    w[: H // 2 : 3] *= 2.0 ** 100
    w = w.to(wtype).to(DEV)
    check(x, w, 1e-6, norm(x, w, 1e-6, None, y=True, q=True))
    y = norm(x, w, 1e-6, None, y=True, q=False)["y"]
    assert torch.equal(y, norm(x, w, 1e-6, None, y=True, q=True)["y"])


@pytest.mark.parametrize("H", SIZES)
def test_norm_grad_of_one_huge_element_among_small_ones(H):
    g = gen(H + 2)
    s = torch.rand(4, H, generator=g) + 1.0
    for i, (huge, small) in enumerate([(52, -45), (52, -50), (127, 30), (60, -40)]):
        s[i] *= 2.0 ** small
        s[i, 3] = 2.0 ** huge
    s = s.bfloat16().to(DEV)
    w = randn(g, H)
    dy = randn(g, 4, H)
    dy[:, 3] = 0.0       # no large term in any sum
    dx, dw = norm_grad(s, w, 0.0, dy)
    check_norm_grad(s, w, 0.0, dy, None, dx, dw)
    for i in range(4):   # a weight's gradient of one row alone
        dx, dw = norm_grad(s[i:i + 1], w, 0.0, dy[i:i + 1])
        check_norm_grad(s[i:i + 1], w, 0.0, dy[i:i + 1], None, dx, dw)
    dy *= 2.0 ** 30      # the mean of the small terms reaches the huge element's dx
    dx, dw = norm_grad(s[:1], w, 0.0, dy[:1])
    check_norm_grad(s[:1], w, 0.0, dy[:1], None, dx, dw)


@pytest.mark.parametrize("H", SIZES)
def test_norm_grad_of_subnormal_rows(H):
    """Without eps 1 / rms is past fp32's largest value; dx is not."""
    g = gen(H + 3)
    s = (torch.randint(-7, 8, (4, H), generator=g).float() * 2.0 ** -133)
    s[:, 0] = 2.0 ** -132
    s = s.bfloat16().to(DEV)
    w = randn(g, H)
    dy, dsum = randn(g, 4, H, scale=2.0 ** -30), randn(g, 4, H)
    dy[1] = 0.0
    dx, dw = norm_grad(s, w, 0.0, dy, dsum)
    check_norm_grad(s, w, 0.0, dy, dsum, dx, dw)
    assert torch.equal(dx[1], dsum[1])


@pytest.mark.parametrize("H", SIZES)
def test_norm_and_gradient_of_extreme_rows_in_place(H):
    """Among ordinary rows that share their wavefronts, with outputs over inputs."""
    g = gen(H + 4)
    x = torch.randn(37, H, generator=g)
    x[1::5] *= 2.0 ** -45
    x[1::5, 2] = 2.0 ** 52
    x[2::5] *= 2.0 ** 45        # s w overflows
    x[3::5] *= 2.0 ** -131      # subnormal
    x = x.bfloat16().to(DEV)
    w = torch.randn(H, generator=g)
    w[::7] *= 2.0 ** 90
    w = w.to(DEV)
    want = norm(x, w, 0.0, None, y=True, q=True)
    y = x.clone()
    binding.moe_rms_norm(y, w, 0.0, y=y, q=(q := torch.empty_like(want["q"])), scale=(s := torch.empty_like(want["scale"])))
    assert torch.equal(y, want["y"]) and torch.equal(q.view(torch.uint8), want["q"].view(torch.uint8)) and torch.equal(s, want["scale"])
    r, zero = x.clone(), torch.zeros_like(x)
    binding.moe_rms_norm(zero, w, 0.0, residual=r, sum=r, y=zero)
    assert torch.equal(r, x) and torch.equal(zero, want["y"])

    w = randn(g, H)
    dy, dsum = randn(g, 37, H, scale=2.0 ** -20), randn(g, 37, H)
    dx, dw = norm_grad(x, w, 0.0, dy, dsum)
    check_norm_grad(x, w, 0.0, dy, dsum, dx, dw)
    ws = torch.empty(binding.moe_rms_norm_grad_workspace_bytes(37, H), dtype=torch.uint8, device=DEV)
    for over_dy in (True, False):
        d, e, out = dy.clone(), dsum.clone(), torch.empty(H, device=DEV)
        binding.moe_rms_norm_grad(x, w, 0.0, d, d if over_dy else e, out, ws, dsum=e)
        assert torch.equal(d if over_dy else e, dx) and torch.equal(out, dw)

"""Adapters at values where the parts of the inner sums show: what they make of infinite weights, and how
much of a sum they hold.  Each form of the call is taken by its sizes: one launch for a few rows, two
launches, one launch for many.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_block import DEV, HALF, U, check_lora, close, f64, gen, randn, run_lora

pytestmark = pytest.mark.gpu

FORMS = [(1, 16), (40, 24), (300, 8), (300, 40), (300, 72), (300, 136), (4000, 128), (7000, 16), (7000, 24), (7000, 64)]


@pytest.mark.parametrize("M,R", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("whole", [False, True])
def test_lora_infinite_weights(M, R, dtype, whole):
    """An infinity in B gives an infinity of its sign and the inner sum's, NaN only where the formula does."""
    N, K, L = 72, 64, 3
    g = gen(M * 3 + R)
    x, a = randn(g, M, K), randn(g, L, R, K, scale=K ** -0.5)
    if whole:       # inner sums that a single part holds
        x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
        x[torch.arange(M), torch.arange(M) % K] = 1.0
    b = randn(g, L, N, R, scale=R ** -0.5)
    inf = float("inf")
    b[0, 3, 0], b[1, 3, 1], b[1, 60, R - 1] = inf, -inf, inf
    b[0, 20, 2], b[0, 20, 5] = inf, -inf       # of both signs: an infinity or NaN by the sums' signs
    b[0, 71, 4], b[1, 70, 6] = float("nan"), -inf
    a[1, 6, 2], a[1, 6, 5], a[1, 6, 6] = 0.0, 0.0, 0.0
    if whole:
        x[M // 2] = 0.0                         # 0 times an infinity
    ids = np.random.default_rng(M + R).integers(-1, L, size=M) if M > 1 else np.zeros(1, int)
    s = torch.tensor([0.5, -2.0, 1.5], device=DEV)
    base = randn(g, M, N, dtype=dtype)
    y = run_lora(x, a, b, s, ids, base, dtype)
    X, A, B, S = f64(x), f64(a), f64(b), f64(s)
    want = f64(base).copy()
    for l in range(L):
        at = np.nonzero(ids == l)[0]
        with np.errstate(all="ignore"):
            want[at] += S[l] * ((X[at] @ A[l].T)[:, None, :] * B[l][None]).sum(axis=2)
    got = f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.where(np.isinf(got), got, 0.0), np.where(np.isinf(want), want, 0.0))
    b[~b.isfinite()] = 0.0                      # the other results are as without them
    rest = f64(run_lora(x, a, b, s, ids, base, dtype))
    assert np.array_equal(np.where(np.isfinite(want), got, 0.0), np.where(np.isfinite(want), rest, 0.0))
    check_lora(x, a, b, s, ids, base, torch.from_numpy(rest).to(dtype))


@pytest.mark.parametrize("M,R", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_holds_2_to_minus_17_of_an_inner_sum(M, R, dtype):
    """An inner sum of 24 bits, less its upper two parts by two other ranks: what is left is the third part,
    and 2^-17 of the sum for bf16 results."""
    P, N = 64, 72
    g = gen(M + R)
    v = 1.0 + torch.randint(0, 2 ** 23, (P,), generator=g).double() * 2.0 ** -23
    v[0] = 1.0 + 2.0 ** -8 + 2.0 ** -16
    v[1] = 1.0 + 2.0 ** -7 + 2.0 ** -8 + 2.0 ** -15 + 2.0 ** -16
    v[2] = 2.0 - 2.0 ** -23
    v *= torch.where(torch.rand(P, generator=g) < 0.5, -1.0, 1.0).double()
    v *= 2.0 ** torch.randint(-20, 21, (P,), generator=g).double()
    hi = v.bfloat16()
    mid = (v - hi.double()).bfloat16()
    low = (v - hi.double() - mid.double()).bfloat16()
    assert torch.equal(hi.double() + mid.double() + low.double(), v)
    a = torch.zeros(1, R, 3 * P)
    for i, t in enumerate((hi, mid, low)):
        a[0, 0, i::3] = t.float()
    a[0, 1, 0::3], a[0, 2, 1::3] = -hi.float(), -mid.float()
    a = a.bfloat16().to(DEV)
    x = torch.zeros(M, 3 * P)
    of = torch.arange(M) % P
    for i in range(3):
        x[torch.arange(M), 3 * of + i] = 1.0
    x = x.bfloat16().to(DEV)
    b = torch.zeros(1, N, R, dtype=torch.bfloat16, device=DEV)
    b[:, :, :3] = 1.0
    y = f64(run_lora(x, a, b, None, np.zeros(M, int), None, dtype))
    want = low.double().numpy()[of.numpy()][:, None]
    part = 2.0 ** -17 if dtype == torch.bfloat16 else 0.0
    half = HALF if dtype == torch.bfloat16 else U
    # the sum of exact parts in fp32 is exact: they are 24 bits of one sum
    close(y, np.broadcast_to(want, y.shape), part * np.abs(v.numpy()[of.numpy()])[:, None] + half * np.abs(want), "y")

"""The operators around the layer at sizes where their launches grow or are cut: more tokens than a
workgroup's smallest share times the launch, several long sequences side by side, more rows than one
launch of the norm, rows at the borders of the adapters' forms."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from mxfp4_routed_expert_route_amd import binding
from tests.test_gpu_block import DEV, FP8, balance, check_balance, check_lora, check_norm, gen, lora, randn, run_lora

pytestmark = pytest.mark.gpu


def inputs(T, E, k, seed, cuts, dtype):
    g = gen(seed)
    logits = randn(g, T, E, dtype=dtype, scale=1.5)
    ids = torch.rand(T, E, generator=g).argsort(dim=1)[:, :k].to(torch.int32).contiguous().to(DEV)
    offsets = None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device=DEV)
    S = 1 if cuts is None else len(cuts) - 1
    return logits, ids, offsets, (torch.rand(S, generator=g) + 0.5).to(DEV), randn(g, T, E, dtype=dtype, scale=0.01)


def some_cuts(T, n, seed, lead, trail):
    """Sequences of all lengths, many of them short, a few that take most of the tokens."""
    r = np.random.default_rng(seed)
    lengths = np.floor(np.exp(r.uniform(0.0, np.log(T / 4), size=n))).astype(int)
    lengths[r.integers(0, n, size=n // 8)] = 0
    cuts = lead + np.concatenate([[0], np.cumsum(lengths)])
    return np.minimum(cuts, T - trail).tolist()


BALANCE = [(33000, 24, 4, None), (33000, 20, 8, [0, 16500, 33000]), (33000, 7, 3, some_cuts(33000, 300, 1, 77, 33)),
           (65537, 12, 6, some_cuts(65537, 90, 2, 0, 1)), (65537, 40, 8, [5, 1030, 2060, 3085, 9000, 30000, 65000]),
           (65537, 33, 2, None), (300001, 8, 8, some_cuts(300001, 60, 3, 1000, 500)), (300001, 10, 2, None),
           (300001, 12, 4, some_cuts(300001, 2000, 4, 3, 3)), (300001, 6, 5, [0, 1640, 3281, 150000, 300001])]


@pytest.mark.parametrize("i", range(len(BALANCE)))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_of_many_tokens(i, score):
    T, E, k, cuts = BALANCE[i]
    dtype = torch.bfloat16 if i % 3 == 1 else torch.float32
    logits, ids, offsets, dloss, add = inputs(T, E, k, 100 + i, cuts, dtype)
    add = add if i % 2 else None
    check_balance(logits, ids, offsets, dloss, add, score, balance(logits, ids, offsets, dloss, add, score))


@pytest.mark.parametrize("k", [1, 4, 5, 8])
def test_balance_of_long_sequences_side_by_side(k):
    """Sequences just over and just under the length that is counted by a launch of its own, several of them in
    one counting chunk's reach."""
    n = 8192 // k
    cuts = np.cumsum([100, n + 1, n + 1, n, n + 2, 1, n + 1, 3 * n, n - 1, n + 5]).tolist()
    T = cuts[-1] + 40
    logits, ids, offsets, dloss, add = inputs(T, 16, k, 7 + k, cuts, torch.float32)
    check_balance(logits, ids, offsets, dloss, add, "softmax", balance(logits, ids, offsets, dloss, add, "softmax"))


@pytest.mark.parametrize("H", [16, 136])
def test_norm_of_more_rows_than_a_launch(H):
    rows = 2 ** 21 + 3
    g = gen(H)
    few = randn(g, 4099, H)
    x = few.repeat(rows // 4099 + 1, 1)[:rows].contiguous()
    r = randn(g, 5003, H, scale=3.0).repeat(rows // 5003 + 1, 1)[:rows].contiguous()
    w = randn(g, H)
    q = H % 16 == 0
    out = dict(sum=torch.zeros_like(x), y=torch.zeros_like(x))
    if q:
        out.update(q=torch.zeros(rows, H, dtype=FP8, device=DEV), scale=torch.zeros(rows, -(-H // 128), device=DEV))
    binding.moe_rms_norm(x, w, 1e-6, residual=r, **out)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(0, 50), torch.arange(2 ** 20 - 20, 2 ** 20 + 20), torch.arange(rows - 60, rows)]).to(DEV)
    check_norm(x[at], w, 1e-6, r[at], {n: (t.view(torch.uint8)[at].view(FP8) if t.dtype == FP8 else t[at]) for n, t in out.items()})
    # every other row: as from launches of fewer rows
    for r0 in range(0, rows, 2 ** 20 + 1):
        r1 = min(r0 + 2 ** 20 + 1, rows)
        part = {n: torch.empty_like(t[r0:r1]) for n, t in out.items()}
        binding.moe_rms_norm(x[r0:r1], w, 1e-6, residual=r[r0:r1], **part)
        for n, t in part.items():
            assert torch.equal(t.view(torch.uint8), out[n][r0:r1].view(torch.uint8)), n


@pytest.mark.parametrize("M,R", [(4199, 16), (4200, 16), (3952, 24), (3953, 24), (1976, 40), (1977, 40), (11856, 8), (11857, 8),
                                 (11857, 64), (24144, 32), (24145, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_at_the_borders_of_one_launch(M, R, dtype):
    """With 8 adapters: 17 and 18 (16 and 17, 8 and 9) rows a tile, the most rows of a round of tiles and one more."""
    N, K, L = 72, 64, 8
    ids = np.sort(np.random.default_rng(M).integers(-1, L, size=M))
    x, a, b, s, base = lora(M, N, K, R, L, ids, M + R, dtype)
    check_lora(x, a, b, s, ids, base, run_lora(x, a, b, s, ids, base, dtype))

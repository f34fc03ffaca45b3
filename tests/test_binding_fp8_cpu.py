"""The Python binding of scored routing and the FP8 operators (CPU: no call reaches the library)."""
from __future__ import annotations

import pytest
import torch

from mxfp4_routed_expert_route_amd import binding


def _calls():
    """One call of each entry point, on CPU tensors of the right types and shapes."""
    T, E, k, H, I = 4, 8, 2, 128, 128
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    f32, bf16 = torch.zeros, lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    logits = (f32(T, E), bf16(T, E))
    for l in logits:
        yield lambda l=l: binding.moe_route_scored(l, k, i32(T, k), f32(T, k), bias=f32(E))
        yield lambda l=l: binding.moe_route_scored_and_group(l, k, i32(T, k), f32(T, k), i32(T, 1), i32(E), i32(E + 1),
                                                             i32(T * k), i32(T * k), u8(64))
    yield lambda: binding.moe_quantize_fp8(bf16(T, H), u8(T, H), f32(T, 1))
    yield lambda: binding.moe_gemm_fp8(u8(T, H), f32(T, 1), u8(I, H), f32(1, 1), bf16(T, I), u8(16))
    yield lambda: binding.moe_gemm_fp8(u8(T, H), f32(T, 1), u8(I, H), f32(1, 1), f32(T, I))
    yield lambda: binding.moe_grouped_ffn_fp8(bf16(T, H), k, u8(E, 2 * I, H), f32(E, 2, 1), u8(E, H, I), f32(E, 1, 1),
                                              i32(E), i32(E + 1), i32(T * k), 10.0, bf16(T * k, H), u8(64))


def test_every_argument_is_given_to_the_native_checks_as_they_take_it(monkeypatch):
    # the native check takes a tuple of types and a tuple shape; anything else goes the slow way
    seen = []

    def arg(t, dtypes, shape, dev, name):
        assert isinstance(dtypes, tuple) and isinstance(shape, tuple), name
        assert t.dtype in dtypes and tuple(t.shape) == shape, name
        seen.append(name)
        return 0

    monkeypatch.setattr(binding, "_arg", arg)
    monkeypatch.setattr(binding, "_run", lambda *a: None)
    for call in _calls():
        call()
    assert seen.count("logits") == 4 and len(seen) == 2 * 4 + 2 * 9 + 3 + 6 + 5 + 10

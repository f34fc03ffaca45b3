"""Refusals of scored routing and the FP8 operators through the C ABI (CPU: no call here
passes its host checks, so nothing touches a GPU)."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

from mxfp4_routed_expert_route_amd import binding
from mxfp4_routed_expert_route_amd import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
P = 4096   # an aligned stand-in pointer that no check reads


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(build_mod.LIB):
        build_mod.build_library()
    return binding.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_fp8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text)) | {"moe_route_scored", "moe_route_scored_and_group"}
    out = subprocess.run(["nm", "-D", "--defined-only", build_mod.LIB], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\sT\s+(\S+)", out))
    assert names <= set(binding.EXPORTS) and all(callable(getattr(binding, n)) for n in names)


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "moe_fp8.h"\nint main(void) { return MOE_F32 + MOE_SCORE_SOFTMAX; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-fsyntax-only",
                    str(src)], check=True)


def test_route_scored_refusals(lib):
    def call(logits=P, kind=0, T=16, E=256, k=6, score=1, bias=P, groups=8, topk_groups=4, group_top=2, ids=P,
             w=P):
        return lib.moe_route_scored(logits, kind, T, E, k, score, bias, groups, topk_groups, group_top, 1, 1.0,
                                    ids, w, None)
    for bad in (dict(T=-1), dict(E=0, groups=1), dict(k=0), dict(kind=2), dict(kind=-1), dict(score=2),
                dict(score=-1), dict(groups=0), dict(groups=7), dict(topk_groups=0), dict(topk_groups=9),
                dict(group_top=0), dict(group_top=3), dict(E=8, k=2, topk_groups=1), dict(logits=None),
                dict(ids=None), dict(w=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(E=1025, groups=1, topk_groups=1), dict(k=9), dict(groups=128), dict(T=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=P + 2), dict(logits=P + 1, kind=1), dict(bias=P + 2), dict(ids=P + 2), dict(w=P + 1)):
        assert call(**bad) == MISALIGNED, bad
    assert call(T=0, logits=None, ids=None, w=None) == OK


def test_route_scored_and_group_refusals(lib):
    def call(T=16, ids=P, bm=P, counts=P, offsets=P, gather=P, scatter=P, ws=P, ws_bytes=1 << 20, groups=8):
        return lib.moe_route_scored_and_group(P, 0, T, 256, 6, 1, None, groups, 4, 2, 1, 1.0, ids, P, bm, counts,
                                              offsets, gather, scatter, ws, ws_bytes, None)
    for bad in (dict(bm=None), dict(counts=None), dict(offsets=None), dict(gather=None), dict(scatter=None),
                dict(ws=None), dict(groups=3), dict(T=0, counts=None)):
        assert call(**bad) == INVALID, bad
    assert call(ws_bytes=16 * 4 - 1) == WS_SMALL
    assert call(ws=P + 8) == MISALIGNED and call(gather=P + 2) == MISALIGNED


def test_quantize_refusals(lib):
    call = lambda x=P, rows=4, K=256, q=P, s=P: lib.moe_quantize_fp8(x, rows, K, q, s, None)
    for bad in (dict(rows=-1), dict(K=0), dict(K=-16), dict(x=None), dict(q=None), dict(s=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=8), dict(K=120), dict(K=65536 + 16), dict(rows=1 << 31)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(x=P + 8), dict(q=P + 8), dict(s=P + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert call(rows=0, x=None, q=None, s=None) == OK


def test_gemm_refusals(lib):
    def call(xq=P, xs=P, M=4, N=256, K=256, w=P, ws=P, kind=1, y=P, work=P, nbytes=1 << 40):
        return lib.moe_gemm_fp8(xq, xs, M, N, K, w, ws, kind, y, work, nbytes, None)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(kind=2), dict(xq=None), dict(xs=None), dict(w=None),
                dict(ws=None), dict(y=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=100), dict(K=65536 + 16), dict(N=(1 << 24) + 1), dict(M=1 << 31), dict(M=1 << 20, N=1 << 20)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(xq=P + 8), dict(w=P + 4), dict(y=P + 4), dict(xs=P + 2), dict(ws=P + 1), dict(work=P + 8)):
        assert call(**bad) == MISALIGNED, bad
    assert call(M=0, xq=None, xs=None, w=None, ws=None, y=None) == OK
    assert lib.moe_gemm_fp8_workspace_bytes(-1, 256, 256) == 0 == lib.moe_gemm_fp8_workspace_bytes(4, 0, 256)


def test_gemm_workspace_is_checked(lib):
    for M, N, K in ((1, 256, 4096), (64, 256, 16384), (300, 500, 4096), (512, 4096, 2048), (8191, 4096, 4096)):
        need = lib.moe_gemm_fp8_workspace_bytes(M, N, K)
        if need:
            assert lib.moe_gemm_fp8(P, P, M, N, K, P, P, 1, P, P, need - 1, None) == WS_SMALL
            assert lib.moe_gemm_fp8(P, P, M, N, K, P, P, 1, P, None, need, None) == INVALID


def test_ffn_refusals(lib):
    ws = lib.moe_fp8_workspace_bytes(16, 256, 6, 4096, 2048)
    def call(x=P, T=16, H=4096, I=2048, E=256, k=6, w1=P, w1s=P, w2=P, w2s=P, counts=P, offsets=P, gather=P, y=P,
             work=P, nbytes=ws):
        return lib.moe_grouped_ffn_fp8(x, T, H, I, E, k, w1, w1s, w2, w2s, counts, offsets, gather, 10.0, y, work,
                                       nbytes, None)
    assert ws > 0
    for bad in (dict(T=-1), dict(H=0), dict(I=-128), dict(k=0), dict(k=300), dict(E=0),
                *[{n: None} for n in ("x", "w1", "w1s", "w2", "w2s", "counts", "offsets", "gather", "y", "work")]):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=4100), dict(I=100), dict(H=65536 + 128), dict(H=65536, I=32768), dict(E=1025), dict(k=9),
                dict(T=1 << 20, k=6)):
        assert call(**bad) == UNSUPPORTED, bad
    for n in ("x", "w1", "w2", "y", "work"):
        assert call(**{n: P + 8}) == MISALIGNED
    for n in ("w1s", "w2s", "counts", "offsets", "gather"):
        assert call(**{n: P + 2}) == MISALIGNED
    assert call(nbytes=ws - 1) == WS_SMALL
    assert call(T=0, x=None, y=None, work=None, nbytes=0) == OK
    for bad in ((-1, 256, 6, 4096, 2048), (16, 256, 6, 4100, 2048), (16, 256, 6, 65536, 65536)):
        assert lib.moe_fp8_workspace_bytes(*bad) == 0
    # one buffer serves the routing calls too
    assert lib.moe_fp8_workspace_bytes(8191, 256, 6, 128, 128) >= 16 * 256 * 4


def test_binding_refuses_cpu_tensors_shapes_and_types(lib):
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_quantize_fp8(x, torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 1))
    with pytest.raises(ValueError, match="score"):
        binding.moe_route_scored(torch.zeros(2, 8), 2, None, None, score="relu")
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        binding.moe_route_scored(torch.zeros(2, 8, dtype=torch.float16), 2, None, None)
    for call in (lambda: binding.moe_route_scored(torch.zeros(8), 2, None, None),
                 lambda: binding.moe_quantize_fp8(torch.zeros(8), None, None),
                 lambda: binding.moe_gemm_fp8(torch.zeros(8), None, x, None, x),
                 lambda: binding.moe_grouped_ffn_fp8(x, 1, x, None, None, None, None, None, None, 0.0, None, None)):
        with pytest.raises(ValueError):
            call()


def test_native_argument_checks_are_in_use(lib):
    assert binding._arg is binding._marshal.arg
    x = torch.zeros(2, 4)
    for bad, match in (((x, (torch.float32,), (2, 4), -1, "x"), "GPU tensor"),
                       ((x, (torch.int32,), (2, 4), 0, "x"), "must be torch.int32"),
                       ((None, (torch.float32,), (2, 4), 0, "x"), "got None")):
        with pytest.raises(ValueError, match=match):
            binding._arg(*bad)
    with pytest.raises(TypeError):
        binding._arg(x)


@pytest.mark.parametrize("E,k,H,I", [(256, 6, 128, 128), (8, 2, 128, 128), (1, 1, 128, 256), (64, 8, 256, 512), (1024, 8, 128, 128)])
def test_ffn_workspace_never_shrinks_with_the_batch(lib, E, k, H, I):
    sizes = [binding.moe_fp8_workspace_bytes(T, E, k, H, I) for T in range(1, 6000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0


def test_host_checks_run_under_sanitizers():
    # the checks and the workspace layout at the ends of their ranges, with address and undefined-behaviour checks
    r = subprocess.run([build_mod.build_validate_check()], capture_output=True, text=True)
    assert r.returncode == 0 and not r.stderr, r.stdout + r.stderr
    assert "scored routing and fp8 checks ok" in r.stdout


def test_gemm_takes_no_workspace(lib):
    # 0 bytes at every size, and a call without a workspace is refused for its misaligned y alone
    for M, N, K in ((1, 1, 16), (1, 256, 4096), (64, 256, 16384), (512, 4096, 2048), (8191, 4096, 4096), (17, 70000, 144)):
        assert lib.moe_gemm_fp8_workspace_bytes(M, N, K) == 0
        for kind in (0, 1):
            assert lib.moe_gemm_fp8(P, P, M, N, K, P, P, kind, P + 8, None, 0, None) == MISALIGNED
            assert lib.moe_gemm_fp8(P, P, M, N, K, P, P, kind, P + 8, P, 0, None) == MISALIGNED

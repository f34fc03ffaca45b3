"""Refusals of the operators around the routed layer, through the C ABI and the binding (CPU: no
call here passes its host checks, so nothing touches a GPU)."""
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
Q = 8192   # another
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(build_mod.LIB):
        build_mod.build_library()
    return binding.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_block.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text))
    assert len(names) == 9
    out = subprocess.run(["nm", "-D", "--defined-only", build_mod.LIB], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\sT\s+(\S+)", out))
    assert names <= set(binding.EXPORTS) and all(callable(getattr(binding, n)) for n in names)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "moe_block.h"\nint main(void) { return MOE_F32 + MOE_SCORE_SOFTMAX; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-fsyntax-only",
                    str(src)], check=True)


def change(good, call, cases):
    for kw, want in cases:
        assert call(**{**good, **kw}) == want, (kw, want)


def test_norm_refusals(lib):
    good = dict(x=P, xs=256, res=P, rows=4, H=256, wt=0, w=P, eps=1e-6, sum=Q, y=P, q=P, scale=P)

    def call(x, xs, res, rows, H, wt, w, eps, sum, y, q, scale):
        return lib.moe_rms_norm(x, xs, res, rows, H, wt, w, eps, sum, y, q, scale, None)

    change(good, call, [
        (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(rows=2 ** 31), UNSUPPORTED), (dict(H=0), INVALID),
        (dict(H=260), UNSUPPORTED), (dict(H=264, xs=264), UNSUPPORTED), (dict(H=65552, xs=65552), UNSUPPORTED),
        (dict(xs=248), INVALID), (dict(xs=260), UNSUPPORTED), (dict(xs=2 ** 31 + 7), UNSUPPORTED),
        (dict(wt=2), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
        (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None, q=None, scale=None), INVALID),
        (dict(scale=None), INVALID), (dict(q=None), INVALID), (dict(res=None), INVALID),
        (dict(xs=264), INVALID), (dict(sum=P, y=P), INVALID),
        (dict(x=P + 8), MISALIGNED), (dict(res=P + 8), MISALIGNED), (dict(w=P + 4), MISALIGNED),
        (dict(sum=P + 8), MISALIGNED), (dict(y=P + 8), MISALIGNED), (dict(q=P + 8), MISALIGNED),
        (dict(scale=P + 2), MISALIGNED)])


def test_norm_grad_refusals(lib):
    need = lib.moe_rms_norm_grad_workspace_bytes(4, 256)
    assert need >= 4 * 256 * 4
    good = dict(s=P, ss=256, rows=4, H=256, wt=1, w=P, eps=0.0, dy=P, dsum=P, dx=Q, dw=P, ws=P, n=need)

    def call(s, ss, rows, H, wt, w, eps, dy, dsum, dx, dw, ws, n):
        return lib.moe_rms_norm_grad(s, ss, rows, H, wt, w, eps, dy, dsum, dx, dw, ws, n, None)

    change(good, call, [
        (dict(rows=-1), INVALID), (dict(rows=2 ** 31), UNSUPPORTED), (dict(H=4), UNSUPPORTED), (dict(H=-8), INVALID),
        (dict(ss=128), INVALID), (dict(ss=257), UNSUPPORTED), (dict(wt=-1), INVALID), (dict(eps=-1.0), INVALID),
        (dict(dx=None, dw=None, dsum=None), INVALID), (dict(dx=None), INVALID), (dict(s=None), INVALID),
        (dict(w=None), INVALID), (dict(dy=None), INVALID), (dict(ws=None), INVALID), (dict(dx=P), INVALID),
        (dict(rows=0, dw=None, dx=Q), OK), (dict(dw=P + 4), MISALIGNED), (dict(s=P + 8), MISALIGNED),
        (dict(dy=P + 8), MISALIGNED), (dict(dsum=P + 8), MISALIGNED), (dict(dx=P + 8), MISALIGNED),
        (dict(ws=P + 8), MISALIGNED), (dict(n=need - 1), WS_SMALL)])
    for bad in ((-1, 256), (4, 0), (4, 12), (4, 65544), (2 ** 31, 8)):
        assert lib.moe_rms_norm_grad_workspace_bytes(*bad) == 0
    sizes = [lib.moe_rms_norm_grad_workspace_bytes(r, 4096) for r in range(0, 3000, 7)]
    assert sizes == sorted(sizes)


def test_balance_refusals(lib):
    need = lib.moe_balance_loss_workspace_bytes(100, 64, 3)
    good = dict(l=P, lt=0, T=100, E=64, k=4, sc=0, ids=P, so=P, S=3, loss=P, c=P, dl=P, add=P, d=P, ws=P, n=need)

    def call(l, lt, T, E, k, sc, ids, so, S, loss, c, dl, add, d, ws, n):
        return lib.moe_balance_loss(l, lt, T, E, k, sc, ids, so, S, loss, c, dl, add, d, ws, n, None)

    change(good, call, [
        (dict(T=-1), INVALID), (dict(T=2 ** 30), UNSUPPORTED), (dict(E=0), INVALID), (dict(E=1025), UNSUPPORTED),
        (dict(k=0), INVALID), (dict(k=9), UNSUPPORTED), (dict(k=65), INVALID), (dict(lt=2), INVALID), (dict(sc=2), INVALID),
        (dict(S=0), INVALID), (dict(S=2 ** 20 + 1), UNSUPPORTED), (dict(so=None), INVALID), (dict(l=None), INVALID),
        (dict(ids=None), INVALID), (dict(loss=None), INVALID), (dict(c=None), INVALID), (dict(dl=None), INVALID),
        (dict(d=None), INVALID), (dict(d=None, dl=None), INVALID), (dict(ws=None), INVALID), (dict(l=P + 2), MISALIGNED),
        (dict(ids=P + 2), MISALIGNED), (dict(so=P + 1), MISALIGNED), (dict(loss=P + 2), MISALIGNED),
        (dict(c=P + 2), MISALIGNED), (dict(dl=P + 2), MISALIGNED), (dict(add=P + 2), MISALIGNED),
        (dict(d=P + 2), MISALIGNED), (dict(ws=P + 8), MISALIGNED), (dict(n=need - 1), WS_SMALL),
        (dict(lt=1, l=P + 1), MISALIGNED)])
    good2 = dict(l=P, lt=1, T=100, E=64, k=4, sc=1, so=None, S=1, c=P, dl=P, add=None, d=P)

    def grad(l, lt, T, E, k, sc, so, S, c, dl, add, d):
        return lib.moe_balance_loss_grad(l, lt, T, E, k, sc, so, S, c, dl, add, d, None)

    change(good2, grad, [
        (dict(T=0), OK), (dict(S=2), INVALID), (dict(l=None), INVALID), (dict(c=None), INVALID), (dict(dl=None), INVALID),
        (dict(d=None), INVALID), (dict(d=P + 1), MISALIGNED), (dict(c=P + 2), MISALIGNED), (dict(E=2000), UNSUPPORTED)])
    for bad in ((-1, 64, 1), (1, 0, 1), (1, 1025, 1), (1, 64, 0), (1, 64, 2 ** 20 + 1), (2 ** 31, 64, 1)):
        assert lib.moe_balance_loss_workspace_bytes(*bad) == 0
    sizes = [lib.moe_balance_loss_workspace_bytes(T, 64, 5) for T in range(0, 300000, 997)]
    assert sizes == sorted(sizes)


def test_lora_refusals(lib):
    assert lib.moe_lora_group(P, 4, 0, P, P, None) == INVALID
    assert lib.moe_lora_group(P, 4, 1025, P, P, None) == UNSUPPORTED
    assert lib.moe_lora_group(P, -1, 4, P, P, None) == INVALID
    assert lib.moe_lora_group(P, 2 ** 31, 4, P, P, None) == UNSUPPORTED
    assert lib.moe_lora_group(None, 4, 4, P, P, None) == INVALID
    assert lib.moe_lora_group(P, 4, 4, None, P, None) == INVALID
    assert lib.moe_lora_group(P, 4, 4, P, None, None) == INVALID
    assert lib.moe_lora_group(P + 2, 4, 4, P, P, None) == MISALIGNED
    assert lib.moe_lora_group(P, 4, 4, Q, P, None) == INVALID and lib.moe_lora_group(P, 4, 4, Q, P + 12, None) == INVALID
    assert lib.moe_lora_group(P, 4, 4, P + 12, Q, None) == INVALID and lib.moe_lora_group(P + 16, 4, 4, P, Q, None) == INVALID
    assert lib.moe_lora_group(P, 4, 4, Q, Q + 16, None) == INVALID and lib.moe_lora_group(P, 4, 4, Q + 12, Q, None) == INVALID
    need = lib.moe_lora_add_workspace_bytes(10, 96, 128, 16, 3)
    good = dict(x=P, xs=128, M=10, K=128, N=96, R=16, L=3, a=P, b=P, sc=P, off=P, rows=P, yt=1, base=P, bs=96, y=Q, ys=96,
                ws=P, n=need)

    def call(x, xs, M, K, N, R, L, a, b, sc, off, rows, yt, base, bs, y, ys, ws, n):
        return lib.moe_lora_add(x, xs, M, K, N, R, L, a, b, sc, off, rows, yt, base, bs, y, ys, ws, n, None)

    change(good, call, [
        (dict(M=0), OK), (dict(M=-1), INVALID), (dict(M=2 ** 31), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=124), UNSUPPORTED),
        (dict(K=65544, xs=65544), UNSUPPORTED), (dict(N=0), INVALID), (dict(N=2 ** 24 + 1), UNSUPPORTED), (dict(R=0), INVALID),
        (dict(R=12), UNSUPPORTED), (dict(R=264), UNSUPPORTED), (dict(L=0), INVALID), (dict(L=1025), UNSUPPORTED),
        (dict(xs=120), INVALID), (dict(xs=132), UNSUPPORTED), (dict(ys=95), INVALID), (dict(bs=95), INVALID),
        (dict(ys=2 ** 31), UNSUPPORTED), (dict(yt=2), INVALID), (dict(x=None), INVALID), (dict(a=None), INVALID),
        (dict(b=None), INVALID), (dict(off=None), INVALID), (dict(rows=None), INVALID), (dict(y=None), INVALID),
        (dict(ws=None), INVALID), (dict(y=P, ys=104), INVALID), (dict(x=P + 8), MISALIGNED), (dict(a=P + 8), MISALIGNED),
        (dict(b=P + 8), MISALIGNED), (dict(sc=P + 2), MISALIGNED), (dict(off=P + 2), MISALIGNED), (dict(rows=P + 2), MISALIGNED),
        (dict(base=P + 8), MISALIGNED), (dict(y=Q + 8), MISALIGNED), (dict(ws=P + 8), MISALIGNED), (dict(n=need - 1), WS_SMALL)])
    for bad in ((-1, 96, 128, 16, 3), (1, 0, 128, 16, 3), (1, 96, 4, 16, 3), (1, 96, 128, 264, 3), (1, 96, 128, 16, 0)):
        assert lib.moe_lora_add_workspace_bytes(*bad) == 0
    sizes = [lib.moe_lora_add_workspace_bytes(M, 4096, 4096, 16, 8) for M in range(0, 9000, 11)]
    assert sizes == sorted(sizes)


def test_binding_refuses_unsuitable_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, f = torch.zeros(64), torch.zeros(4, 64)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_rms_norm(x, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="weight"):
        binding.moe_rms_norm(x, w.double(), 1e-6, y=x)
    with pytest.raises(ValueError, match="rows, H"):
        binding.moe_rms_norm(x[0], w, 1e-6, y=x)
    with pytest.raises(ValueError, match="GPU tensor|x must"):
        binding.moe_rms_norm(torch.zeros(4, 128, dtype=torch.bfloat16)[:, :64], w, 1e-6, y=x)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_rms_norm_grad(x, w, 1e-6, x, x, w, None)
    with pytest.raises(ValueError, match="score"):
        binding.moe_balance_loss(f, i, torch.zeros(1), torch.zeros(1, 64, dtype=torch.int32), None, score="relu")
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        binding.moe_balance_loss_grad(f.half(), 2, torch.zeros(1, 64, dtype=torch.int32), torch.zeros(1), f)
    with pytest.raises(ValueError, match="32 bits"):
        binding.moe_balance_loss_grad(f, 2 ** 32 + 2, torch.zeros(1, 64, dtype=torch.int32), torch.zeros(1), f)
    with pytest.raises(ValueError, match="32 bits"):
        binding.moe_lora_group(torch.zeros(4, dtype=torch.int32), 2 ** 32 + 4, w, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        binding.moe_lora_group(torch.zeros(4, dtype=torch.int32), 4, torch.zeros(5, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="y must be"):
        binding.moe_lora_add(x, x.view(1, 4, 64), x.view(1, 64, 4), None, i, i, None, f.half(), None)
    big = 2 ** 32 + 16
    assert binding.moe_rms_norm_grad_workspace_bytes(4, big) == 0
    assert binding.moe_balance_loss_workspace_bytes(4, 64, big) == 0
    assert binding.moe_lora_add_workspace_bytes(4, 64, 64, big, 2) == 0

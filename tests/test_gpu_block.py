"""The operators around the routed layer on the GPU against the float64 oracle.

Tolerances, with u = 2^-24 (half a step of fp32) and h = 2^-8 (of bf16), each relative to the
magnitudes that the rounded numbers have:
  sums of n fp32 terms in chains of c additions are within (c + 1) u of the terms' magnitudes;
  a norm's row has chains of at most 64 (a lane's 8 x 8 squares) + 6 + 16, its rstd half that, and
  three more roundings: NORM u;
  p of the balance loss: the exponential's argument is rounded (u times it, at most 104 before it is
  0) and adds 3u, the sum 24 u, the quotient 2u: (D + 32) u with the argument D;
  an inner sum of the adapters: K / 128 MFMAs in a wavefront, each adding 32 products, and 16 partial
  sums: (K / 128 + 32 + 16) 2u of the products' magnitudes, its two bf16 parts 2^-17 (three: none),
  the outer sum (R + 8) 2u.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from mxfp4_routed_expert_route_amd import binding
from oracle import block
from oracle.fp8 import decode_e4m3, quantize_fp8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, HALF = 2.0 ** -24, 2.0 ** -8
NORM = 50 * U
FP8 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def guarded(rows, n, dtype, fill=7):
    """A matrix with a row in front and behind it, for writes past its ends; also the whole."""
    whole = torch.full((rows + 2, n), fill, dtype=torch.float32, device=DEV).to(dtype)
    return whole[1:-1], whole


def untouched(whole, fill=7):
    ends = torch.stack([whole[0], whole[-1]]).float()
    return bool((ends == torch.full_like(ends, fill).to(whole.dtype).float()).all())


def close(got, want, tol, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3],
                           np.broadcast_to(tol, got.shape)[bad][:3])


# ---------------------------------------------------------------- norm

def norm(x, w, eps, residual=None, y=True, q=False, sums=True):
    rows, H = x.shape
    out = {}
    if residual is not None and sums:
        out["sum"], out["_sum"] = guarded(rows, H, torch.bfloat16)
    if y:
        out["y"], out["_y"] = guarded(rows, H, torch.bfloat16)
    if q:
        out["q"], out["_q"] = guarded(rows, H, FP8)
        out["scale"], out["_scale"] = guarded(rows, -(-H // 128), torch.float32)
    binding.moe_rms_norm(x, w, eps, residual=residual, **{n: t for n, t in out.items() if n[0] != "_"})
    torch.cuda.synchronize()
    assert all(untouched(t) for n, t in out.items() if n[0] == "_")
    return out


def check_norm(x, w, eps, residual, out):
    s, y = block.rms_norm(f64(x), None if residual is None else f64(residual), f64(w), eps)
    if "sum" in out:
        assert np.array_equal(f64(out["sum"]), s)
    if "y" in out:
        close(out["y"], y, np.abs(y) * (HALF + NORM) + 2.0 ** -133, "y")
    if "q" in out:
        codes = out["q"].view(torch.uint8).cpu().numpy()
        # rstd is common to a row: the codes are those of s w, times any power of two that keeps the
        # runs off the format's floor
        z = s * f64(w)
        want, _ = quantize_fp8(z * np.exp2(-np.floor(np.log2(np.abs(z).max(axis=1, keepdims=True)))))
        if w.dtype == torch.bfloat16:   # s w and the quotient have too few digits to be near a border
            assert np.array_equal(codes, want)
        else:                           # off by one code where the quotient is within 2^-21 of a border
            a, b = decode_e4m3(codes), decode_e4m3(want)
            assert (codes != want).mean() < 1e-3
            assert (np.abs(a - b) <= np.abs(b) * 2.0 ** -3 + 2.0 ** -9).all()
        amax = np.maximum.reduceat(np.abs(y), np.arange(0, y.shape[1], 128), axis=1)
        scale = np.maximum(amax, 2.0 ** -100) / 448.0
        close(out["scale"], scale, scale * (NORM + 2 * U), "scale")


SHAPES = [(1, 8), (3, 16), (1, 504), (5, 520), (66, 136), (257, 512), (2, 1024), (9, 1032), (7, 2064), (4, 2048), (1, 4096),
          (130, 4096), (3, 4112), (2, 8192), (3, 8208), (2, 16384), (2, 16400), (2, 32768), (1, 32784), (2, 65536)]


@pytest.mark.parametrize("rows,H", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
def test_norm(rows, H, residual, wtype):
    g = gen(rows * 31 + H)
    x = randn(g, rows, H)
    w = randn(g, H, dtype=wtype)
    r = randn(g, rows, H, scale=3.0) if residual else None
    out = norm(x, w, 1e-6, r, y=True, q=H % 16 == 0)
    check_norm(x, w, 1e-6, r, out)


@pytest.mark.parametrize("rows", [1, 4, 300])
@pytest.mark.parametrize("H", [16, 400, 4096])
def test_norm_outputs_do_not_depend_on_one_another(rows, H):
    g = gen(5)
    x, w, r = randn(g, rows, H), randn(g, H), randn(g, rows, H)
    both = norm(x, w, 1e-5, r, y=True, q=True)
    for y, q, sums in ((True, False, True), (False, True, False), (True, False, False)):
        one = norm(x, w, 1e-5, r, y=y, q=q, sums=sums)
        for n in one:
            if n[0] != "_":
                assert torch.equal(one[n].view(torch.uint8), both[n].view(torch.uint8)), n


@pytest.mark.parametrize("H", [64, 208, 400, 4096])
def test_norm_of_rows_at_every_magnitude(H):
    g = gen(6)
    x = torch.randn(40, H, generator=g)
    for i in range(40):
        x[i] *= 2.0 ** (-130 + 6.4 * i)
    x[3] = 0.0
    x = x.clamp(-3e38, 3e38).bfloat16().to(DEV)
    w = randn(g, H)
    for eps in (1e-6, 1e-30):
        out = norm(x, w, eps, None, y=True, q=False)
        check_norm(x, w, eps, None, out)
    live = [i for i in range(40) if i != 3]
    out = norm(x[live].contiguous(), w, 0.0, None, y=True, q=True)
    check_norm(x[live].contiguous(), w, 0.0, None, out)


def test_norm_runs_below_the_scale_floor():
    """Runs whose y, or whose s w, is below 2^-100 are quantised from y at the floor's scale."""
    g = gen(7)
    x = randn(g, 6, 512)
    x[0, 128:256] *= 2.0 ** -110          # y far below the floor
    x[1, 128:256] = 0.0
    x[2] *= 2.0 ** -120                   # s w below, y above (eps 0)
    x[3] *= 2.0 ** -40
    x[3, 256:384] *= 2.0 ** -62           # near the floor
    x[4] *= 2.0 ** -60
    x[4, :128] *= 2.0 ** -60
    w = randn(g, 512)
    out = norm(x, w, 0.0, None, y=True, q=True)
    _, y = block.rms_norm(f64(x), None, f64(w), 0.0)
    amax = np.maximum.reduceat(np.abs(y), np.arange(0, 512, 128), axis=1)
    scale = np.maximum(amax, 2.0 ** -100) / 448.0
    close(out["scale"], scale, scale * (NORM + 2 * U), "scale")
    back = f64(out["q"].float()) * np.repeat(f64(out["scale"]), 128, axis=1)
    # half a step of E4M3 relative, half its smallest step below 2^-6 of the scale's unit
    close(back, y, np.abs(y) * (2.0 ** -4 + 2 * NORM) + np.repeat(scale, 128, axis=1) * 2.0 ** -10 * 1.01, "q")


def test_norm_of_infinities_and_nan():
    g = gen(8)
    x, w = randn(g, 5, 512), randn(g, 512)
    x[1, 200] = float("inf")
    x[2, 3] = float("nan")
    x[3, 0] = float("-inf")
    x[3, 511] = float("inf")
    out = norm(x, w, 1e-6, None, y=True, q=True)
    s, y = block.rms_norm(f64(x), None, f64(w), 1e-6)
    got = f64(out["y"])
    assert np.array_equal(np.isnan(got), np.isnan(y))
    for i in (1, 3):
        assert np.isnan(y[i]).sum() == (1 if i == 1 else 2) and not np.nan_to_num(got[i]).any()
    codes, scale = out["q"].view(torch.uint8).cpu().numpy(), f64(out["scale"])
    bad = np.isnan(np.maximum.reduceat(y, np.arange(0, 512, 128), axis=1))
    assert np.array_equal(np.isnan(scale), bad)
    assert ((codes == 0x7F) == np.repeat(bad, 128, axis=1)).all()
    check_norm(x[[0, 4]].contiguous(), w, 1e-6, None, norm(x[[0, 4]].contiguous(), w, 1e-6, None, q=True))


def test_norm_of_zero_rows_without_eps_is_nan():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    x[1] = 1.0
    out = norm(x, w, 0.0, None, y=True, q=True)
    assert out["y"][0].isnan().all() and (out["y"][1] == 1.0).all()
    assert out["scale"][0].isnan().all() and (out["q"].view(torch.uint8)[0] == 0x7F).all()


@pytest.mark.parametrize("H", [512, 2064])
def test_norm_of_a_slice_of_wider_rows(H):
    g = gen(9)
    wide = randn(g, 37, H + 64)
    x, w, r = wide[:, :H], randn(g, H), randn(g, 37, H)
    check_norm(x, w, 1e-6, r, norm(x, w, 1e-6, r, y=True, q=True))
    check_norm(wide[:, 64:], w, 1e-6, None, norm(wide[:, 64:], w, 1e-6, None, y=True, q=True))


def test_norm_in_place():
    g = gen(10)
    for H in (400, 4096):
        x, w, r = randn(g, 9, H), randn(g, H), randn(g, 9, H)
        want = norm(x, w, 1e-6, r)
        a, b = x.clone(), r.clone()
        binding.moe_rms_norm(a, w, 1e-6, residual=b, sum=b, y=a)      # the stream and the branch
        assert torch.equal(b, want["sum"]) and torch.equal(a, want["y"])
        a, b = x.clone(), r.clone()
        binding.moe_rms_norm(a, w, 1e-6, residual=b, sum=a, y=b)
        assert torch.equal(a, want["sum"]) and torch.equal(b, want["y"])


# ---------------------------------------------------------------- its gradient

def check_norm_grad(s, w, eps, dy, dsum, dx, dw):
    S, W, D = f64(s), f64(w), f64(dy)
    want, wantw = block.rms_norm_grad(S, W, eps, D, None if dsum is None else f64(dsum))
    r = 1.0 / np.sqrt(np.mean(S * S, axis=1, keepdims=True) + eps)
    u, z = S * r, D * W
    if dx is not None:
        size = r * (np.abs(z) + 2 * np.abs(u) * np.mean(np.abs(z * u), axis=1, keepdims=True))
        size = size + (0.0 if dsum is None else np.abs(f64(dsum)))
        close(dx, want, np.abs(want) * HALF + size * 2 * NORM + 2.0 ** -133, "dx")
    if dw is not None:
        # chains: the rows of one wavefront, the wavefronts, the partial rows; u's own error
        chain = S.shape[0] / 512 + 1 + 4 + 32 + 16
        close(dw, wantw, np.sum(np.abs(D * u), axis=0) * (chain * U + NORM) + 2.0 ** -140, "dweight")


def norm_grad(s, w, eps, dy, dsum=None, want_dx=True, want_dw=True):
    rows, H = s.shape
    dx, dxw = guarded(rows, H, torch.bfloat16)
    dw = torch.full((H + 8,), 5.0, device=DEV)
    n = binding.moe_rms_norm_grad_workspace_bytes(rows, H)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN, if it is read unwritten
    binding.moe_rms_norm_grad(s, w, eps, dy, dx if want_dx else None, dw[:H] if want_dw else None, ws[:n], dsum=dsum)
    torch.cuda.synchronize()
    assert untouched(dxw) and (dw[H:] == 5.0).all() and (ws[n:] == 0xFF).all()
    return dx if want_dx else None, dw[:H] if want_dw else None


@pytest.mark.parametrize("rows,H", SHAPES + [(513, 64), (2100, 24), (1500, 4096)])
@pytest.mark.parametrize("beside", [False, True])
def test_norm_grad(rows, H, beside):
    g = gen(rows * 17 + H)
    wtype = torch.float32 if (rows + H // 8) % 2 else torch.bfloat16
    s, dy, w = randn(g, rows, H, scale=2.0), randn(g, rows, H), randn(g, H, dtype=wtype)
    dsum = randn(g, rows, H) if beside else None
    dx, dw = norm_grad(s, w, 1e-6, dy, dsum)
    check_norm_grad(s, w, 1e-6, dy, dsum, dx, dw)


@pytest.mark.parametrize("rows,H", [(5, 136), (1100, 512), (3, 8192)])
def test_norm_grad_of_one_output_alone(rows, H):
    g = gen(11)
    s, dy, w, dsum = randn(g, rows, H), randn(g, rows, H), randn(g, H), randn(g, rows, H)
    dx, dw = norm_grad(s, w, 1e-6, dy, dsum)
    assert torch.equal(norm_grad(s, w, 1e-6, dy, dsum, want_dw=False)[0], dx)
    assert torch.equal(norm_grad(s, w, 1e-6, dy, None, want_dx=False)[1], dw)
    out = torch.empty_like(s)
    binding.moe_rms_norm_grad(s, w, 1e-6, dy, out, None, None, dsum=dsum)      # no workspace
    assert torch.equal(out, dx)


def test_norm_grad_in_place_and_of_a_slice():
    g = gen(12)
    wide = randn(g, 21, 600)
    s, dy, w, dsum = wide[:, 8:520], randn(g, 21, 512), randn(g, 512), randn(g, 21, 512)
    dx, dw = norm_grad(s.contiguous(), w, 1e-6, dy, dsum)
    ws = torch.empty(binding.moe_rms_norm_grad_workspace_bytes(21, 512), dtype=torch.uint8, device=DEV)
    for t in (dy.clone(), dsum.clone()):
        d, e = (t, dsum) if torch.equal(t, dy) else (dy, t)
        out = torch.empty(512, device=DEV)
        binding.moe_rms_norm_grad(s, w, 1e-6, d, t, out, ws, dsum=e)
        assert torch.equal(t, dx) and torch.equal(out, dw)


@pytest.mark.parametrize("H", [64, 256, 512, 4096])
def test_norm_grad_of_extreme_rows(H):
    g = gen(13)
    s = torch.randn(12, H, generator=g)
    for i in range(12):
        s[i] *= 2.0 ** (-120 + 20 * i)
    s = s.bfloat16().to(DEV)
    # dy beside it, so that dx stays within bf16
    dy = randn(g, 12, H)
    for i in range(12):
        dy[i] *= 2.0 ** min(0, -60 + 20 * i)
    w = randn(g, H)
    dx, dw = norm_grad(s, w, 0.0, dy)
    check_norm_grad(s, w, 0.0, dy, None, dx, dw)
    z = torch.zeros(4, H, dtype=torch.bfloat16, device=DEV)       # zero rows: dx = dy w / sqrt(eps)
    dx, dw = norm_grad(z, w, 1e-6, dy[4:8].contiguous())
    check_norm_grad(z, w, 1e-6, dy[4:8].contiguous(), None, dx, dw)
    assert not dw.any()


def test_norm_without_rows():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    dw = torch.ones(64, device=DEV)
    binding.moe_rms_norm(e, w, 1e-6, y=e)
    binding.moe_rms_norm_grad(e, w, 1e-6, e, e, dw, None)
    torch.cuda.synchronize()
    assert not dw.any()


# ---------------------------------------------------------------- balance loss

def case(T, E, k, seed, dtype=torch.float32, cuts=None, scale=1.5):
    g = gen(seed)
    logits = randn(g, T, E, dtype=dtype, scale=scale)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).to(DEV) if T else \
        torch.empty(0, k, dtype=torch.int32, device=DEV)
    offsets = None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device=DEV)
    S = 1 if cuts is None else len(cuts) - 1
    return logits, ids, offsets, (torch.rand(S, generator=g) + 0.5).to(DEV), randn(g, T, E, dtype=dtype, scale=0.01)


def balance(logits, ids, offsets, dloss, add, score, grad=True):
    T, E = logits.shape
    S, k = dloss.shape[0], ids.shape[1]
    loss, counts = torch.full((S + 2,), 9.0, device=DEV), torch.full((S * E + 2,), 9, dtype=torch.int32, device=DEV)
    d, dw = guarded(T, E, logits.dtype)
    n = binding.moe_balance_loss_workspace_bytes(T, E, S)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    kw = dict(dloss=dloss, dlogits=d, add_to=add) if grad else {}
    if grad and d.data_ptr() % (16 if logits.dtype == torch.float32 else 8) == 0:
        pass
    binding.moe_balance_loss(logits, ids, loss[1:-1], counts[1:-1].view(S, E), ws, score=score, seq_offsets=offsets, **kw)
    torch.cuda.synchronize()
    assert loss[0] == 9.0 and loss[-1] == 9.0 and counts[0] == 9 and counts[-1] == 9 and untouched(dw)
    if grad:   # the gradient apart from the loss: the same bits
        d2 = torch.empty_like(d)
        binding.moe_balance_loss_grad(logits, k, counts[1:-1].view(S, E).clone(), dloss, d2, score=score,
                                      seq_offsets=offsets, add_to=add)
        assert torch.equal(d.view(torch.uint8), d2.view(torch.uint8))
    return loss[1:-1], counts[1:-1].view(S, E), d


def check_balance(logits, ids, offsets, dloss, add, score, out):
    l, cuts = f64(logits), None if offsets is None else offsets.cpu().tolist()
    I = ids.cpu().numpy()
    T, E = l.shape
    k = I.shape[1]
    loss, counts, d = out
    want, wantc = block.balance_loss(l, I, score, cuts)
    assert np.array_equal(counts.cpu().numpy(), wantc)
    p = block.shares(l, score)
    fin = np.where(np.isfinite(l), l, 0.0)
    tol = (np.minimum(np.ptp(fin, axis=1, keepdims=True), 104.0) + 32) * U if T else np.zeros((0, 1))
    g = block.balance_loss_grad(l, k, wantc, f64(dloss), score, cuts, None if add is None else f64(add))
    gtol = np.zeros((T, E))
    for s, (t0, t1) in enumerate(block.sequences(T, cuts)):
        n = t1 - t0
        if n == 0:
            assert f64(loss)[s] == 0.0
            continue
        c = np.abs(wantc[s] - (n * k // E))
        each = (p[t0:t1] * tol[t0:t1] * c).sum(1, keepdims=True)       # error of d
        lt = E / (k * n * n) * (2 * each.sum() + n * U * (n * k // E)) + np.abs(want[s]) * U + 1e-40
        assert abs(f64(loss)[s] - want[s]) <= lt, (s, f64(loss)[s], want[s], lt)
        f = abs(float(dloss[s])) * E / (k * n * n)
        dd = (p[t0:t1] * c).sum(1, keepdims=True)
        gtol[t0:t1] = f * p[t0:t1] * (2 * each + (c + dd) * (2 * tol[t0:t1] + 8 * U)) + f * 2.0 ** -120 * (c + dd)
    half = HALF if logits.dtype == torch.bfloat16 else U
    close(d, g, gtol + np.abs(g) * half + (0 if add is None else np.abs(f64(add)) * U) + 2.0 ** -133, "dlogits")


@pytest.mark.parametrize("T,E,k,cuts", [
    (1, 1, 1, None), (1, 2, 1, None), (3, 7, 3, None), (5, 8, 8, None), (64, 60, 6, None), (65, 64, 4, [0, 1, 65]),
    (100, 65, 2, [0, 30, 30, 99]), (130, 96, 6, [3, 20, 20, 20, 127]), (77, 128, 8, [0, 77]), (90, 129, 5, [0, 45, 90]),
    (300, 256, 6, [0, 0, 1, 2, 255, 256, 290]), (33, 257, 4, [0, 33]), (70, 512, 8, [10, 60]), (40, 513, 3, None),
    (41, 1024, 8, [0, 8, 16, 17, 41]), (1500, 16, 2, [0, 700, 1500]), (9000, 12, 3, [0, 8000, 8999, 9000])])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance(T, E, k, cuts, score, dtype):
    logits, ids, offsets, dloss, add = case(T, E, k, T * 7 + E, dtype, cuts)
    add = add if (T + E) % 2 else None
    check_balance(logits, ids, offsets, dloss, add, score, balance(logits, ids, offsets, dloss, add, score))


def test_balance_loss_alone_is_the_same():
    for T, E, k, cuts in ((300, 256, 6, [0, 100, 290]), (50, 33, 3, None)):
        logits, ids, offsets, dloss, add = case(T, E, k, 3, cuts=cuts)
        a, b = balance(logits, ids, offsets, dloss, add, "softmax"), balance(logits, ids, offsets, dloss, None, "softmax", False)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_of_many_sequences(score):
    """More sequences than lanes that look for them, most of them empty or of one token."""
    g = np.random.default_rng(4)
    cuts = np.sort(g.integers(0, 700, size=5000)).tolist()
    logits, ids, offsets, dloss, add = case(720, 24, 4, 5, cuts=cuts)
    check_balance(logits, ids, offsets, dloss, add, score, balance(logits, ids, offsets, dloss, add, score))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [20, 96, 256, 600])
def test_balance_of_excluded_experts_and_extreme_logits(score, E):
    logits, ids, offsets, dloss, add = case(40, E, 4, 6, cuts=[0, 18, 40])
    logits[0, ::2] = float("-inf")
    logits[1] = float("-inf")
    logits[2, 5] = float("nan")
    logits[3] = float("nan")
    logits[4] -= 1000.0
    logits[5] -= 60.0
    logits[6] -= 39.9
    logits[7] -= 100.0
    logits[7, 3] = 50.0
    logits[8, 4] = float("inf")
    logits[9, 4] = logits[9, 7] = float("inf")
    logits[10] = torch.finfo(torch.float32).min
    logits[11, :] = 0.0
    logits[12] += 200.0
    logits[13, 1] = torch.finfo(torch.float32).max
    check_balance(logits, ids, offsets, dloss, None, score, balance(logits, ids, offsets, dloss, None, score))


def test_balance_of_an_even_load_has_no_gradient():
    T, E, k = 4096, 64, 4
    logits = randn(gen(7), T, E, dtype=torch.float32)
    ids = torch.arange(T * k, dtype=torch.int32).remainder(E).view(T, k).to(DEV)
    for score in ("softmax", "sigmoid"):
        loss, counts, d = balance(logits, ids, None, torch.ones(1, device=DEV), None, score)
        assert (counts == T * k // E).all() and not d.any() and abs(float(loss[0]) - 1.0) <= 2 * U


def test_balance_ids_outside_the_experts_count_nowhere():
    logits, ids, offsets, dloss, add = case(30, 16, 3, 8, cuts=[0, 20, 30])
    ids[::3, 1] = -1
    ids[1, 0], ids[2, 0] = 16, 2 ** 31 - 1
    check_balance(logits, ids, offsets, dloss, None, "softmax", balance(logits, ids, offsets, dloss, None, "softmax"))


def test_balance_of_the_same_expert_in_every_slot():
    logits, ids, offsets, dloss, _ = case(2000, 16, 4, 9)
    ids[:] = 5
    check_balance(logits, ids, offsets, dloss, None, "softmax", balance(logits, ids, offsets, dloss, None, "softmax"))


def test_balance_in_place_and_without_tokens():
    logits, ids, offsets, dloss, add = case(130, 96, 6, 10, cuts=[0, 50, 120])
    want = balance(logits, ids, offsets, dloss, add, "softmax")[2]
    counts, ws = torch.empty(2, 96, dtype=torch.int32, device=DEV), torch.empty(4096, dtype=torch.uint8, device=DEV)
    loss = torch.empty(2, device=DEV)
    for place in ("add", "logits"):
        l, a = logits.clone(), add.clone()
        binding.moe_balance_loss(l, ids, loss, counts, ws, seq_offsets=offsets, dloss=dloss, add_to=a,
                                 dlogits=a if place == "add" else l)
        assert torch.equal(a if place == "add" else l, want)
    loss.fill_(5.0), counts.fill_(5)
    e = torch.empty(0, 96, device=DEV)
    binding.moe_balance_loss(e, torch.empty(0, 6, dtype=torch.int32, device=DEV), loss, counts, None,
                             seq_offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    binding.moe_balance_loss_grad(e, 6, counts, dloss, e, seq_offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert not loss.any() and not counts.any()


def test_balance_rows_that_are_not_on_16_bytes():
    logits, ids, offsets, dloss, add = case(70, 64, 4, 11, cuts=[0, 70])
    want = balance(logits, ids, offsets, dloss, add, "softmax")
    flat = torch.empty(70 * 64 + 1, device=DEV)
    shifted = flat[1:].view(70, 64)
    shifted.copy_(logits)
    got = balance(shifted, ids, offsets, dloss, add, "softmax")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- adapters

def group(ids, L):
    t = torch.tensor(np.asarray(ids), dtype=torch.int32, device=DEV)
    M = t.numel()
    offsets, rows = (torch.full((n + 2,), 77, dtype=torch.int32, device=DEV) for n in (L + 1, M))
    binding.moe_lora_group(t, L, offsets[1:-1], rows[1:-1])
    torch.cuda.synchronize()
    assert offsets[0] == 77 and offsets[-1] == 77 and rows[0] == 77 and rows[-1] == 77
    return offsets[1:-1].clone(), rows[1:-1].clone()


@pytest.mark.parametrize("M,L", [(0, 3), (1, 1), (5, 2), (63, 64), (64, 1), (65, 7), (512, 64), (1000, 1024), (1025, 700),
                                 (1024, 3), (1026, 3), (8191, 8), (20000, 300), (70000, 895), (300000, 5), (400001, 900)])
def test_lora_group(M, L):
    r = np.random.default_rng(M + L)
    for ids in (r.integers(-1, L, size=M), np.full(M, L - 1), np.full(M, -1), np.sort(r.integers(-2, L + 2, size=M)),
                r.integers(-2 ** 31, 2 ** 31, size=M)):
        offsets, rows = group(ids, L)
        want = block.lora_group(ids, L)
        assert np.array_equal(offsets.cpu().numpy(), want[0]) and np.array_equal(rows.cpu().numpy(), want[1])


def lora(M, N, K, R, L, ids, seed, dtype, base=True, scaling=True):
    g = gen(seed)
    x, a, b = randn(g, M, K), randn(g, L, R, K, scale=K ** -0.5), randn(g, L, N, R, scale=R ** -0.5)
    s = (torch.rand(L, generator=g) + 0.25).to(DEV) if scaling else None
    return x, a, b, s, randn(g, M, N, dtype=dtype) if base else None


def run_lora(x, a, b, s, ids, base, dtype, y=None):
    M, K = x.shape
    L, R, _ = a.shape
    N = b.shape[1]
    offsets, rows = group(ids, L)
    whole = None
    if y is None:
        y, whole = guarded(M, N, dtype)
        if y.data_ptr() % 16:   # the row in front of it is not a multiple of 16 bytes
            pad = 16 // y.element_size()
            flat = torch.full((M * N + 2 * pad,), 7.0, device=DEV).to(dtype)
            y, whole = flat[pad:-pad].view(M, N), torch.stack([flat[:pad], flat[-pad:]])
            tail = flat
    n = binding.moe_lora_add_workspace_bytes(M, N, K, R, L)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    binding.moe_lora_add(x, a, b, s, offsets, rows, base, y, ws)
    torch.cuda.synchronize()
    if whole is not None and whole.shape[0] == M + 2:
        assert untouched(whole)
    elif whole is not None:
        assert (tail[:pad].float() == 7).all() and (tail[-pad:].float() == 7).all()
    return y


def check_lora(x, a, b, s, ids, base, y):
    K, R = x.shape[1], a.shape[1]
    want, split, inner = block.lora_add(f64(x), f64(a), f64(b), None if s is None else f64(s), ids,
                                        None if base is None else f64(base))
    half = HALF if y.dtype == torch.bfloat16 else U
    # the inner sums' parts leave 2^-17 of them for bf16 results; all 24 bits for fp32 ones
    part = 2.0 ** -17 if y.dtype == torch.bfloat16 else 0.0
    tol = split * (part + (R + 8) * 2 * U) + inner * (K / 128 + 48) * 2 * U
    tol = tol + np.abs(want) * half + (0.0 if base is None else np.abs(f64(base)) * U)
    close(y, want, tol, "y")


LORA = [(1, 1, 8, 8, 1), (1, 64, 64, 16, 3), (2, 17, 24, 8, 2), (16, 256, 128, 16, 1), (17, 257, 136, 24, 4), (33, 1003, 264, 8, 5),
        (40, 48, 2064, 40, 3), (100, 520, 512, 64, 6), (70, 96, 1024, 72, 2), (50, 272, 256, 128, 3), (37, 80, 192, 136, 2),
        (65, 304, 320, 256, 2), (300, 512, 4096, 16, 64), (200, 64, 72, 32, 70), (1, 4096, 4096, 16, 8), (3, 96, 65536, 8, 2),
        (1500, 600, 200, 16, 4), (1500, 600, 136, 32, 4), (1500, 530, 1032, 64, 3), (1300, 1000, 72, 8, 2), (600, 2048, 64, 16, 40),
        (2100, 2049, 128, 200, 5), (900, 4096, 64, 24, 300), (10, 300, 4096, 64, 2), (5, 70, 2064, 40, 2)]


@pytest.mark.parametrize("M,N,K,R,L", LORA)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lora_add(M, N, K, R, L, dtype):
    r = np.random.default_rng(M + N + R)
    ids = r.integers(-1, L, size=M) if M > 2 else np.full(M, L - 1)
    x, a, b, s, base = lora(M, N, K, R, L, ids, M * 3 + K, dtype)
    check_lora(x, a, b, s, ids, base, run_lora(x, a, b, s, ids, base, dtype))


@pytest.mark.parametrize("M,N,K,R,L", [(6500, 72, 64, 16, 1), (7000, 100, 72, 40, 3), (8191, 64, 136, 64, 8), (6300, 130, 1032, 24, 2),
                                       (20000, 65, 64, 8, 5), (9000, 33, 8, 64, 9), (7777, 264, 520, 32, 4), (40000, 16, 64, 48, 200),
                                       (3300, 96, 200, 72, 2), (5000, 80, 1032, 256, 3), (4000, 70, 2064, 128, 40)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [False, True])
def test_lora_add_many_rows(M, N, K, R, L, dtype, packed):
    r = np.random.default_rng(M + N + R)
    ids = r.integers(-1, L, size=M)
    if packed:      # requests of different lengths, in the batch's order
        cuts = np.sort(r.integers(0, M, size=2 * L))
        ids = r.integers(-1, L, size=2 * L + 1)[np.searchsorted(cuts, np.arange(M), side="right")]
    x, a, b, s, base = lora(M, N, K, R, L, ids, M + K, dtype)
    y = run_lora(x, a, b, s, ids, base, dtype)
    check_lora(x, a, b, s, ids, base, y)
    place = base.clone()
    assert torch.equal(run_lora(x, a, b, s, ids, place, dtype, place), y)
    check_lora(x, a, b, s, ids, None, run_lora(x, a, b, s, ids, None, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 7, 130, 600])
def test_lora_base_in_place_and_without(M, dtype):
    r = np.random.default_rng(M)
    ids = r.integers(-1, 3, size=M)
    x, a, b, s, base = lora(M, 200, 160, 16, 3, ids, 1, dtype)
    want = run_lora(x, a, b, s, ids, base, dtype)
    y = base.clone()
    assert torch.equal(run_lora(x, a, b, s, ids, y, dtype, y), want)
    check_lora(x, a, b, s, ids, None, run_lora(x, a, b, s, ids, None, dtype))
    check_lora(x, a, b, None, ids, base, run_lora(x, a, b, None, ids, base, dtype))


def test_lora_rows_without_an_adapter_are_the_base():
    x, a, b, s, base = lora(90, 72, 64, 8, 2, None, 2, torch.bfloat16)
    base[3, 5], base[4, 0] = float("nan"), float("inf")
    ids = np.full(90, -1)
    assert torch.equal(run_lora(x, a, b, s, ids, base, torch.bfloat16).view(torch.int16), base.view(torch.int16))
    assert not run_lora(x, a, b, s, ids, None, torch.bfloat16).any()


def test_lora_unused_adapters_and_other_rows_do_not_matter():
    """Infinities and NaN in adapters without rows, and in the rows of other requests."""
    ids = np.array([1] * 5 + [-1] * 3 + [1] * 12 + [3] * 9)
    x, a, b, s, base = lora(29, 96, 128, 16, 5, ids, 3, torch.float32)
    want = run_lora(x, a, b, s, ids, base, torch.float32)
    a[0], b[2], s[4] = float("nan"), float("inf"), float("nan")
    x[6] = float("nan")
    assert torch.equal(run_lora(x, a, b, s, ids, base, torch.float32), want)
    x[25, 3] = float("nan")
    got = run_lora(x, a, b, s, ids, base, torch.float32)
    assert got[25].isnan().all() and torch.equal(got[:25], want[:25]) and torch.equal(got[26:], want[26:])


def test_lora_infinite_inner_sums_stay_infinite():
    ids = np.zeros(2, int)
    x, a, b, s, base = lora(2, 32, 64, 8, 1, ids, 4, torch.float32)
    x[0, 0] = float("inf")
    a[0, :, 0] = 1.0
    b[0] = b[0].abs() + 0.5
    y = run_lora(x, a, b, s, ids, base, torch.float32)
    assert (y[0] == float("inf")).all() and y[1].isfinite().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [61, 700, 7000])
def test_lora_on_slices_of_wider_rows(dtype, M):
    """The adapters of one of several projections whose results share rows."""
    r = np.random.default_rng(5)
    ids = r.integers(-1, 4, size=M)
    x, a, b, s, _ = lora(M, 136, 128, 16, 4, ids, 6, dtype)
    wide_x, wide = randn(gen(7), M, 200), randn(gen(8), M, 408, dtype=dtype)
    xs, ys = wide_x[:, 64:192], wide[:, 136:272]
    before = wide.clone()
    check_lora(xs, a, b, s, ids, before[:, 136:272], run_lora(xs, a, b, s, ids, ys, dtype, ys))
    assert torch.equal(wide[:, :136], before[:, :136]) and torch.equal(wide[:, 272:], before[:, 272:])
    odd = randn(gen(9), M, 411, dtype=dtype)      # rows on no 16 bytes
    ys, base = odd[:, :136], before[:, :136]
    check_lora(xs, a, b, s, ids, base, run_lora(xs, a, b, s, ids, base, dtype, ys))


def test_lora_without_rows():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    a, b = randn(gen(1), 2, 8, 64), randn(gen(2), 2, 64, 8)
    offsets, rows = group(np.empty(0, int), 2)
    binding.moe_lora_add(e, a, b, None, offsets, rows, None, e.clone(), None)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- together

def _block(seed, T=90, E=32, k=4, H=512, I=256, N=384, L=3, R=16):
    """Inputs of layer.run_block_fp8 and their float64 values."""
    r = np.random.default_rng(seed)
    g = gen(seed)

    def fp8(n, K, lead=()):
        q = torch.from_numpy(quantize_fp8(r.normal(size=(int(np.prod(lead, dtype=int)) * n, K)))[0]).view(*lead, n, K)
        s = (r.random((*lead, -(-n // 128), -(-K // 128))) + 0.5) * 400.0 / 448.0 / 100.0 / K ** 0.5
        return q.to(DEV), torch.from_numpy(s.astype(np.float32)).to(DEV)

    dev = dict(x=randn(g, T, H), residual=randn(g, T, H), norm=(1 + 0.2 * torch.randn(H, generator=g)).to(DEV))
    for name, n in (("router", E), ("shared", N)):
        dev[name], dev[name + "_s"] = fp8(n, H)
        dev[name + "_a"], dev[name + "_b"] = randn(g, L, R, H, scale=H ** -0.5), randn(g, L, n, R, scale=R ** -0.5)
    dev["w1"], dev["w1_s"] = fp8(2 * I, H, (E,))
    dev["w2"], dev["w2_s"] = fp8(H, I, (E,))
    dev["adapter"] = torch.from_numpy(r.integers(-1, L, size=T).astype(np.int32)).to(DEV)
    dev["scaling"] = torch.from_numpy((r.random(L) + 0.5).astype(np.float32)).to(DEV)
    return dev, (T, E, k, H, I, N, L, R)


def test_block_runs_its_parts_together():
    """norm -> FP8 router and projection, each with adapters -> routed experts, against the parts' oracles."""
    from mxfp4_routed_expert_route_amd import layer
    from oracle.fp8 import gemm_fp8, route_scored
    dev, (T, E, k, H, I, N, L, R) = _block(3)
    b = layer.BlockBuffers.allocate_fp8(T, E, k, H, I, N, L, R)
    how = dict(score="sigmoid", scale=1.5)
    layer.run_block_fp8(dev, b, 10.0, **how)
    torch.cuda.synchronize()
    check_norm(dev["x"], dev["norm"], 1e-6, dev["residual"], dict(sum=b.sum, y=b.h, q=b.hq, scale=b.hs))
    ids = dev["adapter"].cpu().numpy()
    for name, y in (("router", b.logits), ("shared", b.shared)):
        base, _ = gemm_fp8(b.hq.view(torch.uint8).cpu().numpy(), f64(b.hs), dev[name].cpu().numpy(), f64(dev[name + "_s"]))
        want = block.lora_add(f64(b.h), f64(dev[name + "_a"]), f64(dev[name + "_b"]), f64(dev["scaling"]), ids, base)[0]
        # bf16: the product rounds once, its adapters' sum again, of the rounded value
        tol = 4 * HALF if y.dtype == torch.bfloat16 else 2.0 ** -14
        assert np.abs(f64(y) - want).max() <= tol * np.abs(want).max()
    want = route_scored(f64(b.logits), k, score="sigmoid", scale=1.5)
    assert np.array_equal(b.layer.topk_ids.cpu().numpy(), want[0])
    alone = layer.LayerBuffers.allocate_fp8(T, E, k, H, I)
    layer.run_layer_fp8(dict(dev, x=b.h, logits=b.logits), alone, 10.0, **how)
    assert torch.equal(alone.y, b.layer.y) and b.layer.y.isfinite().all() and b.layer.y.any()
    # the next block's stream takes this one's result; without adapters the call is the dense products alone
    dev2 = dict(dev, x=b.layer.y, residual=b.sum, adapter=None)
    b2 = layer.BlockBuffers.allocate_fp8(T, E, k, H, I, N)
    layer.run_block_fp8(dev2, b2, 10.0, **how)
    y = torch.empty_like(b2.shared)
    binding.moe_gemm_fp8(b2.hq, b2.hs, dev["shared"], dev["shared_s"], y)
    assert torch.equal(y, b2.shared) and b2.layer.y.isfinite().all()


def test_router_training_step_against_differences():
    """The balance loss's gradient through the router's product and the norm, against differences of the
    loss in 64 bits."""
    T, H, E, k, eps = 48, 64, 12, 2, 1e-5
    g = gen(17)
    x, w, router = randn(g, T, H), (1 + 0.2 * torch.randn(H, generator=g)).to(DEV), randn(g, E, H, scale=0.2)
    cuts = torch.tensor([0, 20, 45], dtype=torch.int32, device=DEV)
    dloss = torch.tensor([0.7, 1.3], device=DEV)
    h = torch.empty_like(x)
    binding.moe_rms_norm(x, w, eps, y=h)
    logits = (h.float() @ router.float().t()).contiguous()
    ids, weights = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    binding.moe_route_scored(logits, k, ids, weights)
    loss, counts = torch.empty(2, device=DEV), torch.empty(2, E, dtype=torch.int32, device=DEV)
    ws = torch.empty(binding.moe_balance_loss_workspace_bytes(T, E, 2), dtype=torch.uint8, device=DEV)
    dlogits = torch.empty_like(logits)
    binding.moe_balance_loss(logits, ids, loss, counts, ws, seq_offsets=cuts, dloss=dloss, dlogits=dlogits)
    scale = 2.0 ** 10      # dh in bf16, far from its smallest values
    dh = (dlogits @ router.float() * scale).bfloat16()
    dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
    nws = torch.empty(binding.moe_rms_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    binding.moe_rms_norm_grad(x, w, eps, dh, dx, dw, nws)

    X, W, Q, I, C = f64(x), f64(w), f64(router), ids.cpu().numpy(), cuts.cpu().tolist()

    def total(X, W):
        return (block.balance_loss(block.rms_norm(X, None, W, eps)[1] @ Q.T, I, "softmax", C)[0] * f64(dloss)).sum()

    r = np.random.default_rng(1)
    for _ in range(6):      # along random directions of x and of the weight
        u, v = r.normal(size=X.shape), r.normal(size=W.shape)
        d = 1e-5
        by_x = (total(X + d * u, W) - total(X - d * u, W)) / (2 * d) * scale
        by_w = (total(X, W + d * v) - total(X, W - d * v)) / (2 * d) * scale
        # h, dh and dx are rounded to bf16: three half steps of each term, and as much for h in the logits
        assert abs((f64(dx) * u).sum() - by_x) <= 6 * HALF * np.abs(f64(dx) * u).sum()
        assert abs((f64(dw) * v).sum() - by_w) <= 6 * HALF * np.abs(f64(dw) * v).sum()


# ---------------------------------------------------------------- streams and graphs

def _all_calls(seed):
    """One call of every operator; returns a function that makes them and their outputs."""
    g = gen(seed)
    rows, H, E, k, L, R, N = 70, 1024, 64, 4, 5, 16, 320
    x, r, w = randn(g, rows, H), randn(g, rows, H), randn(g, H)
    out = dict(sum=torch.empty_like(x), y=torch.empty_like(x), q=torch.empty(rows, H, dtype=FP8, device=DEV),
               scale=torch.empty(rows, 8, device=DEV), dx=torch.empty_like(x), dw=torch.empty(H, device=DEV),
               loss=torch.empty(3, device=DEV), counts=torch.empty(3, E, dtype=torch.int32, device=DEV))
    nws = torch.empty(binding.moe_rms_norm_grad_workspace_bytes(rows, H), dtype=torch.uint8, device=DEV)
    logits, ids, offsets, dloss, add = case(rows, E, k, seed, cuts=[0, 20, 50, 66])
    out["dlogits"], out["dlogits2"] = torch.empty_like(logits), torch.empty_like(logits)
    bws = torch.empty(binding.moe_balance_loss_workspace_bytes(rows, E, 3), dtype=torch.uint8, device=DEV)
    a, b = randn(g, L, R, H, scale=0.03), randn(g, L, N, R, scale=0.25)
    adapter = torch.randint(-1, L, (rows,), generator=g, dtype=torch.int32).to(DEV)
    base = randn(g, rows, N)
    out.update(at=torch.empty(L + 1, dtype=torch.int32, device=DEV), order=torch.empty(rows, dtype=torch.int32, device=DEV),
               z=torch.empty_like(base))
    lws = torch.empty(binding.moe_lora_add_workspace_bytes(rows, N, H, R, L), dtype=torch.uint8, device=DEV)

    def go(stream=None):
        binding.moe_rms_norm(x, w, 1e-6, residual=r, sum=out["sum"], y=out["y"], q=out["q"], scale=out["scale"], stream=stream)
        binding.moe_rms_norm_grad(out["sum"], w, 1e-6, out["y"], out["dx"], out["dw"], nws, stream=stream)
        binding.moe_balance_loss(logits, ids, out["loss"], out["counts"], bws, seq_offsets=offsets, dloss=dloss,
                                 dlogits=out["dlogits"], add_to=add, stream=stream)
        binding.moe_balance_loss_grad(logits, k, out["counts"], dloss, out["dlogits2"], seq_offsets=offsets, stream=stream)
        binding.moe_lora_group(adapter, L, out["at"], out["order"], stream=stream)
        binding.moe_lora_add(out["y"], a, b, None, out["at"], out["order"], base, out["z"], lws, stream=stream)

    return go, out


def _bits(out):
    return {n: t.view(torch.uint8).clone() for n, t in out.items()}


def test_captured_calls_replay_the_eager_results():
    go, out = _all_calls(21)
    go()
    torch.cuda.synchronize()
    want = _bits(out)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for i in range(5):
        for t in out.values():
            t.view(torch.uint8).fill_(0xA5)
        if i % 2:
            go()
            torch.cuda.synchronize()
            for t in out.values():
                t.view(torch.uint8).fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        got = _bits(out)
        assert all(torch.equal(got[n], want[n]) for n in want), [n for n in want if not torch.equal(got[n], want[n])]


def test_calls_on_two_streams_at_once():
    runs = [_all_calls(30 + i) for i in range(2)]
    want = []
    for go, out in runs:
        go()
        torch.cuda.synchronize()
        want.append(_bits(out))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (go, _), s in zip(runs, streams):
            go(s)
    torch.cuda.synchronize()
    for (_, out), w in zip(runs, want):
        got = _bits(out)
        assert all(torch.equal(got[n], w[n]) for n in w)


def test_calls_are_deterministic():
    go, out = _all_calls(40)
    go()
    torch.cuda.synchronize()
    want = _bits(out)
    for _ in range(10):
        go()
        torch.cuda.synchronize()
        got = _bits(out)
        assert all(torch.equal(got[n], want[n]) for n in want)

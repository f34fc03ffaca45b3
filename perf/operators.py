"""Measured cases of the FP8 expert path: scored routing, activation quantisation, the
block-scaled FP8 product, and the grouped expert FFN over block-scaled FP8 weights.

Formats.  FP8 is OCP E4M3 (largest value 448).  An activation row is cut into runs of 128
elements, each with one fp32 scale; a weight matrix into 128 x 128 blocks, each with one
fp32 scale; the last run or block of a row may be shorter.

  route     scores s = softmax(l) or sigmoid(l) of the router logits; keys s + bias; with
            groups, the experts of the groups with the largest group keys (the group's
            largest key, or the sum of its two largest); the k largest keys, ties to the
            lower index; weights s of the chosen, renormalised or not, times a factor.
  quantize  per run: a = max(max |x|, 2^-100), scale = a / 448, q = E4M3(448 x / a).
  gemm      y[m][n] = sum over runs b of xs[m][b] ws[n / 128][b] (xq[m] . wq[n]) over run b.
  ffn       rows grouped by expert: x quantised, gate|up product, clamped SwiGLU, h quantised
            from fp32, second product; y in expert-major order.

With `own` false, run() computes them with elementary torch operations; with `own` true it
calls the library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
FP8 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100
LIMIT = 10.0
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _route(name, T, E, k, score, groups, topk_groups, group_top, bias, renorm, scale, bf16, grouped):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, groups=groups, topk_groups=topk_groups,
                group_top=group_top, bias=bias, renorm=renorm, scale=scale, bf16=bf16, grouped=grouped)


def _gemm(name, M, N, K, f32):
    return dict(name=name, op="gemm", M=M, N=N, K=K, f32=f32)


def _ffn(name, T, E, k, H, I, skew):
    return dict(name=name, op="ffn", T=T, E=E, k=k, H=H, I=I, skew=skew)


def listed():
    return [
        # one stream's verify step (1 + 7 tokens): sigmoid scores with a balance bias and
        # expert groups, through the call that also groups the rows by expert
        _route("route-verify", 8, 256, 6, "sigmoid", 8, 4, 2, True, True, 2.5, False, True),
        # a long prompt batch, softmax over all experts with a balance bias
        _route("route-prompt", 8191, 256, 6, "softmax", 1, 1, 1, True, False, 1.0, False, False),
        # activations ahead of a product: a verify step, a prompt batch
        dict(name="quantize-verify", op="quantize", rows=8, K=4096),
        dict(name="quantize-prompt", op="quantize", rows=8191, K=4096),
        # one token through a dense layer (decode)
        _gemm("gemm-token", 1, 4096, 4096, False),
        # odd sizes: a few dozen rows, N no multiple of anything, a short last run of K, fp32 out
        _gemm("gemm-odd", 77, 1003, 2064, True),
        # 64 streams of 8 tokens
        _gemm("gemm-burst", 512, 4096, 2048, False),
        # a long prompt batch
        _gemm("gemm-prompt", 8191, 4096, 4096, False),
        # the routed experts: verify step (fewer rows than experts), burst (12 rows an expert),
        # prompt chunk (48 rows an expert), skewed load (a few experts hold most rows)
        _ffn("ffn-verify", 8, 256, 6, 4096, 2048, False),
        _ffn("ffn-burst", 512, 256, 6, 4096, 2048, False),
        _ffn("ffn-prefill", 2048, 256, 6, 4096, 2048, False),
        _ffn("ffn-skewed", 8191, 256, 6, 4096, 2048, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "ffn"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(1, -(-8 // groups)), 256 // groups)
        topk_groups = rng.randint(max(1, (groups + 1) // 2), groups)
        k = rng.randint(1, min(8, topk_groups * (E // groups)))
        case = _route("", _log(rng, 1, 8191), E, k, rng.choice(["softmax", "sigmoid"]), groups, topk_groups,
                      rng.choice([1, 2]), rng.random() < 0.6, rng.random() < 0.6, rng.choice([1.0, 2.5]),
                      rng.random() < 0.3, rng.random() < 0.5)
    elif op == "quantize":
        case = dict(name="", op="quantize", rows=_log(rng, 1, 8191), K=16 * _log(rng, 1, 256))
    elif op == "gemm":
        N = _log(rng, 1, 4096)
        case = _gemm("", _log(rng, 1, 8191), N, 16 * _log(rng, 1, 256), rng.random() < 0.3)
    else:
        E = _log(rng, 4, 256)
        case = _ffn("", _log(rng, 1, 4096), E, rng.randint(1, min(6, E)), 128 * _log(rng, 1, 32),
                    128 * _log(rng, 1, 16), rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _blocks(n):
    return -(-n // BLOCK)


def _weights(g, n, K, E=None):
    """E4M3 codes of normal weights with their block scales, sized so that W has unit-variance products."""
    lead = () if E is None else (E,)
    w = torch.empty(lead + (n, K), dtype=torch.uint8, device=DEV)
    flat = w.view(-1, K)
    step = max(1, (1 << 25) // K)
    for r in range(0, flat.shape[0], step):
        part = flat[r:r + step]
        v = torch.randn(part.shape, device=DEV, generator=g)
        part.copy_((v * 90.0).clamp_(-448.0, 448.0).to(FP8).view(torch.uint8))
    s = torch.rand(lead + (_blocks(n), _blocks(K)), device=DEV, generator=g) + 0.5
    return w, s / (90.0 * math.sqrt(K))


def _rank_bias(E, g):
    rank = torch.randperm(E, device=DEV, generator=g) + 1
    return -2.0 * torch.log(rank.float())


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn(T, E, device=DEV, generator=g)
        s["logits"] = logits.bfloat16() if case["bf16"] else logits
        s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g) if case["bias"] else None
    elif op == "quantize":
        # activations with a few large channels, as hidden states have
        rows, K = case["rows"], case["K"]
        gain = torch.exp(torch.randn(K, device=DEV, generator=g) * 0.7)
        s["x"] = (torch.randn(rows, K, device=DEV, generator=g) * gain).bfloat16()
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        x = torch.randn(M, K, device=DEV, generator=g).bfloat16()
        q, sc = _quantize_plain(x)
        s["xq"], s["xs"] = q.view(torch.uint8), sc
        s["w"], s["ws"] = _weights(g, N, K)
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        logits = torch.randn(T, E, device=DEV, generator=g)
        if case["skew"]:
            logits = logits + _rank_bias(E, g)
        ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        counts, offsets, gather, _ = _group_plain(ids, E)
        s.update(x=torch.randn(T, H, device=DEV, generator=g).bfloat16(), counts=counts, offsets=offsets,
                 gather=gather, host_counts=counts.tolist())
        s["w1"], s["w1s"] = _weights(g, 2 * I, H, E)
        s["w2"], s["w2s"] = _weights(g, H, I, E)
    return s


# ---------------------------------------------------------------- plain forms

def _group_plain(ids, E):
    flat = ids.reshape(-1)
    gather = torch.sort(flat, stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    scatter = torch.empty_like(gather)
    scatter[gather] = torch.arange(gather.numel(), device=gather.device)
    return tuple(t.to(torch.int32) for t in (counts, offsets, gather, scatter))


def _bitmatrix_plain(ids, E):
    words = (E + 31) // 32
    bm = torch.zeros(ids.shape[0], words, dtype=torch.int64, device=ids.device)
    bm.scatter_add_(1, ids // 32, torch.ones_like(ids) << (ids % 32))
    return bm.to(torch.int32)


def _route_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    # keys in 64 bits: experts whose scores are closer than fp32 tells apart are ordered too
    l = s["logits"].double()
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        grouped = key.view(T, c["groups"], -1)
        best = torch.sort(grouped, dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        live = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(live[:, :, None], grouped, -math.inf).view(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = [ids.to(torch.int32), (w * c["scale"]).float()]
    if c["grouped"]:
        out += [_bitmatrix_plain(ids, E), *_group_plain(ids, E)]
    return out


def _quantize_plain(x):
    rows, K = x.shape
    nb = _blocks(K)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - K)).view(rows, nb, BLOCK)
    a = v.abs().amax(2, keepdim=True).clamp_min(FLOOR)
    # quotients in 64 bits: many lie on the border between two codes
    q = (v.double() * 448.0 / a.double()).float().to(FP8).view(rows, nb * BLOCK)[:, :K].contiguous()
    return q, (a.double() / 448.0).float().squeeze(2)


def _dequant_weights(w, ws):
    n, K = w.shape
    full = ws.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :K]
    return w.view(FP8).float() * full


def _dequant_rows(q, sc):
    return q.view(FP8).float() * sc.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _gemm_plain(s):
    y = _dequant_rows(s["xq"], s["xs"]) @ _dequant_weights(s["w"], s["ws"]).t()
    return y if s["case"]["f32"] else y.bfloat16()


def _ffn_plain(s):
    c = s["case"]
    k, H, I = c["k"], c["H"], c["I"]
    x = _dequant_rows(*_quantize_plain(s["x"]))
    y = torch.empty(s["gather"].numel(), H, dtype=torch.bfloat16, device=DEV)
    begin = 0
    for e, n in enumerate(s["host_counts"]):
        if n == 0:
            continue
        rows = x[s["gather"][begin:begin + n].long() // k]
        gu = rows @ _dequant_weights(s["w1"][e], s["w1s"][e]).t()
        gate = gu[:, :I].clamp(max=LIMIT)
        h = gate / (1.0 + torch.exp(-gate)) * gu[:, I:].clamp(-LIMIT, LIMIT)
        h = _dequant_rows(*_quantize_plain(h))
        y[begin:begin + n] = (h @ _dequant_weights(s["w2"][e], s["w2s"][e]).t()).bfloat16()
        begin += n
    return y


# ---------------------------------------------------------------- one pass

def _buffers(s):
    """The outputs and workspace that a program keeps from call to call."""
    from mxfp4_routed_expert_route_amd import binding
    c = s["case"]
    i32 = dict(dtype=torch.int32, device=DEV)
    b = {}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        b["ids"] = torch.empty(T, k, **i32)
        b["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        if c["grouped"]:
            b["bitmatrix"] = torch.empty(T, (E + 31) // 32, **i32)
            b["counts"], b["offsets"] = torch.empty(E, **i32), torch.empty(E + 1, **i32)
            b["gather"], b["scatter"] = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
            b["ws"] = torch.empty(binding.moe_workspace_bytes(T, E, k, 128, 128), dtype=torch.uint8, device=DEV)
    elif c["op"] == "quantize":
        b["q"] = torch.empty(c["rows"], c["K"], dtype=FP8, device=DEV)
        b["scale"] = torch.empty(c["rows"], _blocks(c["K"]), dtype=torch.float32, device=DEV)
    elif c["op"] == "gemm":
        b["y"] = torch.empty(c["M"], c["N"], dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
        b["ws"] = torch.empty(binding.moe_gemm_fp8_workspace_bytes(c["M"], c["N"], c["K"]), dtype=torch.uint8,
                              device=DEV)
    else:
        T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
        b["y"] = torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV)
        b["ws"] = torch.empty(binding.moe_fp8_workspace_bytes(T, E, k, H, I), dtype=torch.uint8, device=DEV)
    return b


def run(state):
    s, c = state, state["case"]
    if own:
        from mxfp4_routed_expert_route_amd import binding
        b = s.get("buffers")
        if b is None:
            b = s["buffers"] = _buffers(s)
        if c["op"] == "route":
            how = dict(score=c["score"], bias=s["bias"], groups=c["groups"], topk_groups=c["topk_groups"],
                       group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
            if c["grouped"]:
                binding.moe_route_scored_and_group(s["logits"], c["k"], b["ids"], b["weights"], b["bitmatrix"],
                                                   b["counts"], b["offsets"], b["gather"], b["scatter"], b["ws"],
                                                   **how)
                return [b[n] for n in ("ids", "weights", "bitmatrix", "counts", "offsets", "gather", "scatter")]
            binding.moe_route_scored(s["logits"], c["k"], b["ids"], b["weights"], **how)
            return [b["ids"], b["weights"]]
        if c["op"] == "quantize":
            binding.moe_quantize_fp8(s["x"], b["q"], b["scale"])
            return [b["q"], b["scale"]]
        if c["op"] == "gemm":
            binding.moe_gemm_fp8(s["xq"], s["xs"], s["w"], s["ws"], b["y"], b["ws"])
            return [b["y"]]
        binding.moe_grouped_ffn_fp8(s["x"], c["k"], s["w1"], s["w1s"], s["w2"], s["w2s"], s["counts"],
                                    s["offsets"], s["gather"], LIMIT, b["y"], b["ws"])
        return [b["y"]]
    if c["op"] == "route":
        return _route_plain(s)
    if c["op"] == "quantize":
        return list(_quantize_plain(s["x"]))
    if c["op"] == "gemm":
        return [_gemm_plain(s)]
    return [_ffn_plain(s)]


# ---------------------------------------------------------------- work

def _touched(c):
    """Expected number of experts with rows: expert e is chosen by a token with probability about k p_e."""
    w = [1.0 / (r * r) if c["skew"] else 1.0 for r in range(1, c["E"] + 1)]
    total = sum(w)
    return sum(1.0 - (1.0 - min(1.0, c["k"] * v / total)) ** c["T"] for v in w)


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        out = 8 * T * k
        if c["grouped"]:
            out += 8 * T * k + 4 * T * ((E + 31) // 32) + 8 * E + 4
        return dict(bytes=T * E * (2 if c["bf16"] else 4) + (4 * E if c["bias"] else 0) + out, flops=4 * T * E)
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        return dict(bytes=3 * n + 4 * c["rows"] * _blocks(c["K"]), flops=4 * n)
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        nbytes = M * K + N * K + 4 * (M + _blocks(N)) * _blocks(K) + M * N * (4 if c["f32"] else 2)
        return dict(bytes=nbytes, flops=2 * M * N * K)
    T, k, H, I = c["T"], c["k"], c["H"], c["I"]
    rows = T * k
    weights = 3 * H * I + 4 * 3 * (H // BLOCK) * (I // BLOCK)
    return dict(bytes=int(_touched(c) * weights) + 2 * T * H + 2 * rows * H + 4 * rows, flops=6 * rows * H * I)


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3(v):
    """Nearest E4M3 value, ties to even: 4 significant bits, steps of 2^-9 below 2^-6, 448 at most."""
    a = v.abs().clamp(max=448.0)
    _, ex = torch.frexp(a)
    step = ((ex.to(torch.int64) - 4).clamp(min=-9) + 1023 << 52).view(torch.float64)   # a power of two
    return torch.copysign(torch.round(a / step) * step, v)


def _quantize_exact(x):
    """Codes as values and scales, of x in float64."""
    rows, K = x.shape
    q, sc = torch.empty_like(x), x.new_empty(rows, _blocks(K))
    for b in range(_blocks(K)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        a = part.abs().max(1, keepdim=True).values.clamp(min=FLOOR)
        q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(part * 448.0 / a)
        sc[:, b:b + 1] = a / 448.0
    return q, sc


def _product_exact(q, sc, w, ws):
    """sum over K blocks of (scales) x (products of the codes), in float64."""
    y = q.new_zeros(q.shape[0], w.shape[0])
    codes = w.view(FP8).double()
    row_block = torch.arange(w.shape[0], device=DEV) // BLOCK
    for b in range(_blocks(q.shape[1])):
        cut = slice(b * BLOCK, (b + 1) * BLOCK)
        y += (q[:, cut] * sc[:, b:b + 1]) @ (codes[:, cut] * ws.double()[row_block, b:b + 1]).t()
    return y


def _route_exact(c, s):
    l = s["logits"].double().cpu().numpy()
    T, E, k = c["T"], c["E"], c["k"]
    if c["score"] == "softmax":
        z = np.exp(l - l.max(1)[:, None])
        score = z / z.sum(1)[:, None]
    else:
        score = np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
    key = score + (0.0 if s["bias"] is None else s["bias"].double().cpu().numpy()[None, :])
    per = E // c["groups"]
    group_of = np.arange(E) // per
    if c["groups"] > 1:
        top = -np.sort(-key.reshape(T, c["groups"], per), axis=2)[:, :, :c["group_top"]].sum(2)
        rank = np.argsort(np.argsort(-top, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(rank[:, group_of] < c["topk_groups"], key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(score, ids, 1)
    if c["renorm"]:
        w = w / w.sum(1)[:, None]
    out = [ids.astype(np.int32), torch.from_numpy(w * c["scale"])]
    if c["grouped"]:
        bits = np.zeros((T, (E + 31) // 32), np.uint32)
        for j in range(k):
            np.bitwise_or.at(bits, (np.arange(T), ids[:, j] // 32), np.uint32(1) << (ids[:, j] % 32).astype(np.uint32))
        flat = ids.reshape(-1)
        counts = np.bincount(flat, minlength=E)
        gather = np.argsort(flat, kind="stable")
        scatter = np.empty_like(gather)
        scatter[gather] = np.arange(flat.size)
        out += [bits.view(np.int32), counts.astype(np.int32), np.r_[0, np.cumsum(counts)].astype(np.int32),
                gather.astype(np.int32), scatter.astype(np.int32)]
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return _route_exact(c, s)
    if c["op"] == "quantize":
        return list(_quantize_exact(s["x"].double()))
    if c["op"] == "gemm":
        return [_product_exact(s["xq"].view(FP8).double(), s["xs"].double(), s["w"], s["ws"])]
    H, I, k = c["H"], c["I"], c["k"]
    q, sc = _quantize_exact(s["x"].double())
    y = torch.zeros(s["gather"].numel(), H, dtype=torch.float64, device=DEV)
    token = s["gather"].long() // k
    ends = np.cumsum(s["host_counts"]).tolist()
    for e in range(c["E"]):
        rows = slice(ends[e] - s["host_counts"][e], ends[e])
        if rows.start == rows.stop:
            continue
        gu = _product_exact(q[token[rows]], sc[token[rows]], s["w1"][e], s["w1s"][e])
        gate = torch.minimum(gu[:, :I], gu.new_tensor(LIMIT))
        up = gu[:, I:].clamp(-LIMIT, LIMIT)
        hq, hs = _quantize_exact(gate * torch.sigmoid(gate) * up)
        y[rows] = _product_exact(hq, hs, s["w2"][e], s["w2s"][e])
    return [y]

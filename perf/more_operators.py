"""Measured cases of the operators around the routed experts: the norm in front of them, the
adapters beside a shared projection, and the loss that keeps the router's load balanced.

  norm          s = bf16(x + residual) (or x); y = s rstd w, rstd = 1 / sqrt(mean(s^2) + eps);
                y in bf16, or in E4M3 with one scale per run of 128 (a = max(max |y|, 2^-100)
                over the run, scale = a / 448, q = E4M3(448 y / a)), or both, with s beside them.
  norm_grad     of y with respect to s and w: with z = dy w,
                ds = rstd z - s rstd^3 mean(z s), plus the gradient that reaches s beside the
                norm; dw = sum over rows of dy s rstd.
  balance       p = softmax(l), or sigmoid(l) divided by its sum; per packed sequence of n tokens
                loss = E / (k n^2) sum_e count_e sum_t p_te, count_e the slots that chose e, and
                the gradient of sum_s g_s loss_s with respect to the logits, the choices being
                constants: dl = g E / (k n^2) p (c - sum_i p_i c_i), for sigmoid scores times
                1 - sigmoid(l).  Tokens behind the last sequence are padding.
  balance_grad  that gradient alone, from counts kept since the forward pass; added to a gradient
                that comes from elsewhere, if there is one.
  lora          y = base + scaling_a (x A_a^T) B_a^T with the adapter a of each row, base alone for
                rows without one; where `group` is set, the rows are grouped by adapter first.

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
EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _norm(name, rows, H, residual, y, q, wf32):
    return dict(name=name, op="norm", rows=rows, H=H, residual=residual, y=y, q=q, wf32=wf32)


def _norm_grad(name, rows, H, beside, wf32):
    return dict(name=name, op="norm_grad", rows=rows, H=H, beside=beside, wf32=wf32)


def _balance(name, op, T, E, k, score, seqs, bf16, add):
    return dict(name=name, op=op, T=T, E=E, k=k, score=score, seqs=seqs, bf16=bf16, add=add)


def _lora(name, M, N, K, R, L, packed, group, f32):
    return dict(name=name, op="lora", M=M, N=N, K=K, R=R, L=L, packed=packed, group=group, f32=f32)


def listed():
    return [
        # one token of one stream in front of its experts: bf16 for the experts, FP8 for the dense products
        _norm("norm-token", 1, 4096, True, True, True, False),
        # a long prompt batch, both outputs
        _norm("norm-prompt", 8191, 4096, True, True, True, False),
        # training: a few dozen rows of an odd width, frozen stream beside it; a long batch
        _norm_grad("norm-grad-odd", 77, 2064, False, True),
        _norm_grad("norm-grad-batch", 8191, 4096, True, False),
        # the router's loss in a training step: a short batch of ragged sequences with sigmoid scores
        # in bf16; a full batch of 16 packed sequences
        _balance("balance-odd", "balance", 1021, 96, 6, "sigmoid", 5, True, False),
        _balance("balance-batch", "balance", 65536, 256, 6, "softmax", 16, False, False),
        # its gradient in a backward pass of its own, and added to the gradient that the routing weights bring
        _balance("balance-grad-odd", "balance_grad", 1021, 96, 6, "sigmoid", 5, True, False),
        _balance("balance-grad-batch", "balance_grad", 65536, 256, 6, "softmax", 16, False, True),
        # one token of one stream (decode), eight adapters loaded
        _lora("lora-token", 1, 4096, 4096, 16, 8, False, False, False),
        # a router's fp32 logits: odd sizes
        _lora("lora-odd", 77, 1003, 2064, 8, 5, False, False, True),
        # 64 streams of 8 tokens, each stream with an adapter of its own, grouped in the step
        _lora("lora-burst", 512, 4096, 4096, 16, 64, True, True, False),
        # a long prompt batch of packed requests, eight adapters
        _lora("lora-prompt", 8191, 4096, 4096, 64, 8, True, False, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "balance", "balance_grad", "lora", "lora"])
    if op == "norm":
        y, q = rng.choice([(True, False), (False, True), (True, True)])
        case = _norm("", _log(rng, 1, 8191), 16 * _log(rng, 1, 256) if q else 8 * _log(rng, 1, 512),
                     rng.random() < 0.7, y, q, rng.random() < 0.5)
    elif op == "norm_grad":
        case = _norm_grad("", _log(rng, 1, 8191), 8 * _log(rng, 1, 512), rng.random() < 0.5, rng.random() < 0.5)
    elif op in ("balance", "balance_grad"):
        E = _log(rng, 8, 256)
        case = _balance("", op, _log(rng, 1, 65536), E, rng.randint(1, min(8, E // 2)),
                        rng.choice(["softmax", "sigmoid"]), rng.randint(1, 16), rng.random() < 0.4, rng.random() < 0.4)
    else:
        R = 8 * rng.choice([1, 1, 2, 2, 3, 4, 8, 16])
        case = _lora("", _log(rng, 1, 8191), _log(rng, 1, 4096), 8 * _log(rng, 2, 512), R,
                     _log(rng, 1, min(64, 512 // R)), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _hidden(g, rows, H):
    """Hidden states: a few channels are much larger than the others."""
    return (_randn(g, rows, H) * torch.exp(_randn(g, H) * 0.7)).bfloat16()


def _cuts(g, n, total):
    """Offsets [n + 1] of packed sequences of different lengths in the first 15/16 of `total` rows."""
    end = total - total // 16
    inner = torch.sort(torch.randint(0, end + 1, (n - 1,), device=DEV, generator=g)).values
    return torch.cat([inner.new_zeros(1), inner, inner.new_full((1,), end)]).to(torch.int32)


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case=case)
    if c["op"] in ("norm", "norm_grad"):
        rows, H = c["rows"], c["H"]
        w = 1.0 + 0.2 * _randn(g, H)
        s["w"] = w if c["wf32"] else w.bfloat16()
        s["x"] = _hidden(g, rows, H)
        if c["op"] == "norm":
            s["residual"] = _hidden(g, rows, H) if c["residual"] else None
        else:
            s["dy"] = (_randn(g, rows, H) * 0.01).bfloat16()
            s["beside"] = (_randn(g, rows, H) * 0.01).bfloat16() if c["beside"] else None
    elif c["op"] in ("balance", "balance_grad"):
        T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
        # some experts are favoured, as a loss of this kind meets them
        logits = _randn(g, T, E) + 0.5 * _randn(g, E)
        s["logits"] = logits.bfloat16() if c["bf16"] else logits
        s["ids"] = torch.topk(s["logits"].float(), k, dim=1).indices.to(torch.int32)
        s["cuts"] = _cuts(g, S, T)
        s["dloss"] = 0.01 * (0.5 + torch.rand(S, device=DEV, generator=g))
        s["add"] = (_randn(g, T, E) * 1e-4).to(s["logits"].dtype) if c["add"] else None
        if c["op"] == "balance_grad":
            s["counts"] = _counts(s["ids"], _sequence(s["cuts"], T), S, E)
    else:
        M, N, K, R, L = (c[n] for n in ("M", "N", "K", "R", "L"))
        if c["packed"]:   # requests of different lengths, one adapter each; some have none
            n = min(2 * L, M)
            of = torch.randint(0, L, (n + 1,), device=DEV, generator=g)
            of[torch.rand(n + 1, device=DEV, generator=g) < 0.1] = -1
            ids = of[_sequence(_cuts(g, n, M), M).long()]
        else:             # each row is a stream of its own
            ids = torch.randint(0, L, (M,), device=DEV, generator=g)
            ids[1:][torch.rand(M - 1, device=DEV, generator=g) < 0.1] = -1
        s["ids"] = ids.to(torch.int32)
        s["offsets"], s["rows"] = _group(s["ids"], L)
        s["x"] = _randn(g, M, K).bfloat16()
        s["a"] = (_randn(g, L, R, K) / math.sqrt(K)).bfloat16()
        s["b"] = (_randn(g, L, N, R) / math.sqrt(R)).bfloat16()
        s["scaling"] = 0.25 + torch.rand(L, device=DEV, generator=g)
        base = _randn(g, M, N)
        s["base"] = base if c["f32"] else base.bfloat16()
    return s


# ---------------------------------------------------------------- plain forms

def _sequence(cuts, T):
    """The sequence of each of T tokens; behind the last one, their number."""
    return (torch.arange(T, device=cuts.device)[:, None] >= cuts[None, 1:]).sum(1)


def _counts(ids, seq, S, E):
    flat = (seq[:, None] * E + ids.long()).reshape(-1)
    n = torch.zeros((S + 1) * E, dtype=torch.int32, device=ids.device)
    return n.scatter_add_(0, flat, torch.ones_like(flat, dtype=torch.int32)).view(S + 1, E)[:S].contiguous()


def _group(ids, L):
    """Offsets [L + 1] of the adapters' rows, and all rows in the adapters' order, those without one last."""
    key = torch.where((ids >= 0) & (ids < L), ids, L).long()
    rows = torch.sort(key, stable=True).indices.to(torch.int32)
    counts = torch.zeros(L + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    return torch.cat([counts.new_zeros(1), counts[:L].cumsum(0)]).to(torch.int32), rows


def _quantize_plain(v):
    rows, K = v.shape
    nb = -(-K // BLOCK)
    v = torch.nn.functional.pad(v, (0, nb * BLOCK - K)).view(rows, nb, BLOCK)
    a = v.abs().amax(2, keepdim=True).clamp_min(FLOOR)
    # quotients in 64 bits: many lie near the border between two codes
    q = (v.double() * 448.0 / a.double()).float().to(FP8).view(rows, nb * BLOCK)[:, :K].contiguous()
    return q, (a.double() / 448.0).float().squeeze(2)


def _rstd(s):
    return 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)


def _norm_plain(st):
    c, out = st["case"], []
    s = st["x"]
    if c["residual"]:
        s = (s.float() + st["residual"].float()).bfloat16()
        out.append(s)
    s = s.float()
    y = s * _rstd(s) * st["w"].float()
    if c["y"]:
        out.append(y.bfloat16())
    if c["q"]:
        out += _quantize_plain(y)
    return out


def _norm_grad_plain(st):
    s, dy = st["x"].float(), st["dy"].float()
    r = _rstd(s)
    z = dy * st["w"].float()
    ds = r * z - s * (r * r * r * (z * s).mean(1, keepdim=True))
    if st["beside"] is not None:
        ds = ds + st["beside"].float()
    return [ds.bfloat16(), (dy * s * r).sum(0)]


def _probabilities(l, score):
    """p, and what dp/dl has on top of the softmax's Jacobian."""
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), None
    e = 1.0 / (1.0 + torch.exp(-l))
    return e / e.sum(1, keepdim=True), 1.0 / (1.0 + torch.exp(l))


def _gradient_plain(st, seq, p, slope, counts, n):
    c = st["case"]
    factor = torch.cat([st["dloss"].double() * c["E"] / (c["k"] * n * n), n.new_zeros(1)]).float()[seq][:, None]
    count = torch.cat([counts, counts.new_zeros(1, c["E"])]).float()[seq]
    d = factor * p * (count - (p * count).sum(1, keepdim=True))
    if slope is not None:
        d = d * slope
    if st["add"] is not None:
        d = d + st["add"].float()
    return d.to(st["logits"].dtype)


def _balance_plain(st):
    c = st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    seq = _sequence(st["cuts"], T)
    p, slope = _probabilities(st["logits"].float(), c["score"])
    n = (st["cuts"][1:] - st["cuts"][:-1]).double().clamp_min(1.0)
    if c["op"] == "balance_grad":
        return [_gradient_plain(st, seq, p, slope, st["counts"], n)]
    counts = _counts(st["ids"], seq, S, E)
    # sums over a sequence's tokens in 64 bits: they are long
    upto = torch.cumsum(torch.cat([p.new_zeros(1, E), p]).t().contiguous(), 1, dtype=torch.float64)
    upto = upto[:, st["cuts"].long()]
    total = (upto[:, 1:] - upto[:, :-1]).t()
    loss = ((counts * total).sum(1) * E / (k * n * n)).float()
    return [loss, counts, _gradient_plain(st, seq, p, slope, counts, n)]


def _lora_plain(st):
    c = st["case"]
    M, N, K, R, L = (c[n] for n in ("M", "N", "K", "R", "L"))
    ids = st["ids"].long()
    # every adapter's products, the others' set to zero
    v = (st["x"].float() @ st["a"].view(L * R, K).float().t()).view(M, L, R)
    mine = torch.arange(L, device=DEV)[None, :] == ids[:, None]
    v = torch.where(mine, st["scaling"][None, :], 0.0)[:, :, None] * v
    y = st["base"].float() + v.view(M, L * R) @ st["b"].float().transpose(1, 2).reshape(L * R, N)
    out = list(_group(st["ids"], L)) if c["group"] else []
    return out + [y if c["f32"] else y.bfloat16()]


_PLAIN = dict(norm=_norm_plain, norm_grad=_norm_grad_plain, balance=_balance_plain, balance_grad=_balance_plain,
              lora=_lora_plain)


# ---------------------------------------------------------------- one pass

def _buffers(st):
    """The outputs and workspace that a program keeps from call to call."""
    from mxfp4_routed_expert_route_amd import binding
    c = st["case"]
    b = {}

    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    def space(n):
        return new(n, dtype=torch.uint8)

    if c["op"] == "norm":
        rows, H = c["rows"], c["H"]
        b["sum"] = new(rows, H, dtype=torch.bfloat16) if c["residual"] else None
        b["y"] = new(rows, H, dtype=torch.bfloat16) if c["y"] else None
        b["q"] = new(rows, H, dtype=FP8) if c["q"] else None
        b["scale"] = new(rows, -(-H // BLOCK)) if c["q"] else None
    elif c["op"] == "norm_grad":
        b["dx"], b["dw"] = torch.empty_like(st["x"]), new(c["H"])
        b["ws"] = space(binding.moe_rms_norm_grad_workspace_bytes(c["rows"], c["H"]))
    elif c["op"] == "balance":
        b["loss"], b["counts"] = new(c["seqs"]), new(c["seqs"], c["E"], dtype=torch.int32)
        b["dlogits"] = torch.empty_like(st["logits"])
        b["ws"] = space(binding.moe_balance_loss_workspace_bytes(c["T"], c["E"], c["seqs"]))
    elif c["op"] == "balance_grad":
        b["dlogits"] = torch.empty_like(st["logits"])
    else:
        b["y"] = torch.empty_like(st["base"])
        b["offsets"], b["rows"] = torch.empty_like(st["offsets"]), torch.empty_like(st["rows"])
        b["ws"] = space(binding.moe_lora_add_workspace_bytes(c["M"], c["N"], c["K"], c["R"], c["L"]))
    return b


def run(state):
    st, c = state, state["case"]
    if own:
        from mxfp4_routed_expert_route_amd import binding
        b = st.get("buffers")
        if b is None:
            b = st["buffers"] = _buffers(st)
        if c["op"] == "norm":
            binding.moe_rms_norm(st["x"], st["w"], EPS, residual=st["residual"], sum=b["sum"], y=b["y"], q=b["q"],
                                 scale=b["scale"])
            return [b[n] for n in ("sum", "y", "q", "scale") if b[n] is not None]
        if c["op"] == "norm_grad":
            binding.moe_rms_norm_grad(st["x"], st["w"], EPS, st["dy"], b["dx"], b["dw"], b["ws"], dsum=st["beside"])
            return [b["dx"], b["dw"]]
        if c["op"] == "balance":
            binding.moe_balance_loss(st["logits"], st["ids"], b["loss"], b["counts"], b["ws"], score=c["score"],
                                     seq_offsets=st["cuts"], dloss=st["dloss"], dlogits=b["dlogits"],
                                     add_to=st["add"])
            return [b["loss"], b["counts"], b["dlogits"]]
        if c["op"] == "balance_grad":
            binding.moe_balance_loss_grad(st["logits"], c["k"], st["counts"], st["dloss"], b["dlogits"],
                                          score=c["score"], seq_offsets=st["cuts"], add_to=st["add"])
            return [b["dlogits"]]
        offsets, rows, out = st["offsets"], st["rows"], []
        if c["group"]:
            offsets, rows = b["offsets"], b["rows"]
            binding.moe_lora_group(st["ids"], c["L"], offsets, rows)
            out = [offsets, rows]
        binding.moe_lora_add(st["x"], st["a"], st["b"], st["scaling"], offsets, rows, st["base"], b["y"], b["ws"])
        return out + [b["y"]]
    return _PLAIN[c["op"]](st)


# ---------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["H"]
        each = 2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0) + (1 if c["q"] else 0)
        scales = 4 * c["rows"] * -(-c["H"] // BLOCK) if c["q"] else 0
        return dict(bytes=n * each + scales + c["H"] * (4 if c["wf32"] else 2), flops=n * 5)
    if c["op"] == "norm_grad":
        n = c["rows"] * c["H"]
        return dict(bytes=n * (8 if c["beside"] else 6) + c["H"] * (8 if c["wf32"] else 6), flops=n * 11)
    if c["op"] in ("balance", "balance_grad"):
        T, E, S = c["T"], c["E"], c["seqs"]
        n, size = T * E, 2 if c["bf16"] else 4
        ids = 4 * T * c["k"] if c["op"] == "balance" else 0
        return dict(bytes=n * size * (3 if c["add"] else 2) + ids + 4 * S * (E + 3) + 4, flops=n * 10)
    M, N, K, R, L = (c[n] for n in ("M", "N", "K", "R", "L"))
    used = L * (1.0 - (1.0 - 0.9 / L) ** (min(2 * L, M) if c["packed"] else M))   # adapters that have rows
    touched = int(used * R * (N + K)) * 2
    rows = M * (2 * K + 2 * N * (4 if c["f32"] else 2) + 4)
    return dict(bytes=touched + rows + 8 * L + (4 * M + 4 * L if c["group"] else 0), flops=2 * M * R * (N + K))


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3(v):
    """Nearest E4M3 value, ties to even: 4 significant bits, steps of 2^-9 below 2^-6, 448 at most."""
    a = v.abs().clamp(max=448.0)
    _, ex = torch.frexp(a)
    step = ((ex.to(torch.int64) - 4).clamp(min=-9) + 1023 << 52).view(torch.float64)   # a power of two
    return torch.copysign(torch.round(a / step) * step, v)


def _norm_exact(c, s):
    out = []
    x = s["x"].double()
    if c["residual"]:
        # the sum of two bf16 values to the nearest bf16: 8 significant bits, ties to even
        x = x + s["residual"].double()
        _, ex = torch.frexp(x)
        step = ((ex.to(torch.int64) - 8).clamp(min=-133) + 1023 << 52).view(torch.float64)
        x = torch.round(x / step) * step
        out.append(x)
    y = x * torch.rsqrt(x.square().sum(1, keepdim=True) / c["H"] + EPS) * s["w"].double()
    if c["y"]:
        out.append(y)
    if c["q"]:
        q, sc = torch.empty_like(y), y.new_empty(y.shape[0], -(-c["H"] // BLOCK))
        for b in range(sc.shape[1]):
            part = y[:, b * BLOCK:(b + 1) * BLOCK]
            a = part.abs().max(1, keepdim=True).values.clamp(min=FLOOR)
            q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3(part * 448.0 / a)
            sc[:, b:b + 1] = a / 448.0
        out += [q, sc]
    return out


def _norm_grad_exact(c, s):
    x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
    rms = torch.sqrt(x.square().sum(1, keepdim=True) / c["H"] + EPS)
    unit = x / rms                                      # y = unit w
    g = dy * w
    dx = (g - unit * (g * unit).sum(1, keepdim=True) / c["H"]) / rms
    if s["beside"] is not None:
        dx += s["beside"].double()
    return [dx, (dy * unit).sum(0)]


def _log_scores(l, score):
    """log p of p = scores divided by their sum."""
    a = l.double()
    if score == "sigmoid":
        a = -torch.logaddexp(a.new_zeros(()), -a)
    return a - torch.logsumexp(a, 1, keepdim=True)


def _balance_exact(c, s):
    E, k = c["E"], c["k"]
    ends = s["cuts"].tolist()
    loss, counts = [], np.zeros((c["seqs"], E), np.int32)
    ids = s["ids"].cpu().numpy()
    for i, (t0, t1) in enumerate(zip(ends, ends[1:])):
        if t0 == t1:
            loss.append(0.0)
            continue
        counts[i] = np.bincount(ids[t0:t1].reshape(-1), minlength=E)
        mean = torch.exp(_log_scores(s["logits"][t0:t1], c["score"])).mean(0)
        share = torch.from_numpy(counts[i] / (k * (t1 - t0))).to(DEV)
        loss.append(E * float((share * mean).sum()))
    grad = _balance_grad_exact(c, dict(s, counts=torch.from_numpy(counts).to(DEV)))
    return [torch.tensor(loss, dtype=torch.float64), counts, *grad]


def _balance_grad_exact(c, s):
    E, k = c["E"], c["k"]
    ends = s["cuts"].tolist()
    d = torch.zeros(c["T"], E, dtype=torch.float64, device=DEV)
    for i, (t0, t1) in enumerate(zip(ends, ends[1:])):
        if t0 == t1:
            continue
        l = s["logits"][t0:t1]
        p = torch.exp(_log_scores(l, c["score"]))
        share = s["counts"][i].double() / (k * (t1 - t0))
        dp = float(s["dloss"][i].double()) * E * share / (t1 - t0)      # the loss by p of one token
        da = p * (dp - p @ dp[:, None])                                 # by the logarithms of the scores
        d[t0:t1] = da * torch.sigmoid(-l.double()) if c["score"] == "sigmoid" else da
    return [d if s["add"] is None else d + s["add"].double()]


def _lora_exact(c, s):
    L, ids = c["L"], s["ids"].tolist()
    y = s["base"].double()
    of = [[] for _ in range(L + 1)]
    for t, a in enumerate(ids):
        of[a if 0 <= a < L else L].append(t)
    for a in range(L):
        if of[a]:
            at = torch.tensor(of[a], device=DEV)
            inner = s["x"][at].double() @ s["a"][a].double().t()
            y[at] += float(s["scaling"][a].double()) * (inner @ s["b"][a].double().t())
    if not c["group"]:
        return [y]
    offsets = np.r_[0, np.cumsum([len(r) for r in of[:L]])].astype(np.int32)
    return [offsets, np.array(sum(of, []), np.int32), y]


_EXACT = dict(norm=_norm_exact, norm_grad=_norm_grad_exact, balance=_balance_exact,
              balance_grad=_balance_grad_exact, lora=_lora_exact)


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))

"""Cases of the MoE router and the FP8 block-scaled operators, each in a plain form and as the library's calls.

Operators (the "op" of a case):
  route     softmax router: top-k, weights, per-expert counts, expert-sorted rows, balance loss
  balance   one training step of the router: the routing above and the gradient of its logits
            from the balance loss and the weights of the selected experts
  quantize  bf16 -> E4M3 codes with a scale for each block of 128
  gemm      y = a b^T on E4M3 codes with a scale for each block of 128
  grouped   the same product for each expert's rows (MoE)

With `own` false, run() computes them with elementary torch operations in 32 bits; with `own`
true, through moe_nvfp4_gemm_gb300.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0


def listed():
    return [
        # one token of a decode loop through a 256-expert, top-8 router: launch latency
        {"name": "route_one_token", "op": "route", "T": 1, "E": 256, "k": 8, "bf16": False, "renorm": True, "masked": False},
        # a packed prefill batch with padding tokens and switched-off experts, bf16 logits
        {"name": "route_prefill_masked", "op": "route", "T": 40961, "E": 256, "k": 8, "bf16": True, "renorm": True,
         "masked": True},
        # a small training batch, few experts, top-2
        {"name": "balance_small", "op": "balance", "T": 1001, "E": 8, "k": 2, "bf16": False, "renorm": False, "masked": True},
        # the router of a large training batch
        {"name": "balance_large", "op": "balance", "T": 65536, "E": 256, "k": 8, "bf16": False, "renorm": True,
         "masked": False},
        # 512 decode tokens sent to 8 experts each, gathered into expert order while quantised
        {"name": "quantize_gather", "op": "quantize", "M": 512, "K": 6144, "rows": 4096, "block_rows": 1, "transposed": False},
        # activations of a training batch for the forward product and for the weight gradient
        {"name": "quantize_train", "op": "quantize", "M": 4099, "K": 8192, "rows": 0, "block_rows": 1, "transposed": True},
        # one decode token through a square linear layer: bound by the weight's bytes
        {"name": "gemm_one_token", "op": "gemm", "M": 1, "N": 8192, "K": 8192, "b_rows": 128, "f32": False},
        # a small batch against a weight of odd sizes
        {"name": "gemm_odd", "op": "gemm", "M": 77, "N": 5003, "K": 2064, "b_rows": 128, "f32": False},
        # prefill through the gate/up projection of a feed-forward layer: bound by the tensor cores
        {"name": "gemm_prefill", "op": "gemm", "M": 4096, "N": 28672, "K": 8192, "b_rows": 128, "f32": False},
        # weight gradient: both operands scaled along the tokens, fp32 sums out
        {"name": "gemm_weight_grad", "op": "gemm", "M": 4096, "N": 6144, "K": 4112, "b_rows": 1, "f32": True},
        # decode: 512 tokens, 8 of 256 experts each, gate/up projection
        {"name": "grouped_decode", "op": "grouped", "E": 256, "T": 512, "k": 8, "N": 4096, "K": 6144},
        # prefill: 4096 tokens, 8 of 256 experts each, down projection
        {"name": "grouped_prefill", "op": "grouped", "E": 256, "T": 4096, "k": 8, "N": 6144, "K": 2048},
    ]


def _count(rng, lo, hi):
    """A number of lo..hi, spread over its logarithm: odd, or a power of two."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.3:
        v = 1 << max(0, v.bit_length() - 1)
    else:
        v |= 1
    return max(lo, min(hi, v))


def _depth(rng, lo, hi):
    """A contraction length: one of the usual ones, or an odd multiple of 16."""
    if rng.random() < 0.5:
        return rng.choice([v for v in (512, 1024, 2048, 4096, 6144, 8192) if lo <= v <= hi])
    return 16 * (_count(rng, max(1, lo // 16), hi // 16 - 1) | 1)


def _width(rng, lo, hi):
    """A number of output columns: one of the usual ones, a multiple of 8, or odd."""
    r = rng.random()
    if r < 0.4:
        return rng.choice([v for v in (512, 2048, 4096, 6144, 8192, 28672) if lo <= v <= hi])
    v = _count(rng, lo, hi - 1) | 1
    return v * 8 if r < 0.7 and v * 8 <= hi else v


def draw(rng):
    op = rng.choice(["route", "balance", "quantize", "gemm", "gemm", "grouped"])
    if op in ("route", "balance"):
        E = rng.choice([4, 8, 16, 60, 64, 96, 128, 160, 256])
        return {"op": op, "T": _count(rng, 1, 65536 if E <= 128 else 32768), "E": E, "k": rng.randint(1, min(8, E)),
                "bf16": rng.random() < 0.5, "renorm": rng.random() < 0.5, "masked": rng.random() < 0.5}
    if op == "quantize":
        M = _count(rng, 1, 8192)
        K = _depth(rng, 256, 8192 if M <= 4096 else 4096)
        form = rng.choice(["rows", "gather", "square", "both", "both_square"])
        return {"op": op, "M": M, "K": K, "rows": _count(rng, 1, 4096) if form == "gather" else 0,
                "block_rows": 128 if form.endswith("square") else 1, "transposed": form.startswith("both")}
    if op == "gemm":
        while True:
            c = {"op": op, "M": _count(rng, 1, 8192), "N": _width(rng, 128, 28672), "K": _depth(rng, 256, 8192),
                 "b_rows": rng.choice([128, 128, 1]), "f32": rng.random() < 0.3}
            if c["M"] * c["N"] * c["K"] <= 4096 * 28672 * 8192 // 2:
                return c
    while True:
        c = {"op": op, "E": rng.choice([4, 8, 32, 64, 256]), "T": _count(rng, 1, 4096), "k": rng.randint(1, 4),
             "N": _width(rng, 256, 6144), "K": _depth(rng, 512, 6144)}
        if c["E"] * c["N"] * c["K"] <= 256 * 4096 * 2048 and c["T"] * c["k"] * c["N"] * c["K"] <= 1 << 38:
            return c


# ---- inputs ------------------------------------------------------------------------------------


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """bf16 activations: N(0, 1), one value in a thousand twenty times as large."""
    x = _normal(g, M, K)
    x *= torch.where(torch.rand(M, K, generator=g, device="cuda") < 1e-3, 20.0, 1.0)
    return x.bfloat16()


def _routing_logits(g, case):
    """Router logits with some experts more popular than others, as they are early in training."""
    T, E = case["T"], case["E"]
    l = _normal(g, T, E) + 0.5 * _normal(g, 1, E)
    valid = None
    if case["masked"]:
        # padding tokens hold whatever the buffer held; a tenth of the experts is switched off for a token
        valid = torch.rand(T, generator=g, device="cuda") < 0.85
        l[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -math.inf
        l[torch.rand(T, generator=g, device="cuda") < 0.002] = -math.inf
        l[~valid] = math.nan
    return l.bfloat16() if case["bf16"] else l, valid


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("route", "balance"):
        s["logits"], s["valid"] = _routing_logits(g, case)
        if op == "balance":
            s["d_loss"] = torch.full((1,), 0.01, device="cuda")
            s["d_w"] = _normal(g, case["T"], case["k"]) * 1e-3
    elif op == "quantize":
        s["x"] = _activations(g, case["M"], case["K"])
        s["rows"] = None
        if case["rows"]:
            s["rows"] = torch.randint(0, case["M"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
    elif op == "gemm":
        s["a"], s["sa"] = _quantize(_activations(g, case["M"], case["K"]), 1)
        if case["b_rows"] == 128:
            s["b"], s["sb"] = _quantize((_normal(g, case["N"], case["K"]) * 0.02).bfloat16(), 128)
        else:
            s["b"], s["sb"] = _quantize(_activations(g, case["N"], case["K"]), 1)
    else:
        E, N, K, rows = case["E"], case["N"], case["K"], case["T"] * case["k"]
        # the router's result: some experts more popular than others, some without a row
        p = torch.softmax(0.3 * _normal(g, E), 0)
        expert = torch.multinomial(p, rows, replacement=True, generator=g)
        counts = torch.bincount(expert, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        s["most"] = int(counts.max())  # of the plain form's padded batch
        s["a"], s["sa"] = _quantize(_activations(g, rows, K), 1)
        s["b"] = torch.empty(E, N, K, dtype=FP8, device="cuda")
        s["sb"] = torch.empty(E, _blocks(N), _blocks(K), device="cuda")
        for e in range(E):
            s["b"][e], s["sb"][e] = _quantize((_normal(g, N, K) * 0.02).bfloat16(), 128)
    return s


# ---- plain forms ---------------------------------------------------------------------------------


def _blocks(n):
    return (n + 127) // 128


def _quantize(x, block_rows):
    """Codes [M, K] and scales: [K/128, M] for blocks of 1 x 128, [M/128, K/128] for 128 x 128."""
    M, K = x.shape
    mb = M if block_rows == 1 else _blocks(M) * 128
    xp = torch.zeros(mb, _blocks(K) * 128, device=x.device)
    xp[:M, :K] = x.float()
    v = xp.view(mb // block_rows, block_rows, _blocks(K), 128)
    amax = v.abs().amax((1, 3))
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, FP8_MAX))
    q = (v / scale[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(mb, -1)[:M, :K].contiguous().to(FP8)
    return q, (scale.t().contiguous() if block_rows == 1 else scale)


def _spread(scale, block_rows, rows, K):
    """A scale for each element, [rows, K]."""
    if block_rows == 1:
        return scale.t().repeat_interleave(128, 1)[:, :K]
    return scale.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :K]


def _plain_route(l, valid, k, renorm):
    T, E = l.shape
    x = l.float()
    routed = (x > -math.inf).any(1)
    if valid is not None:
        routed = routed & valid
    x = torch.where(routed[:, None], x, torch.full_like(x, -math.inf))
    top = torch.where(routed[:, None], x, torch.zeros_like(x)).amax(1, keepdim=True)
    e = torch.exp(x - top)
    p = e / torch.where(routed[:, None], e.sum(1, keepdim=True), torch.ones_like(top))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = torch.gather(x, 1, order) > -math.inf
    idx = torch.where(chosen, order, -1)
    w = torch.where(chosen, torch.gather(p, 1, order), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    flat = torch.where(chosen, order, E).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device).index_add_(0, flat, torch.ones_like(flat))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    by_expert = torch.sort(flat, stable=True).indices
    row = torch.empty_like(flat)
    row[by_expert] = torch.arange(T * k, device=l.device)
    slot_row = torch.where(chosen.reshape(-1), row, -1).view(T, k)
    row_token = torch.where(torch.arange(T * k, device=l.device) < offsets[-1], by_expert // k, -1)
    n = routed.sum()
    mean = p.sum(0) / n.clamp(min=1)
    loss = E * (counts.float() / (n * k).clamp(min=1) * mean).sum()
    out = {"topk_idx": idx.int(), "topk_w": w, "slot_row": slot_row.int(), "counts": counts.int(),
           "expert_offsets": offsets.int(), "row_token": row_token.int(), "mean_prob": mean,
           "balance_loss": loss.view(1), "routed_tokens": n.int().view(1)}
    return out, p


def _plain_route_backward(l, r, p, d_w, d_loss, renorm):
    T, E = l.shape
    k = d_w.shape[1]
    n = r["routed_tokens"].float().clamp(min=1)
    G = (d_loss * E * r["counts"].float() / (k * n * n)).expand(T, E)
    at = r["topk_idx"].long()
    dw = torch.where(at >= 0, d_w, torch.zeros_like(d_w))
    at = at.clamp(min=0)
    if renorm:
        own_part = r["topk_w"] * (dw - (r["topk_w"] * dw).sum(1, keepdim=True))
        d = p * (G - (p * G).sum(1, keepdim=True))
        d = d.scatter_add(1, at, own_part)
    else:
        G = G.scatter_add(1, at, dw)
        d = p * (G - (p * G).sum(1, keepdim=True))
    return d.to(l.dtype)


def _plain_gemm(s, c):
    a = s["a"].float() * _spread(s["sa"], 1, c["M"], c["K"])
    b = s["b"].float() * _spread(s["sb"], c["b_rows"], c["N"], c["K"])
    y = a @ b.t()
    return y if c["f32"] else y.bfloat16()


def _plain_grouped(s, c):
    rows, cap = s["a"].shape[0], s["most"]
    at = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), at.int(), right=True)
    place = expert * cap + at - s["offsets"][expert]
    x = torch.zeros(c["E"] * cap, c["K"], device="cuda")
    x[place] = s["a"].float() * _spread(s["sa"], 1, rows, c["K"])
    w = s["b"].float()
    w *= _spread(s["sb"], 128, c["N"], c["K"])
    y = torch.bmm(x.view(c["E"], cap, c["K"]), w.transpose(1, 2))
    return y.view(c["E"] * cap, c["N"])[place].bfloat16()


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _plain_route(s["logits"], s["valid"], c["k"], c["renorm"])[0]
    if c["op"] == "balance":
        r, p = _plain_route(s["logits"], s["valid"], c["k"], c["renorm"])
        return {"balance_loss": r["balance_loss"], "counts": r["counts"], "topk_w": r["topk_w"],
                "d_logits": _plain_route_backward(s["logits"], r, p, s["d_w"], s["d_loss"], c["renorm"])}
    if c["op"] == "quantize":
        x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
        q, sc = _quantize(x, c["block_rows"])
        if not c["transposed"]:
            return {"q": q, "s": sc}
        M = x.shape[0]
        xt = torch.zeros(c["K"], (M + 15) // 16 * 16, dtype=x.dtype, device=x.device)
        xt[:, :M] = x.t()
        qt, st = _quantize(xt, c["block_rows"])
        return {"q": q, "s": sc, "qt": qt, "st": st}
    return _plain_gemm(s, c) if c["op"] == "gemm" else _plain_grouped(s, c)


# ---- the library's calls ----------------------------------------------------------------------------


def _own(s):
    import moe_nvfp4_gemm_gb300 as m
    c = s["case"]
    if c["op"] == "route":
        return m.nvfp4_moe_route(s["logits"], c["k"], renormalize=c["renorm"], valid=s["valid"])._asdict()
    if c["op"] == "balance":
        r = m.nvfp4_moe_route(s["logits"], c["k"], renormalize=c["renorm"], valid=s["valid"])
        d = m.nvfp4_moe_route_backward(s["logits"], r, d_w=s["d_w"], d_loss=s["d_loss"], renormalize=c["renorm"],
                                       valid=s["valid"])
        return {"balance_loss": r.balance_loss, "counts": r.counts, "topk_w": r.topk_w, "d_logits": d}
    if c["op"] == "quantize":
        out = m.nvfp4_fp8_quantize(s["x"], block_rows=c["block_rows"], row_token=s["rows"], transposed=c["transposed"])
        return dict(zip(("q", "s", "qt", "st"), out))
    if c["op"] == "gemm":
        return m.nvfp4_fp8_gemm(s["a"], s["sa"], s["b"], s["sb"], c["M"], c["N"], c["K"], b_block_rows=c["b_rows"],
                                out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    return m.nvfp4_fp8_grouped_gemm(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], c["E"], s["a"].shape[0], c["N"],
                                    c["K"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- definitions in 64 bits ----------------------------------------------------------------------


def _exact_route(s, c):
    l, k = s["logits"].double(), c["k"]
    T, E = l.shape
    on = torch.isfinite(l).any(1) if s["valid"] is None else s["valid"] & (l.nan_to_num(0.0) > -1e300).any(1)
    l[~on] = -math.inf
    z = l - l.amax(1, keepdim=True).clamp(min=-1e300)
    p = z.exp()
    p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    # the selection: experts that fewer than k others precede (larger, or equal and of a lower index)
    idx = torch.full((T, k), -1, dtype=torch.int64, device=l.device)
    left, rows = l.clone(), torch.arange(T, device=l.device)
    lowest = torch.arange(E, 0, -1, device=l.device)
    for j in range(k):
        best = left.amax(1, keepdim=True)
        at = ((left == best) * lowest).argmax(1)
        some = best[:, 0] > -math.inf
        idx[:, j] = torch.where(some, at, -1)
        left[rows, at] = -math.inf
    sel = idx >= 0
    w = torch.where(sel, p.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    counts = torch.stack([(idx == e).sum() for e in range(E)]).double()
    n = max(1.0, float(on.sum()))
    mean = p.sum(0) / n
    loss = E * (counts / (n * k) * mean).sum()
    return p, idx, sel, w, counts, n, mean, loss.view(1)


def _exact_balance(s, c):
    p, idx, sel, w, counts, n, mean, loss = _exact_route(s, c)
    dw = torch.where(sel, s["d_w"].double(), 0.0)
    T, E = p.shape
    # d w_s / d l_j = w_s (1[j = idx_s] - q_j), q: w itself at the selected experts (renormalised) or p
    d = torch.zeros_like(p)
    q = torch.zeros_like(p)
    q.scatter_add_(1, idx.clamp(min=0), w)
    q = q if c["renorm"] else p
    for j in range(c["k"]):
        g = (dw[:, j] * w[:, j])[:, None]
        d -= g * q
        d.scatter_add_(1, idx[:, j:j + 1].clamp(min=0), g)
    f = c["E"] * counts / (n * n * c["k"]) * s["d_loss"].double()
    d += p * f - p * (p @ f)[:, None]
    return {"balance_loss": loss, "counts": None, "topk_w": w, "d_logits": d}


def _decode(codes, scale, block_rows):
    v = codes.double()
    rows, K = v.shape
    for c in range(_blocks(K)):
        part = v[:, c * 128:(c + 1) * 128]
        if block_rows == 1:
            part *= scale[c].double()[:, None]
        else:
            part *= scale[:, c].double()[torch.arange(rows, device=v.device) // 128][:, None]
    return v


def _exact_blocks(x, block_rows):
    """Scales and the quotients x / scale before their rounding to codes."""
    M, K = x.shape
    v = x.double()
    s = torch.ones(-(-M // block_rows), _blocks(K), dtype=torch.float64, device=x.device)
    for c in range(_blocks(K)):
        a = v[:, c * 128:(c + 1) * 128].abs().amax(1)
        if block_rows > 1:
            a = torch.stack([b.max() for b in a.split(block_rows)])
        s[:, c] = torch.where(a > 0, a / FP8_MAX, 1.0)
        v[:, c * 128:(c + 1) * 128] /= s[:, c].repeat_interleave(block_rows)[:M, None]
    return v, (s.t().contiguous() if block_rows == 1 else s)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        _, _, _, w, _, _, mean, loss = _exact_route(s, c)
        return {"topk_idx": None, "topk_w": w, "slot_row": None, "counts": None, "expert_offsets": None, "row_token": None,
                "mean_prob": mean, "balance_loss": loss, "routed_tokens": None}
    if c["op"] == "balance":
        return _exact_balance(s, c)
    if c["op"] == "quantize":
        x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
        q, sc = _exact_blocks(x, c["block_rows"])
        out = {"q": q, "s": sc}
        if c["transposed"]:
            qt, st = _exact_blocks(x.t().contiguous(), c["block_rows"])
            out["qt"] = torch.nn.functional.pad(qt, (0, -x.shape[0] % 16))
            out["st"] = st
        return out
    a = _decode(s["a"], s["sa"], 1)
    if c["op"] == "gemm":
        return a @ _decode(s["b"], s["sb"], c["b_rows"]).t()
    off = s["offsets"].tolist()
    return torch.cat([a[off[e]:off[e + 1]] @ _decode(s["b"][e], s["sb"][e], 128).t() for e in range(c["E"])])


def work(case):
    c = case
    if c["op"] in ("route", "balance"):
        T, E, k = c["T"], c["E"], c["k"]
        size = 2 if c["bf16"] else 4
        n_bytes = T * E * size + T * c["masked"] + 16 * T * k + 12 * E
        flops = 5 * T * E
        if c["op"] == "balance":  # read again: the balance gradient needs every token's counts first
            n_bytes += 2 * T * E * size + 12 * T * k
            flops += 10 * T * E
        return {"bytes": n_bytes, "flops": flops}
    if c["op"] == "quantize":
        rows, K = c["rows"] or c["M"], c["K"]
        scales = 4 * _blocks(K) * (rows if c["block_rows"] == 1 else _blocks(rows))
        n_bytes = 2 * c["M"] * K + rows * K + scales
        if c["transposed"]:
            n_bytes += rows * K + scales
        return {"bytes": n_bytes, "flops": 3 * rows * K}
    N, K = c["N"], c["K"]
    if c["op"] == "gemm":
        M = c["M"]
        n_bytes = (M + N) * K + 4 * _blocks(K) * (M + (N if c["b_rows"] == 1 else _blocks(N))) + M * N * (4 if c["f32"] else 2)
        return {"bytes": n_bytes, "flops": 2 * M * N * K}
    M = c["T"] * c["k"]
    busy = c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** M)  # experts that have a row
    return {"bytes": M * K + busy * N * (K + K / 32 / 128) + 4 * _blocks(K) * M + 2 * M * N, "flops": 2 * M * N * K}

"""Cases of the dense feed-forward operators, each in a plain form and as the library's calls.

Operators (the "op" of a case):
  gated     h = act(x Wg^T) * (x Wu^T): both projections of a gated feed-forward block
  train     the same with the gradients: h, dx, dWg, dWu from dh
  quantize  16-bit rows -> int8 codes with a scale for each row
  gemm      y = a b^T on int8 codes with a scale for each row of a (token) and of b (channel)
  clip      the norm over a list of gradients, and the gradients scaled down to a largest norm

With `own` false, run() computes them with elementary torch operations in 32 bits; with `own`
true, through moe_nvfp4_gemm_gb300.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of a decode loop through the gate/up projection of a large layer: bound by the weights' bytes
        {"name": "gated_one_token", "op": "gated", "M": 1, "I": 14336, "K": 8192, "type": "bf16", "act": "silu"},
        # a small batch against weights of odd sizes
        {"name": "gated_odd", "op": "gated", "M": 77, "I": 5000, "K": 2056, "type": "fp16", "act": "gelu_tanh"},
        # prefill through the same large layer: bound by the tensor cores
        {"name": "gated_prefill", "op": "gated", "M": 4096, "I": 14336, "K": 8192, "type": "bf16", "act": "silu"},
        # a step of a small model: latency and ragged tiles
        {"name": "train_small", "op": "train", "M": 333, "I": 2816, "K": 1024, "type": "fp16", "act": "gelu_tanh"},
        # a training batch of a middle-sized layer, its token count not a multiple of a tile
        {"name": "train_large", "op": "train", "M": 4099, "I": 8192, "K": 4096, "type": "bf16", "act": "silu"},
        # the activations of a decode batch, and of a prefill
        {"name": "quantize_decode", "op": "quantize", "M": 16, "K": 6144, "type": "fp16"},
        {"name": "quantize_prefill", "op": "quantize", "M": 4099, "K": 8192, "type": "bf16"},
        # one decode token through a square linear layer: bound by the weight's bytes
        {"name": "int8_one_token", "op": "gemm", "M": 1, "N": 8192, "K": 8192, "out": "bf16"},
        # a small batch against a weight of odd sizes
        {"name": "int8_odd", "op": "gemm", "M": 77, "N": 5003, "K": 2064, "out": "fp32"},
        # prefill through a gate/up projection: bound by the tensor cores
        {"name": "int8_prefill", "op": "gemm", "M": 4096, "N": 28672, "K": 8192, "out": "bf16"},
        # the gradients of one small layer: launch latency
        {"name": "clip_small", "op": "clip", "layers": 1, "I": 136, "K": 64, "type": "fp32", "max_norm": 1.0},
        # the gradients of a model of eight layers, 0.8 billion values
        {"name": "clip_large", "op": "clip", "layers": 8, "I": 8192, "K": 4096, "type": "bf16", "max_norm": 1.0},
    ]


def _count(rng, lo, hi):
    """A number of lo..hi, spread over its logarithm: odd, or a power of two."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.3:
        v = 1 << max(0, v.bit_length() - 1)
    else:
        v |= 1
    return max(lo, min(hi, v))


def _width(rng, lo, hi, step):
    """A width: one of the usual ones, or an odd multiple of `step`."""
    if rng.random() < 0.4:
        return rng.choice([v for v in (512, 1024, 2048, 2816, 4096, 6144, 8192, 14336, 28672) if lo <= v <= hi])
    return step * min(hi // step, _count(rng, max(1, lo // step), hi // step - 1) | 1)


def draw(rng):
    op = rng.choice(["gated", "gated", "train", "quantize", "gemm", "gemm", "clip"])
    if op in ("gated", "train"):
        while True:
            c = {"op": op, "M": _count(rng, 1, 8192), "I": _width(rng, 64, 14336, 8), "K": _width(rng, 64, 8192, 8),
                 "type": rng.choice(["bf16", "fp16"]), "act": rng.choice(["silu", "gelu_tanh"])}
            if c["M"] * c["I"] * c["K"] <= (4096 * 14336 * 8192 // 2 if op == "gated" else 4099 * 8192 * 4096):
                return c
    if op == "quantize":
        return {"op": op, "M": _count(rng, 1, 8192), "K": _width(rng, 256, 8192, 16), "type": rng.choice(["bf16", "fp16"])}
    if op == "gemm":
        while True:
            c = {"op": op, "M": _count(rng, 1, 8192), "N": _width(rng, 128, 28672, 1), "K": _width(rng, 256, 8192, 16),
                 "out": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
            if c["M"] * c["N"] * c["K"] <= 4096 * 28672 * 8192 // 2:
                return c
    while True:
        c = {"op": op, "layers": _count(rng, 1, 24), "I": _width(rng, 64, 8192, 8), "K": _width(rng, 64, 8192, 8),
             "type": rng.choice(["bf16", "fp16", "fp32"]), "max_norm": rng.choice([0.5, 1.0, 1e6])}
        if c["layers"] * c["I"] * c["K"] * (2 if c["type"] == "fp32" else 1) <= 8 * 8192 * 4096:
            return c


# ---- inputs ------------------------------------------------------------------------------------


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K, dtype):
    """Activations: N(0, 1), one value in a thousand twenty times as large."""
    x = _normal(g, M, K)
    x *= torch.where(torch.rand(M, K, generator=g, device="cuda") < 1e-3, 20.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("gated", "train"):
        M, I, K, dtype = case["M"], case["I"], case["K"], TYPES[case["type"]]
        s["x"] = _normal(g, M, K).to(dtype)
        s["wg"] = (_normal(g, I, K) * K ** -0.5).to(dtype)
        s["wu"] = (_normal(g, I, K) * K ** -0.5).to(dtype)
        if op == "train":
            s["dh"] = (_normal(g, M, I) * 0.05).to(dtype)
    elif op == "quantize":
        s["x"] = _activations(g, case["M"], case["K"], TYPES[case["type"]])
    elif op == "gemm":
        s["a"], s["sa"] = _quantize(_activations(g, case["M"], case["K"], torch.bfloat16))
        s["b"], s["sb"] = _quantize((_normal(g, case["N"], case["K"]) * 0.02).bfloat16())
    else:
        # per layer: gate, up and down weights, a norm's weight in fp32 and a bias of an odd size
        dtype, I, K = TYPES[case["type"]], case["I"], case["K"]
        s["grads"] = []
        for _ in range(case["layers"]):
            s["grads"] += [(_normal(g, *shape) * 1e-2).to(dtype) for shape in ((I, K), (I, K), (K, I))]
            s["grads"] += [_normal(g, K) * 1e-1, (_normal(g, I + 1) * 1e-1).to(dtype)]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ---- plain forms ---------------------------------------------------------------------------------


def _gate_factor(g, act):
    """(sigma, act(g) = g sigma, d sigma's argument / d g)."""
    if act == "silu":
        return torch.sigmoid(g), torch.ones_like(g)
    # the tanh form of gelu: 0.5 (1 + tanh(u)) = sigmoid(2 u)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return torch.sigmoid(c * (g + 0.044715 * g * g * g)), c * (1.0 + 3 * 0.044715 * g * g)


def _plain_gated(s, c):
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    sig, slope = _gate_factor(g, c["act"])
    a = g * sig
    h = a * u
    dtype = s["x"].dtype
    if c["op"] == "gated":
        return h.to(dtype)
    dh = s["dh"].float()
    dg = dh * u * (sig + a * (1.0 - sig) * slope)
    du = dh * a
    return {"h": h.to(dtype), "dx": (dg @ wg + du @ wu).to(dtype), "dw_gate": (dg.t() @ x).to(dtype),
            "dw_up": (du.t() @ x).to(dtype)}


def _quantize(x):
    """Codes [M, K] and scales [M]: the largest value of a row becomes 127."""
    v = x.float()
    amax = v.abs().amax(1)
    some = amax > 0
    inv = torch.where(some, 127.0 / torch.where(some, amax, torch.ones_like(amax)), torch.ones_like(amax))
    scale = torch.where(some, amax / 127.0, torch.ones_like(amax))
    return torch.round(v * inv[:, None]).to(torch.int8), scale


def _plain_gemm(s, c):
    # sums over 1,024 of K are whole numbers below 2^24: exact in fp32
    total = torch.zeros(c["M"], c["N"], dtype=torch.int32, device="cuda")
    for k in range(0, c["K"], 1024):
        total += (s["a"][:, k:k + 1024].float() @ s["b"][:, k:k + 1024].float().t()).int()
    y = total.float()
    y *= s["sa"][:, None]
    y *= s["sb"]
    return y.to(TYPES[c["out"]])


def _plain_clip(s, c):
    total = sum((t.double() * t.double()).sum() for t in s["grads"])
    norm = total.sqrt().float()
    factor = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_((t.float() * factor).to(t.dtype))
    return {"norm": norm.view(1), "grads": s["out"]}


def _plain(s):
    c = s["case"]
    if c["op"] in ("gated", "train"):
        return _plain_gated(s, c)
    if c["op"] == "quantize":
        return dict(zip("qs", _quantize(s["x"])))
    return _plain_gemm(s, c) if c["op"] == "gemm" else _plain_clip(s, c)


# ---- the library's calls ----------------------------------------------------------------------------


def _own(s):
    import moe_nvfp4_gemm_gb300 as m
    c = s["case"]
    if c["op"] == "gated":
        return m.nvfp4_gated_ffn(s["x"], s["wg"], s["wu"], activation=c["act"])
    if c["op"] == "train":
        h, gate, up = m.nvfp4_gated_ffn(s["x"], s["wg"], s["wu"], activation=c["act"], save=True)
        dx, dwg, dwu = m.nvfp4_gated_ffn_backward(s["x"], s["wg"], s["wu"], gate, up, s["dh"], activation=c["act"])
        return {"h": h, "dx": dx, "dw_gate": dwg, "dw_up": dwu}
    if c["op"] == "quantize":
        return dict(zip("qs", m.nvfp4_int8_quantize(s["x"])))
    if c["op"] == "gemm":
        return m.nvfp4_int8_gemm(s["a"], s["sa"], s["b"], s["sb"], c["M"], c["N"], c["K"], out_dtype=TYPES[c["out"]])
    norm = m.nvfp4_grad_clip(s["grads"], c["max_norm"], out=s["out"])
    return {"norm": norm, "grads": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- definitions in 64 bits ----------------------------------------------------------------------


def _exact_act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        e = torch.exp(-g)
        return g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
    r = math.sqrt(2 / math.pi)
    t = torch.tanh(r * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * r * (1 + 0.134145 * g * g)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("gated", "train"):
        x = s["x"].double()
        gate, up = torch.matmul(x, s["wg"].double().T), torch.matmul(x, s["wu"].double().T)
        a, slope = _exact_act(gate, c["act"])
        if c["op"] == "gated":
            return a * up
        dh = s["dh"].double()
        d_up = a * dh
        d_gate = slope * up * dh
        dx = torch.matmul(d_gate, s["wg"].double())
        dx += torch.matmul(d_up, s["wu"].double())
        return {"h": a * up, "dx": dx, "dw_gate": torch.matmul(d_gate.T, x), "dw_up": torch.matmul(d_up.T, x)}
    if c["op"] == "quantize":
        x = s["x"].double()
        top = torch.maximum(x.max(1).values, -x.min(1).values)
        scale = torch.where(top > 0, top / 127, 1.0)
        return {"q": x / scale[:, None], "s": scale}
    if c["op"] == "gemm":
        a = s["a"].double() * s["sa"].double()[:, None]
        y = torch.empty(c["M"], c["N"], dtype=torch.float64, device="cuda")
        for n in range(0, c["N"], 4096):
            y[:, n:n + 4096] = a @ (s["b"][n:n + 4096].double() * s["sb"][n:n + 4096].double()[:, None]).T
        return y
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
    factor = min(1.0, c["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "grads": [t.double() * factor for t in s["grads"]]}


def work(case):
    c = case
    if c["op"] in ("gated", "train"):
        M, I, K = c["M"], c["I"], c["K"]
        if c["op"] == "gated":  # x, both weights, h
            return {"bytes": 2 * (M * K + 2 * I * K + M * I), "flops": 4 * M * I * K}
        # x, the weights and dh in; h, dx and the weights' gradients out
        return {"bytes": 2 * (2 * M * K + 4 * I * K + 2 * M * I), "flops": 12 * M * I * K}
    if c["op"] == "quantize":
        return {"bytes": 3 * c["M"] * c["K"] + 4 * c["M"], "flops": 3 * c["M"] * c["K"]}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * K + 4 * (M + N) + M * N * (4 if c["out"] == "fp32" else 2), "flops": 2 * M * N * K}
    I, K, size = c["I"], c["K"], 4 if c["type"] == "fp32" else 2
    values, n_bytes = 3 * I * K + K + I + 1, (3 * I * K + I + 1) * size + 4 * K
    return {"bytes": 2 * c["layers"] * n_bytes, "flops": 3 * c["layers"] * values}

"""The MoE layer of examples/moe_fp8_layer.py: router, quantiser and grouped products together, with
padding tokens, against torch in fp32 on the same quantised weights; the same routing in front of
NVFP4 experts; the router's gradient through the layer against differences.

Rounding an activation to E4M3 is off by at most 2^-4 of it, 2^-4 / sqrt(3) = 3.6 % in the mean square
when it is spread evenly; a product of many keeps that relative size (independent errors), and the
layer rounds twice (input and activation): 5.2 % at most, 4 % or less for values that fill a binade
evenly. Bound: 6 % of the norm.
"""
import os
import sys

import numpy as np
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import moe_fp8_layer
    return moe_fp8_layer


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (37, 16, 4, 512, 272), (300, 8, 3, 1040, 384)])
@pytest.mark.parametrize("padded", [False, True])
def test_layer(ex, T, E, k, H, I, padded):
    g = torch.Generator(device=dev()).manual_seed(T)
    x = torch.randn(T, H, generator=g, device=dev()).bfloat16()
    logits = torch.randn(T, E, generator=g, device=dev())
    valid = torch.rand(T, generator=g, device=dev()) < 0.7 if padded else None
    if padded:
        x[~valid] = torch.nan  # what padding tokens hold must not matter
    experts = ex.Fp8Experts(E, H, I, g)
    y, r, out = ex.forward(x, logits, experts, k, valid)
    clean = x if valid is None else torch.where(valid[:, None], x, torch.zeros_like(x))
    want = ex.reference(clean, logits, experts, k, valid)
    assert torch.isfinite(y).all()
    assert float((y.float() - want).norm()) <= 0.06 * float(want.norm()) + 1e-6
    if padded:
        assert (y[~valid] == 0).all()


def test_routing_feeds_nvfp4_experts(ex):
    T, E, k, H, N = 50, 6, 2, 512, 256
    g = torch.Generator(device=dev()).manual_seed(3)
    x = torch.randn(T, H, generator=g, device=dev()).bfloat16()
    logits = torch.randn(T, E, generator=g, device=dev())
    parts = []
    for e in range(E):
        w = (torch.randn(N, H, generator=g, device=dev()) * 0.02).bfloat16()
        gw = m.nvfp4_amax(w)[1]
        parts.append((*m.nvfp4_quantize(w, gw), gw))
    w_gu = (torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), torch.cat([p[2] for p in parts]))
    y, r = ex.forward_nvfp4_gate_up(x, logits, w_gu, k)
    off = r.expert_offsets.tolist()
    q, sf = m.nvfp4_quantize(x, gx := m.nvfp4_amax(x)[1])
    for e in range(E):  # each expert's rows equal the dense product of the gathered tokens
        tok = r.row_token[off[e]:off[e + 1]].long()
        if len(tok):
            qe, se = m.nvfp4_quantize(x[tok].contiguous(), gx)
            want = m.nvfp4_gemm(qe, se, gx, parts[e][0], parts[e][1], parts[e][2], len(tok), N, H)
            got = y[off[e]:off[e + 1]]
            assert float((got.float() - want.float()).norm()) <= 1e-2 * float(want.float().norm())


def test_router_gradient_through_the_layer(ex):
    """d logits of sum(dy y) + coef L, with the expert outputs held, by central differences in 64 bits
    (error h^2 / 6 of the third derivative plus rounding / h; h = 1e-4)."""
    T, E, k, H, I = 40, 8, 2, 256, 128
    g = torch.Generator(device=dev()).manual_seed(5)
    x = torch.randn(T, H, generator=g, device=dev()).bfloat16()
    logits = torch.randn(T, E, generator=g, device=dev())
    valid = torch.rand(T, generator=g, device=dev()) < 0.8
    dy = torch.randn(T, H, generator=g, device=dev()).bfloat16()
    experts = ex.Fp8Experts(E, H, I, g)
    _, r, out = ex.forward(x, logits, experts, k, valid)
    coef = 0.7
    d = ex.router_step(logits, r, out, dy, coef, valid).double().cpu().numpy()
    l0 = logits.double().cpu().numpy()
    ok = valid.cpu().numpy()
    idx = r.topk_idx.cpu().numpy()
    rows = r.slot_row.cpu().numpy()
    o, dyn = out.double().cpu().numpy(), dy.double().cpu().numpy()
    gain = np.where(rows >= 0, np.einsum("th,tkh->tk", dyn, o[np.maximum(rows, 0)]), 0.0)
    counts, n = r.counts.cpu().numpy(), int(r.routed_tokens)

    def value(l):
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        p = p * ok[:, None]
        w = np.where(idx >= 0, np.take_along_axis(p, np.maximum(idx, 0), 1), 0.0)
        w = w / np.where(w.sum(1) > 0, w.sum(1), 1.0)[:, None]
        return (w * gain).sum() + coef * E * (counts / (n * k) * p.sum(0) / n).sum()

    for seed in range(3):
        v = np.random.default_rng(seed).standard_normal(l0.shape)
        h = 1e-4
        num = (value(l0 + h * v) - value(l0 - h * v)) / (2 * h)
        assert abs(num - (d * v).sum()) <= 1e-4 * np.abs(d * v).sum() + 1e-6

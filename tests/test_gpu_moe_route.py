"""GPU checks of the MoE router (nvfp4_moe_route) and its gradient against 64-bit restatements.

Tolerances. Indices, rows and counts are equal. A probability exp(x) / sum, x = l - max, is off
by the rounding of x and of x log2(e) (relative 3 |x| 2^-24 in all), of ex2 (2^-22), of the sum and
the reciprocal (a few 2^-24): (3 |x| + 32) 2^-24 relative, down to the smallest normal fp32
number, 2^-126, below which no relative bound holds. A gradient p (G - sum p G) adds a few
roundings of its terms: the same factor times p (|G| + sum p |G|), plus the output's own rounding.
"""
import numpy as np
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make_logits(T, E, seed, bf16=False, masked=0.0, off=0.0, scale=1.0, empty=0.0):
    """Logits with ties, and with `masked` padding tokens (their rows NaN and infinities), `off`
    of the experts at -inf, `empty` of the rows at -inf throughout."""
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) * scale).astype(np.float32)
    l = np.round(l * 64) / 64  # many equal values
    l[rng.random((T, E)) < off] = -np.inf
    l[rng.random(T) < empty] = -np.inf
    valid = None
    if masked:
        valid = rng.random(T) >= masked
        junk = np.array([np.nan, np.inf, -np.inf, -3.4e38], np.float32)
        l[~valid] = junk[rng.integers(0, 4, (int((~valid).sum()), E))]
    t = torch.from_numpy(l).to(dev())
    t = t.bfloat16() if bf16 else t
    v = None if valid is None else torch.from_numpy(valid).to(dev())
    return t, v


def reference(logits, valid, k, renorm):
    l = logits.double().cpu().numpy().copy()
    T, E = l.shape
    ok = np.ones(T, bool) if valid is None else valid.cpu().numpy().astype(bool)
    l[~ok] = -np.inf
    routed = (l > -np.inf).any(1)
    x = l - np.where(routed, l.max(1, initial=-np.inf), 0.0)[:, None]
    p = np.where(routed[:, None], np.exp(x), 0.0)
    p /= np.where(routed, p.sum(1), 1.0)[:, None]
    idx = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    xs = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if l[t, e] > -np.inf), key=lambda e: (-l[t, e], e))[:k]
        idx[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        xs[t, :len(order)] = np.abs(x[t, order])
    if renorm:
        w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
    rows = [[] for _ in range(E)]
    for t in range(T):
        for s in range(k):
            if idx[t, s] >= 0:
                rows[idx[t, s]].append((t, s))
    counts = np.array([len(r) for r in rows])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    slot_row = np.full((T, k), -1, np.int64)
    row_token = np.full(T * k, -1, np.int64)
    for e in range(E):
        for i, (t, s) in enumerate(rows[e]):
            slot_row[t, s] = offsets[e] + i
            row_token[offsets[e] + i] = t
    n = int(routed.sum())
    mean = p.sum(0) / max(n, 1)
    loss = E * (counts / max(n * k, 1) * mean).sum()
    return dict(p=p, x=np.where(p > 0, np.abs(np.where(np.isfinite(x), x, 0)), 0), idx=idx, w=w, xs=xs, counts=counts,
                offsets=offsets, slot_row=slot_row, row_token=row_token, n=n, mean=mean, loss=loss)


def check_route(logits, valid, k, renorm, r=None):
    r = m.nvfp4_moe_route(logits, k, renormalize=renorm, valid=valid) if r is None else r
    torch.cuda.synchronize()
    f = reference(logits, valid, k, renorm)
    for got, want in ((r.topk_idx, f["idx"]), (r.slot_row, f["slot_row"]), (r.counts, f["counts"]),
                      (r.expert_offsets, f["offsets"]), (r.row_token, f["row_token"])):
        assert np.array_equal(got.cpu().numpy(), want)
    assert int(r.routed_tokens) == f["n"]
    w = r.topk_w.double().cpu().numpy()
    most = f["x"].max(initial=0.0)
    assert np.all(np.abs(w - f["w"]) <= (3 * f["xs"] + 32) * U * f["w"] * (2 if renorm else 1) + 2.0 ** -126)
    mean = r.mean_prob.double().cpu().numpy()
    # a mean adds the rounding of its sums: at most the tokens of one warp, then the parts
    rel = (3 * most + 32 + logits.shape[0] / 8 + 320) * U
    assert np.all(np.abs(mean - f["mean"]) <= rel * f["mean"] + 1e-30)
    assert abs(float(r.balance_loss) - f["loss"]) <= (rel + 64 * U) * f["loss"]
    return r, f


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (1, 1, 1), (2, 3, 3), (7, 8, 2), (64, 256, 8), (65, 256, 8), (63, 60, 4),
                                   (130, 33, 5), (300, 64, 6), (257, 128, 8), (500, 160, 8), (97, 1024, 32), (33, 1000, 32),
                                   (1025, 512, 3), (3001, 256, 8), (5000, 16, 4), (70, 32, 32)])
@pytest.mark.parametrize("bf16", [False, True])
def test_route(T, E, k, bf16):
    logits, valid = make_logits(T, E, T * 7 + E, bf16)
    check_route(logits, valid, k, renorm=bool((T + E) % 2))


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (50, 256, 8), (333, 60, 6), (2777, 256, 8), (400, 1024, 32)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masked_tokens_and_experts(T, E, k, renorm):
    for bf16 in (False, True):
        logits, valid = make_logits(T, E, 3 * T + E, bf16, masked=0.3, off=0.5, empty=0.1)
        check_route(logits, valid, k, renorm)


def test_route_fewer_experts_on_than_slots():
    logits = torch.full((40, 64), -torch.inf, device=dev())
    logits[:, 5] = 1.0
    logits[::2, 63] = 1.0
    r, f = check_route(logits, None, 4, True)
    assert int(r.counts[5]) == 40 and int(r.counts[63]) == 20 and int(r.expert_offsets[64]) == 60


@pytest.mark.parametrize("T", [1, 40, 1000])
def test_route_nothing_to_route(T):
    logits = torch.full((T, 96), torch.nan, device=dev())
    valid = torch.zeros(T, dtype=torch.bool, device=dev())
    r = m.nvfp4_moe_route(logits, 4, valid=valid)
    assert (r.topk_idx == -1).all() and (r.topk_w == 0).all() and (r.row_token == -1).all() and (r.slot_row == -1).all()
    assert (r.counts == 0).all() and (r.expert_offsets == 0).all() and (r.mean_prob == 0).all()
    assert float(r.balance_loss) == 0.0 and int(r.routed_tokens) == 0
    d = m.nvfp4_moe_route_backward(logits, r, d_w=torch.ones(T, 4, device=dev()), d_loss=torch.ones(1, device=dev()),
                                   valid=valid)
    assert (d == 0).all()


def test_route_no_tokens():
    r = m.nvfp4_moe_route(torch.empty(0, 16, device=dev()), 2)
    assert r.topk_idx.shape == (0, 2) and r.row_token.numel() == 0 and (r.expert_offsets == 0).all()
    assert float(r.balance_loss) == 0.0 and int(r.routed_tokens) == 0 and (r.mean_prob == 0).all()
    d = m.nvfp4_moe_route_backward(torch.empty(0, 16, device=dev()), r)
    assert d.shape == (0, 16)


@pytest.mark.parametrize("T", [20, 900])
def test_route_signed_zeros_tie_and_extremes(T):
    logits = torch.zeros(T, 64, device=dev())
    logits[:, ::2] = -0.0
    r, _ = check_route(logits, None, 6, True)
    assert (r.topk_idx == torch.arange(6, device=dev())).all()
    logits[:, 10] = 3.0e38
    logits[:, 11] = -3.4028234663852886e38  # the type's lowest value is a value, not a mask
    check_route(logits, None, 32, False)


def test_route_skewed_to_one_expert():
    logits, _ = make_logits(4100, 256, 5)
    logits[:, 200] += 100.0
    r, _ = check_route(logits, None, 8, True)
    assert int(r.counts[200]) == 4100


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_route_unaligned_rows(offset):
    """Rows that no vector load can read: the base is only element-aligned."""
    for bf16 in (False, True):
        base, _ = make_logits(131, 257, 9, bf16)
        flat = base.flatten()[offset:offset + 130 * 256].view(130, 256)
        r, f = check_route(flat, None, 8, False)
        check_backward(flat, None, 8, False, r, f, seed=1)


def test_route_repeats_bit_for_bit_and_in_a_graph_on_another_stream():
    logits, valid = make_logits(20000, 256, 77, masked=0.1)
    a = m.nvfp4_moe_route(logits, 8, renormalize=True, valid=valid)
    b = m.nvfp4_moe_route(logits, 8, renormalize=True, valid=valid)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            c = m.nvfp4_moe_route(logits, 8, renormalize=True, valid=valid)
            d = m.nvfp4_moe_route_backward(logits, c, d_loss=torch.ones(1, device=dev()), renormalize=True, valid=valid)
        for _ in range(3):
            g.replay()
    st.synchronize()
    for x, y in zip(a, c):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
    assert torch.isfinite(d).all()


# ---- gradient ---------------------------------------------------------------------------------


def reference_backward(f, k, renorm, dw, dl):
    p, idx, n = f["p"], f["idx"], max(f["n"], 1)
    T, E = p.shape
    G = np.broadcast_to(dl * E * f["counts"] / (k * n * n), (T, E)).copy()
    mag = np.abs(G)
    extra = np.zeros((T, E))
    xmag = np.zeros((T, E))
    sel = idx >= 0
    for s in range(k):
        t = np.nonzero(sel[:, s])[0]
        e = idx[t, s]
        if renorm:
            d = dw - (np.where(sel, f["w"] * dw, 0)).sum(1, keepdims=True)
            extra[t, e] = (f["w"] * d)[t, s]
            xmag[t, e] = (f["w"] * (np.abs(dw) + np.where(sel, f["w"] * np.abs(dw), 0).sum(1, keepdims=True)))[t, s]
        else:
            G[t, e] += dw[t, s]
            mag[t, e] += np.abs(dw[t, s])
    d = p * (G - (p * G).sum(1, keepdims=True)) + extra
    bound = (6 * f["x"].max(initial=0.0) + 160) * U * (p * (mag + (p * mag).sum(1, keepdims=True)) + xmag)
    return d, bound


def check_backward(logits, valid, k, renorm, r, f, seed, with_w=True, with_l=True):
    rng = np.random.default_rng(seed)
    T, E = logits.shape
    dw = rng.standard_normal((T, k)).astype(np.float32) if with_w else np.zeros((T, k), np.float32)
    dl = np.float32(rng.standard_normal() * T) if with_l else np.float32(0)
    d = m.nvfp4_moe_route_backward(logits, r, d_w=torch.from_numpy(dw).to(dev()) if with_w else None,
                                   d_loss=torch.tensor([dl], device=dev()) if with_l else None, renormalize=renorm,
                                   valid=valid)
    assert d.dtype == logits.dtype
    want, bound = reference_backward(f, k, renorm, dw.astype(np.float64), float(dl))
    got = d.double().cpu().numpy()
    # a bf16 output rounds by 2^-9 relative; values below the smallest normal may flush
    out = 2.0 ** -8 * np.abs(want) if d.dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= bound + out + 1e-37)
    return dw, dl, want


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (3, 2, 1), (40, 8, 2), (130, 60, 5), (257, 256, 8), (99, 1000, 32),
                                   (2500, 128, 4)])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_formula(T, E, k, renorm):
    for bf16, masked in ((False, 0.0), (True, 0.25), (False, 0.25)):
        logits, valid = make_logits(T, E, T + E, bf16, masked=masked, off=0.2 if masked else 0.0, empty=0.05)
        r = m.nvfp4_moe_route(logits, k, renormalize=renorm, valid=valid)
        f = reference(logits, valid, k, renorm)
        check_backward(logits, valid, k, renorm, r, f, T)
        check_backward(logits, valid, k, renorm, r, f, T, with_w=False)
        check_backward(logits, valid, k, renorm, r, f, T, with_l=False)


@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(renorm):
    """Directional derivative of sum(dw w) + dl L (selection and counts held) by central differences in 64 bits."""
    T, E, k = 60, 24, 4
    logits, valid = make_logits(T, E, 4, masked=0.2, off=0.1)
    r = m.nvfp4_moe_route(logits, k, renormalize=renorm, valid=valid)
    f = reference(logits, valid, k, renorm)
    dw, dl, want = check_backward(logits, valid, k, renorm, r, f, 8)
    d = m.nvfp4_moe_route_backward(logits, r, d_w=torch.from_numpy(dw).to(dev()), d_loss=torch.tensor([dl], device=dev()),
                                   renormalize=renorm, valid=valid).double().cpu().numpy()
    routed = f["p"].sum(1) > 0
    l0 = np.where(routed[:, None], logits.double().cpu().numpy(), 0.0)
    idx, sel = np.maximum(f["idx"], 0), f["idx"] >= 0

    def value(l):
        p = np.where(routed[:, None], np.exp(l - l.max(1, keepdims=True)), 0.0)
        p /= np.where(routed, p.sum(1), 1.0)[:, None]
        w = np.where(sel, np.take_along_axis(p, idx, 1), 0.0)
        if renorm:
            w = w / np.where(w.sum(1) > 0, w.sum(1), 1.0)[:, None]
        return (dw * w).sum() + dl * E * (f["counts"] / (f["n"] * k) * p.sum(0) / f["n"]).sum()

    for seed in range(4):
        v = np.random.default_rng(seed).standard_normal((T, E))
        h = 1e-4  # central differences: error h^2 / 6 of the third derivative, and 1e-16 / h of rounding
        num = (value(l0 + h * v) - value(l0 - h * v)) / (2 * h)
        scale = np.abs(d * v).sum()
        assert abs(num - (d * v).sum()) <= 1e-5 * scale + 1e-7


# ---- refusals ------------------------------------------------------------------------------------


def test_route_refusals():
    l = torch.zeros(4, 16, device=dev())
    for bad in (l.double(), l.t(), l.cpu(), l[0]):
        with pytest.raises(TypeError):
            m.nvfp4_moe_route(bad, 2)
    with pytest.raises(TypeError):
        m.nvfp4_moe_route(l, 2, valid=torch.ones(3, dtype=torch.bool, device=dev()))
    for k, status in ((0, -1), (17, -1), (-1, -1)):
        with pytest.raises(m.NVFP4Error) as e:
            m.nvfp4_moe_route(l, k)
        assert e.value.status == status
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_moe_route(torch.zeros(2, 1025, device=dev()), 2)
    assert e.value.status == -2
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_moe_route(torch.zeros(2, 64, device=dev()), 33)
    assert e.value.status == -2
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_moe_route(l, 2, workspace=torch.empty(4, dtype=torch.uint8, device=dev()))
    assert e.value.status == -6
    r = m.nvfp4_moe_route(l, 2)
    with pytest.raises(TypeError):
        m.nvfp4_moe_route_backward(l, r, d_w=torch.zeros(4, 3, device=dev()))
    with pytest.raises(TypeError):
        m.nvfp4_moe_route_backward(l, r, d_loss=torch.zeros(1, device=dev(), dtype=torch.float64))
    with pytest.raises(TypeError):
        m.nvfp4_moe_route_backward(torch.zeros(5, 16, device=dev()), r)

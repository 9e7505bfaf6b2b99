"""NaN and +inf logits in valid tokens: such a token is routed (a NaN is never selected, +inf first), its weights,
the means, the loss and its gradient are NaN, and every other row's are those without it. Tolerances as in
test_gpu_moe_route.py."""
import numpy as np
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev
from tests.test_gpu_moe_route import U, make_logits, reference, reference_backward

pytestmark = pytest.mark.gpu


def poisoned(T, E, seed, bf16):
    """Logits, valid, and which valid rows hold a NaN or +inf: one NaN, a lane's whole share of NaN, NaN alone, NaN
    among -inf, NaN among more equal values than a warp ranks at once, +inf, negative NaN."""
    logits, valid = make_logits(T, E, seed, bf16, masked=0.2)
    l = logits.float().cpu().numpy()
    on = valid.cpu().numpy()
    rng = np.random.default_rng(seed)
    bad = np.zeros(T, bool)
    share = 1
    while share * 32 < E:
        share *= 2
    negative = np.array([0xFFC00000], np.uint32).view(np.float32)[0]
    for t in range(T):
        kind = t % 11
        if kind > 6 and T > 7:
            continue
        bad[t] = True
        on[t] = True
        if l.shape[1] and not np.isfinite(l[t]).all():
            l[t] = rng.standard_normal(E).astype(np.float32)
        at = int(rng.integers(E))
        if kind == 0:
            l[t, at] = np.nan
        elif kind == 1:
            first = at // share * share
            l[t, first:first + share] = np.nan
        elif kind == 2:
            l[t] = np.nan
        elif kind == 3:
            l[t] = -np.inf
            l[t, at] = np.nan
        elif kind == 4:
            l[t] = 1.5
            l[t, at] = np.nan
        elif kind == 5:
            l[t, at] = np.inf
        else:
            l[t, at] = negative
    t = torch.from_numpy(l).to(dev())
    return t.bfloat16() if bf16 else t, torch.from_numpy(on).to(dev()), bad


@pytest.mark.parametrize("T", [1, 16, 60, 900])
@pytest.mark.parametrize("E,k", [(8, 2), (32, 4), (60, 5), (64, 6), (256, 8), (1024, 32)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_poisoned_rows(T, E, k, renorm, bf16):
    logits, valid, bad = poisoned(T, E, T + E + 1, bf16)
    r = m.nvfp4_moe_route(logits, k, renormalize=renorm, valid=valid)
    l = logits.double()
    f = reference(torch.where(l.isnan(), -torch.inf, l).clamp(max=1e300), valid, k, renorm)
    on = valid.cpu().numpy()
    n = int((on & (f["p"].sum(1) > 0) | bad).sum())
    for got, want in ((r.topk_idx, f["idx"]), (r.slot_row, f["slot_row"]), (r.counts, f["counts"]),
                      (r.expert_offsets, f["offsets"]), (r.row_token, f["row_token"])):
        assert np.array_equal(got.cpu().numpy(), want)
    assert int(r.routed_tokens) == n
    w = r.topk_w.double().cpu().numpy()
    assert np.isnan(w[bad]).all()
    assert np.all(np.abs(w - f["w"])[~bad] <= ((3 * f["xs"] + 32) * U * f["w"] * (2 if renorm else 1) + 2.0 ** -126)[~bad])
    assert r.mean_prob.isnan().all() and r.balance_loss.isnan().all()

    rng = np.random.default_rng(T)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dl = np.float32(rng.standard_normal() * T)
    f["n"] = n
    f["p"][bad] = 0.0  # their part of the 64-bit gradient is not looked at
    f["x"][bad] = 0.0
    f["w"][bad] = 0.0
    for with_w, with_l in ((True, True), (True, False), (False, True)):
        d = m.nvfp4_moe_route_backward(logits, r, d_w=torch.from_numpy(dw).to(dev()) if with_w else None,
                                       d_loss=torch.tensor([dl], device=dev()) if with_l else None, renormalize=renorm,
                                       valid=valid).double().cpu().numpy()
        want, bound = reference_backward(f, k, renorm, dw.astype(np.float64) * with_w, float(dl) * with_l)
        out = 2.0 ** -8 * np.abs(want) if bf16 else 0.0
        assert np.isnan(d[bad]).all()
        assert np.all((np.abs(d - want) <= bound + out + 1e-37)[~bad])


@pytest.mark.parametrize("T", [3, 500])
def test_padding_with_nan_has_no_effect(T):
    logits = torch.zeros(T, 16, device=dev())
    logits[1:] = torch.nan
    valid = torch.zeros(T, dtype=torch.bool, device=dev())
    valid[0] = True
    r = m.nvfp4_moe_route(logits, 2, valid=valid)
    assert int(r.routed_tokens) == 1 and float(r.balance_loss) == 1.0 and torch.isfinite(r.topk_w).all()
    d = m.nvfp4_moe_route_backward(logits, r, d_loss=torch.ones(1, device=dev()), valid=valid)
    assert (d[1:] == 0).all() and torch.isfinite(d).all()

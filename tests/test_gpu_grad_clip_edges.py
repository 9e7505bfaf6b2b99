"""Clipping at its edges: no limit, and norms beyond fp32."""
import math

import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_grad_clip import TYPES, norm64, tensors

pytestmark = pytest.mark.gpu


# one launch, and two
@pytest.mark.parametrize("n", [5000, 400000])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_no_limit_scales_nothing(n, value):
    """Without a limit the results are the gradients, whatever the norm."""
    grads = tensors(1, [n, 300, 40], TYPES)
    grads[0][777] = value
    before = [t.clone() for t in grads]
    out = [torch.full_like(t, 3.0) for t in grads]
    norms = [m.nvfp4_grad_clip(grads, out=out), m.nvfp4_grad_clip(grads, math.inf), m.nvfp4_grad_clip(grads)]
    assert all((x.isnan() if math.isnan(value) else x == math.inf).all() for x in norms)
    for t, o, b in zip(grads, out, before):
        assert torch.equal(t.nan_to_num(nan=9.0), b.nan_to_num(nan=9.0)) and torch.equal(o.nan_to_num(nan=9.0), b.nan_to_num(nan=9.0))


@pytest.mark.parametrize("n", [2, 300, 400000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("limit", [1e-40, 1e-30, 1e-3, 1.0, 3e38])
@pytest.mark.parametrize("largest", [3.3e38, 1e38])
def test_norm_beyond_fp32(n, dtype, limit, largest):
    """Finite gradients of all sizes whose norm no fp32 number holds, or just still holds: the norm is infinite as an fp32 number,
    the factor is that of the norm in 64 bits, and small results keep all their bits. A result is rounded to fp32 twice
    at most (the factor, the product) and once to the type, and the norm itself is off as everywhere."""
    limit = float(torch.tensor(limit))  # as the call takes it
    g = torch.Generator(device="cuda").manual_seed(n)
    t = ((torch.rand(n, generator=g, device="cuda") - 0.5) * largest / 2 * torch.exp2(-(torch.arange(n, device="cuda") % 230).float())).to(dtype)
    t[0], t[1] = largest, -0.97 * largest
    want = norm64([t])
    before = t.double()
    out = torch.empty_like(t)
    for norm in (m.nvfp4_grad_clip([t], limit, out=[out]), m.nvfp4_grad_clip([t], limit)):
        if want > 3.5e38:
            assert float(norm) == math.inf
        else:
            assert abs(float(norm) - want) <= 33 * 2.0 ** -24 * want
    value = before * min(1.0, limit / want)
    # half a step of the type, and of its smallest numbers (bf16: 2^-133, fp32: 2^-149); of a factor below 2^-252 the fp32 part is
    # off by 2^-150 at most, times a value of up to 4
    tol = (torch.finfo(dtype).eps / 2 * 1.01 + 33 * 2.0 ** -24 + 2.0 ** -22) * value.abs()
    tol += 1.01 * (2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150) + 2.0 ** -148
    for r in (t, out):
        assert ((r.double() - value).abs() <= tol).all()

"""Clipping at its edges: no limit, norms beyond fp32, and the same values at other addresses."""
import math

import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_grad_clip import TYPES, check, norm64, tensors

pytestmark = pytest.mark.gpu

IDS = ["bf16", "fp16", "fp32"]


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


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("sizes", [[20011], [1], [7], [8], [9], [15, 17, 16384, 16385, 16391], [3, 33001, 300007, 5]],
                         ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("scale", [1e-2, 1e-30])
def test_addresses_change_no_bit(dtype, sizes, scale):
    """The same gradients at every offset from a 16-byte boundary: the same norm and the same results, bit for bit. (At
    1e-30 the squares leave fp32's range and are added again in fp64.)"""
    if dtype == torch.float16:
        scale = max(scale, 1e-4)
    grads = tensors(len(sizes), sizes, [dtype] * len(sizes), scale)
    limit = 0.3 * norm64(grads)
    first = None
    for off in range(16 // grads[0].element_size()):
        views = []
        for i, t in enumerate(grads):  # each gradient at another offset, NaN around it
            flat = torch.full((t.numel() + 32,), float("nan"), dtype=dtype, device="cuda")
            at = (off * (2 * i + 1)) % 8
            flat[at:at + t.numel()] = t
            views.append(flat[at:at + t.numel()])
        out = [torch.empty_like(t) for t in grads]
        norm = m.nvfp4_grad_clip(views, limit, out=out)
        alone = m.nvfp4_grad_clip(views)
        assert torch.equal(norm, alone)
        first = first or (norm, out)
        assert torch.equal(norm, first[0]) and all(torch.equal(a, b) for a, b in zip(out, first[1])), off
    check(m, grads, limit)


def test_short_gradients_at_every_offset():
    flat = tensors(5, [4096], [torch.bfloat16], 1.0)[0]
    for n in range(1, 41):
        for at in range(8):
            g = flat[at:at + n]
            want = norm64([g])
            assert abs(float(m.nvfp4_grad_clip([g])) - want) <= 33 * 2.0 ** -24 * want, (n, at)

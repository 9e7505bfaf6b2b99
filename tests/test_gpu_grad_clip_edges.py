"""Clipping at its edges: no limit."""
import math

import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_grad_clip import TYPES, tensors

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

"""The router's gradient is that of the forward call: what it was given (renormalize, valid) is kept with the
routing, and arguments that contradict it are refused instead of giving another function's gradient."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev
from tests.test_gpu_moe_route import check_backward, make_logits, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_backward_takes_what_the_routing_was_made_with(renorm, masked):
    T, E, k = 130, 60, 5
    logits, valid = make_logits(T, E, 3, masked=masked)
    r = m.nvfp4_moe_route(logits, k, renormalize=renorm, valid=valid)
    f = reference(logits, valid, k, renorm)
    dw, dl, _ = check_backward(logits, valid, k, renorm, r, f, 1)  # with the arguments, against 64 bits
    dw, dl = torch.from_numpy(dw).to(dev()), torch.tensor([dl], device=dev())
    want = m.nvfp4_moe_route_backward(logits, r, d_w=dw, d_loss=dl, renormalize=renorm, valid=valid)
    assert torch.equal(want, m.nvfp4_moe_route_backward(logits, r, d_w=dw, d_loss=dl))
    assert torch.equal(want, m.nvfp4_moe_route_backward(logits, r, dw, dl, renorm))
    with pytest.raises(TypeError):
        m.nvfp4_moe_route_backward(logits, r, d_w=dw, d_loss=dl, renormalize=not renorm, valid=valid)
    if valid is None:
        with pytest.raises(TypeError):
            m.nvfp4_moe_route_backward(logits, r, d_w=dw, valid=torch.ones(T, dtype=torch.bool, device=dev()))
    else:
        assert torch.equal(want, m.nvfp4_moe_route_backward(logits, r, d_w=dw, d_loss=dl, valid=valid.to(torch.uint8)))

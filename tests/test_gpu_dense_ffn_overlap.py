"""Results of the dense feed-forward calls beside their operands in one buffer: what shares no element is taken and right,
what does is refused."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_gated_ffn import check_backward, make

pytestmark = pytest.mark.gpu


def test_gradient_between_the_rows_of_an_operand():
    M, I, K = 2, 64, 256
    x, wg, wu, dh = make(M, I, K, torch.bfloat16, seed=1)
    _, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    wide = torch.full((M, 4096), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = x
    dx = wide.view(-1)[K:K + M * K].view(M, K)
    got = m.nvfp4_gated_ffn_backward(wide[:, :K], wg, wu, gate, up, dh, dx=dx)
    assert got[0] is dx and torch.equal(wide[:, :K], x) and (wide[0, K + M * K:] == 7).all() and (wide[1, K:] == 7).all()
    check_backward(x, wg, wu, gate, up, dh, "silu", *got)

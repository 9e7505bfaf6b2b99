"""Input gradient of the grouped FP8 product, dx = dy W_e for each expert's rows, through the experts' transposed
codes (128 x 128 blocks are their own transpose). Tolerances as in test_gpu_fp8.py; against the exact gradient
within what rounding an operand to E4M3 can do, as there."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev
from tests.test_gpu_fp8 import FP8, acts, blocks, check, decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [40, 100, 0, 130, 7], [300, 0, 520]])
@pytest.mark.parametrize("N,K", [(256, 384), (528, 272)])
def test_grouped_input_gradient(counts, N, K):
    E = len(counts)
    off = torch.tensor([0] + counts).cumsum(0)
    rows = int(off[-1])
    dy = acts(rows, N, 1, 0.1)
    w = [acts(N, K, 10 + e, 0.02) for e in range(E)]
    d, ds = m.nvfp4_fp8_quantize(dy)
    wt = torch.empty(E, K, N, dtype=FP8, device=dev())
    wts = torch.empty(E, blocks(K), blocks(N), device=dev())
    for e in range(E):
        _, _, wt[e], wts[e] = m.nvfp4_fp8_quantize(w[e], 128, transposed=True)
    dx = m.nvfp4_fp8_grouped_gemm(d, ds, wt, wts, off.int().to(dev()), E, rows, K, N)
    for e in range(E):
        if not counts[e]:
            continue
        r = slice(int(off[e]), int(off[e + 1]))
        A, B = decode(d[r], ds[:, r].contiguous(), 1), decode(wt[e], wts[e], 128)
        check(dx[r], A, B)
        X, W = dy[r].double(), w[e].double().t()
        one = lambda s, q, b: 2.0 ** -10 * decode(torch.ones_like(q, dtype=torch.float32).to(FP8), s, b)
        e1 = 2.0 ** -4 * X.abs() + one(ds[:, r].contiguous(), d[r], 1)
        e2 = 2.0 ** -4 * W.abs() + one(wts[e], wt[e], 128)
        true = X @ W.t()
        bound = e1 @ W.abs().t() + X.abs() @ e2.t() + e1 @ e2.t()
        out = 4e-3 * true.abs() + 4e-3 * bound + 1e-5 * (A.abs() @ B.abs().t())
        assert ((dx[r].double() - true).abs() <= bound + out).all()

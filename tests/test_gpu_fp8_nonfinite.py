"""NaN and infinities through the FP8 quantiser and products: a NaN leaves its block's scale and the other codes
alone and reaches only what its value enters; an infinity makes its block's values NaN."""
import numpy as np
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev
from tests.test_gpu_fp8 import acts, blocks, check, decode, ref_quantize

pytestmark = pytest.mark.gpu

NEGATIVE_NAN = -0x40  # bf16 0xFFC0 as int16


def with_nan(M, K, seed):
    """Scattered NaN of both signs, one at each corner of a block, a row of a block and a whole block of NaN."""
    x = acts(M, K, seed)
    g = torch.Generator(device=dev()).manual_seed(seed)
    hit = torch.rand(M, K, generator=g, device=dev()) < 0.01
    hit[0, 0] = hit[M - 1, K - 1] = True
    hit[M // 2, :min(128, K)] = True
    if M > 256:
        hit[128:256, 128:256] = True
    x[hit] = torch.nan
    neg = hit & (torch.rand(M, K, generator=g, device=dev()) < 0.5)
    x.view(torch.int16)[neg] = NEGATIVE_NAN
    return x, hit


def same(q, s, x, hit, block_rows):
    wq, ws = ref_quantize(torch.where(hit, torch.zeros_like(x), x), block_rows)
    assert np.array_equal(s.cpu().numpy(), ws)
    got, hit = q.cpu().view(torch.uint8), hit.cpu()
    assert torch.equal(got[~hit], wq.view(torch.uint8)[~hit])
    assert (got[hit] & 0x7F == 0x7F).all()


@pytest.mark.parametrize("M,K", [(1, 16), (3, 144), (130, 400), (300, 512)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_nan(M, K, block_rows):
    x, hit = with_nan(M, K, M + K)
    q, s = m.nvfp4_fp8_quantize(x, block_rows)
    same(q, s, x, hit, block_rows)
    q, s, qt, st = m.nvfp4_fp8_quantize(x, block_rows, transposed=True)
    same(q, s, x, hit, block_rows)
    pad = (M + 15) // 16 * 16 - M
    xt = torch.nn.functional.pad(x, (0, 0, 0, pad)).t().contiguous()
    same(qt, st, xt, torch.nn.functional.pad(hit, (0, 0, 0, pad)).t(), block_rows)
    if block_rows == 1:
        rows = torch.tensor([M - 1, 0, -1, M // 2], dtype=torch.int32, device=dev())
        q, s = m.nvfp4_fp8_quantize(x, row_token=rows)
        inside = (rows >= 0)[:, None]
        at = rows.clamp(min=0).long()
        same(q, s, torch.where(inside, x[at], torch.zeros_like(x[at])), hit[at] & inside, 1)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_infinity_makes_its_block_nan(block_rows):
    x = acts(200, 272, 5)
    x[3, 130] = torch.inf
    q, s, qt, st = m.nvfp4_fp8_quantize(x, block_rows, transposed=True)
    v = decode(q, s, block_rows)
    rows = slice(3, 4) if block_rows == 1 else slice(0, 128)
    assert v[rows, 128:256].isnan().all()
    v[rows, 128:256] = 0.0
    assert v.isfinite().all()
    vt = decode(qt, st, block_rows)[:, :200].t()
    cols = slice(130, 131) if block_rows == 1 else slice(128, 256)
    assert vt[0:128, cols].isnan().all() and vt[128:].isfinite().all()


@pytest.mark.parametrize("M", [1, 20, 100, 300])
@pytest.mark.parametrize("b_rows", [128, 1])
def test_products_pass_a_nan_on_to_its_row_alone(M, b_rows):
    N, K = 300, 656
    x = acts(M, K, 1)
    w = acts(N, K, 2, 0.02)
    x[M // 2, 200] = torch.nan
    a, sa = m.nvfp4_fp8_quantize(x)
    b, sb = m.nvfp4_fp8_quantize(w, b_rows)
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows)
    assert y[M // 2].isnan().all()
    keep = torch.arange(M, device=dev()) != M // 2
    A = decode(a, sa, 1)
    check(y[keep], A[keep], decode(b, sb, b_rows))
    w[7, 100] = torch.nan
    b, sb = m.nvfp4_fp8_quantize(w, b_rows)
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows)
    assert y[:, 7].isnan().all()
    cols = torch.arange(N, device=dev()) != 7
    check(y[keep][:, cols], A[keep], decode(b, sb, b_rows)[cols])

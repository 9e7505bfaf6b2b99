"""Block scales far from 1 through every form of the FP8 products. A product of two scales is rounded by 2^-24 of it
while it is a normal fp32 number, and by up to 2^-150 below 2^-126; a block's sum is below 2^24.7, so that a
block's error below the normal range is under 2^-125 (times sa, where sb meets the sum first)."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev
from tests.test_gpu_fp8 import FP8, blocks, decode

pytestmark = pytest.mark.gpu


def case(M, N, K, b_rows, sa_exp, sb_exp, seed):
    """Codes over E4M3's whole range, scales 2^exp times 1 to 2."""
    g = torch.Generator(device=dev()).manual_seed(seed)

    def codes(R):
        q = torch.randint(0, 256, (R, K), generator=g, device=dev(), dtype=torch.uint8)
        q[(q & 0x7F) == 0x7F] = 0  # no NaN
        return q.view(FP8)

    def scales(shape, exp):
        return (torch.rand(shape, generator=g, device=dev(), dtype=torch.float64) + 1.0).mul(2.0 ** exp).float()

    return (codes(M), scales((blocks(K), M), sa_exp), codes(N),
            scales((blocks(K), N) if b_rows == 1 else (blocks(N), blocks(K)), sb_exp))


def close(y, a, sa, b, sb, b_rows, floor):
    A, B = decode(a, sa, 1), decode(b, sb, b_rows)
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    bound = 1e-5 * mag + floor + (4e-3 * ref.abs() if y.dtype == torch.bfloat16 else 0.0)
    assert ((y.double() - ref).abs() <= bound).all()


FORMS = [(1, 300, 656), (20, 300, 2064), (20, 300, 656), (50, 300, 4112), (100, 300, 656), (300, 300, 656), (300, 260, 3088)]


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sa_exp,sb_exp", [(-63, -63), (-110, -16), (-16, -110), (50, 45), (90, -90), (-90, 90), (95, 0)])
def test_scales_in_the_normal_range(M, N, K, b_rows, out, sa_exp, sb_exp):
    a, sa, b, sb = case(M, N, K, b_rows, sa_exp, sb_exp, M + K)
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows, out_dtype=out)
    # an output below 2^-126 is itself rounded by up to 2^-150 in fp32, 2^-134 in bf16
    close(y, a, sa, b, sb, b_rows, 2.0 ** -134)


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("sa_exp,sb_exp", [(-80, -60), (-130, -17), (-17, -130), (-149, 0), (0, -149)])
def test_scales_below_it(M, N, K, b_rows, sa_exp, sb_exp):
    a, sa, b, sb = case(M, N, K, b_rows, sa_exp, sb_exp, M + K)
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows, out_dtype=torch.float32)
    close(y, a, sa, b, sb, b_rows, blocks(K) * 2.0 ** -125 * 2)  # sa is at most 2


@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [40, 100, 0, 130], [300, 0, 520, 200]])
@pytest.mark.parametrize("sa_exp,sb_exp", [(-63, -63), (-16, -110), (50, 45), (-80, -60)])
def test_grouped(counts, sa_exp, sb_exp):
    N, K, E = 264, 656, len(counts)
    off = torch.tensor([0] + counts).cumsum(0)
    rows = int(off[-1])
    a, sa, _, _ = case(rows, 1, K, 128, sa_exp, sb_exp, 1)
    w = [case(1, N, K, 128, sa_exp, sb_exp, 2 + e)[2:] for e in range(E)]
    y = m.nvfp4_fp8_grouped_gemm(a, sa, torch.stack([q.view(torch.uint8) for q, _ in w]).view(FP8),
                                 torch.stack([s for _, s in w]), off.int().to(dev()), E, rows, N, K)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            close(y[r], a[r], sa[:, r].contiguous(), *w[e], 128, blocks(K) * 2.0 ** -125 + 2.0 ** -134)

"""Many tiles in the persistent kernels of the gated block and of the int8 product: a CTA pair walks three and more tiles
(each TMEM buffer, barrier and store box is used again), in every order of the tiles; clusters of every size in the streaming
kernel; and stages that never arrive in the int8 kernel of 64 tokens."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_dense_ffn_watchdog import status, withhold  # noqa: F401 (a fixture)
from tests.test_gpu_gated_ffn import TYPES, check_backward, check_forward, make
from tests.test_gpu_int8 import codes, product, rand

pytestmark = pytest.mark.gpu

IDS = ["bf16", "fp16"]


@pytest.fixture
def raster():
    yield lambda g: m.nvfp4_tune(m.NVFP4_TUNE_DENSE_RASTER, g)
    m.nvfp4_tune(m.NVFP4_TUNE_DENSE_RASTER, 0)


# 99, 355, 219 and 350 tiles of 256 rows and 128 columns for 76 pairs; the last in bands of 13 and 12 rows of tiles
@pytest.mark.parametrize("M,I,K", [(700, 4104, 136), (1031, 9000, 72), (131, 28000, 64), (6300, 1704, 72)])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_forward(M, I, K, dtype):
    x, wg, wu, _ = make(M, I, K, dtype, seed=M)
    st = status()
    assert m.nvfp4_gated_ffn_workspace_bytes(M, I, K) == 0  # whole tiles
    act = "silu" if dtype == torch.bfloat16 else "gelu_tanh"
    plain = m.nvfp4_gated_ffn(x, wg, wu, act, dev_status=st)
    h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, act, save=True, dev_status=st)
    check_forward(x, wg, wu, act, h, gate, up)
    check_forward(x, wg, wu, act, plain)
    assert int(st) == 0


# dx: 350 tiles of 256 x 256 in bands of 13 and 12 rows; both weights' gradients: 700, in bands; one of them; 196 and 392 tiles in
# one launch; and 474 of dx beside the weights' in eight parts
@pytest.mark.parametrize("M,I,K,need", [(6300, 72, 3336, (True, False, False)), (70, 6296, 3336, (False, True, True)),
                                        (70, 6296, 3336, (False, False, True)), (3400, 3400, 3336, (True, True, True)),
                                        (20000, 136, 1288, (True, True, True))])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gradients(M, I, K, need, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + I)
    x, wg, wu, dh = make(M, I, K, dtype, seed=M)
    gate, up = (torch.randn(M, I, generator=g, device="cuda") for _ in range(2))
    st = status()
    got = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, "gelu_tanh", need=need, dev_status=st)
    assert int(st) == 0
    check_backward(x, wg, wu, gate, up, dh, "gelu_tanh", *got)


@pytest.mark.parametrize("M,I,K", [(6300, 1704, 72), (700, 4104, 136), (3400, 3400, 3336)])
def test_every_order_of_the_tiles(raster, M, I, K):
    x, wg, wu, dh = make(M, I, K, torch.bfloat16, seed=2)

    def results():
        h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
        return (h, gate, up) + m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh)
    want = results()
    for order in (-1, 3, 100):  # columns of tiles first, bands of three rows, rows first
        raster(order)
        assert all(torch.equal(a, b) for a, b in zip(results(), want)), order


# clusters of 3, 5, 6 and 7 CTAs along K: parts of unequal length, owners of different numbers of tokens or of none
@pytest.mark.parametrize("M,I,K", [(77, 5000, 1032), (1, 5000, 1032), (3, 3800, 1288), (128, 3800, 1288), (5, 3104, 1544), (61, 3200, 1600),
                                   (2, 2704, 1800), (36, 2704, 1800)])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_clusters_of_every_size(M, I, K, dtype):
    x, wg, wu, _ = make(M, I, K, dtype, seed=M + I)
    h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    check_forward(x, wg, wu, "silu", h, gate, up)
    assert torch.equal(m.nvfp4_gated_ffn(x, wg, wu), h)


# tiles of 64 and of 128 tokens: 239 in one row, 150 in three rows; of 256: 220 in two rows, 340 in bands
@pytest.mark.parametrize("M,N,K,wide", [(40, 61000, 1168, False), (100, 61003, 80, False), (300, 12700, 80, False), (300, 28001, 144, True),
                                        (5000, 4100, 272, True)])
def test_int8(raster, M, N, K, wide):
    assert (m.nvfp4_int8_gemm_workspace_bytes(M, N, K) > 0) == wide
    a, b, r = codes(M, M, K), codes(N, N, K), rand(K)
    sa, sb = r(M).abs() + 1e-3, r(N).abs() + 1e-4
    want = product(a, sa, b, sb)
    st = status()
    for order in (0, -1, 3):
        raster(order)
        for dtype in (torch.float32, torch.bfloat16):
            y = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=dtype, dev_status=st)
            assert torch.equal(y, want.to(dtype)), (order, dtype)
    assert int(st) == 0


@pytest.mark.parametrize("N,K", [(300, 2048), (9800, 512)])  # in four parts, and whole
@pytest.mark.parametrize("stage", [1, 3])
def test_int8_of_64_tokens_without_a_stage(withhold, N, K, stage):  # noqa: F811
    M = 40
    a, b = codes(1, M, K), codes(2, N, K)
    sa, sb = torch.full((M,), 0.5, device="cuda"), torch.full((N,), 0.25, device="cuda")
    st = status()
    withhold(stage)
    m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, dev_status=st)
    assert int(st) == -7
    withhold(0)
    st.zero_()
    y = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32, dev_status=st)
    assert int(st) == 0 and torch.equal(y, product(a, sa, b, sb))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantiser_by_its_stated_operations(dtype):
    """s = amax (1/127), code = rn(x (127 (1/amax))): every step one fp32 operation, written out (where torch divides by a
    number it may do something else)."""
    r = rand(8)
    x = (r(700, 272) * torch.exp(3 * r(700, 1))).to(dtype)
    q, s = m.nvfp4_int8_quantize(x)
    v = x.float().cpu().numpy()
    one, top = v.dtype.type(1), v.dtype.type(127)
    amax = abs(v).max(1)
    assert (s.cpu().numpy() == amax * (one / top)).all()
    inv = top * (one / amax)
    assert (q.cpu().numpy() == (v * inv[:, None]).round()).all()

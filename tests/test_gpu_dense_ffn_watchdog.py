"""A pipeline stage that never arrives, in each kernel of the gated block and of the int8 product: with a short limit every
wait ends by itself, the clusters' barriers pair, NVFP4_ERR_TIMEOUT is reported, and the next call is right."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_gated_ffn import check_backward, check_forward, make
from tests.test_gpu_int8 import codes, product

pytestmark = pytest.mark.gpu


@pytest.fixture
def withhold():
    def set_stage(stage):
        m.nvfp4_tune(m.NVFP4_TUNE_WATCHDOG_US, 20000 if stage else 0)
        m.nvfp4_tune(m.NVFP4_TUNE_TEST_WITHHOLD_STAGE, stage)

    yield set_stage
    set_stage(0)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# streamed, in one part and in parts of a cluster; tiles, whole and in parts
@pytest.mark.parametrize("M,I,K", [(3, 20000, 256), (3, 512, 2048), (100, 520, 1024), (300, 2816, 512), (256, 256, 4096)])
@pytest.mark.parametrize("stage", [1, 2])
def test_forward(withhold, M, I, K, stage):
    x, wg, wu, _ = make(M, I, K, torch.bfloat16, seed=M)
    st = status()
    withhold(stage)
    m.nvfp4_gated_ffn(x, wg, wu, dev_status=st)
    assert int(st) == -7
    withhold(0)
    st.zero_()
    h = m.nvfp4_gated_ffn(x, wg, wu, dev_status=st)
    assert int(st) == 0
    check_forward(x, wg, wu, "silu", h)


@pytest.mark.parametrize("M,I,K", [(300, 2816, 1024), (2000, 64, 64), (40, 520, 256)])
@pytest.mark.parametrize("stage", [1, 2])
def test_gradients(withhold, M, I, K, stage):
    x, wg, wu, dh = make(M, I, K, torch.float16, seed=M)
    _, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    st = status()
    withhold(stage)
    m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, dev_status=st)
    assert int(st) == -7
    withhold(0)
    st.zero_()
    got = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, dev_status=st)
    assert int(st) == 0
    check_backward(x, wg, wu, gate, up, dh, "silu", *got)


# each size of token tiles, in four parts and whole
@pytest.mark.parametrize("M,N,K", [(3, 300, 2048), (3, 9800, 512), (100, 300, 2048), (100, 9800, 512), (300, 300, 4096), (300, 5003, 512),
                                   (512, 2579, 8192), (1100, 5003, 512)])
@pytest.mark.parametrize("stage", [1, 3])
def test_int8(withhold, M, N, K, stage):
    a, b = codes(1, M, K), codes(2, N, K)
    sa, sb = torch.full((M,), 0.5, device="cuda"), torch.full((N,), 0.25, device="cuda")
    st = status()
    withhold(stage)
    m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, dev_status=st)
    assert int(st) == -7
    withhold(0)
    st.zero_()
    y = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32, dev_status=st)
    assert int(st) == 0
    assert torch.equal(y, product(a, sa, b, sb))

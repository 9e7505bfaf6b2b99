"""The FP8 tile kernel with K in two and four parts: sizes that take it by themselves, every form forced, and a
stage that never arrives. Tolerances as in test_gpu_fp8.py."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev
from tests.test_gpu_fp8 import acts, blocks, check, decode

pytestmark = pytest.mark.gpu


@pytest.fixture
def tune():
    keys = set()

    def set_key(key, value):
        keys.add(key)
        m.nvfp4_tune(key, value)

    yield set_key
    for key in keys:
        m.nvfp4_tune(key, 0)


def product(M, N, K, b_rows, out):
    a, sa = m.nvfp4_fp8_quantize(acts(M, K, M + K))
    b, sb = m.nvfp4_fp8_quantize(acts(N, K, N + K + 1, 0.02), b_rows)
    A, B = decode(a, sa, 1), decode(b, sb, b_rows)

    def run():
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        guard = torch.full((M * N + 64,), 7.0, dtype=out, device=dev())
        y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows, out_dtype=out, y=guard[:M * N].view(M, N),
                             dev_status=st)
        assert (guard[M * N:] == 7.0).all()  # nothing past the output
        return y, int(st)

    return run, lambda y: check(y, A, B)


# 9 to 38 tiles of 256 x 256 and at least 24 blocks of K: two parts; up to 8 tiles: four
TWO = [(256, 4096, 3088), (300, 1801, 4112), (513, 1030, 3088), (129, 2308, 3072), (300, 4864, 3200)]
FOUR = [(130, 260, 3088), (300, 777, 4096), (257, 1026, 3216)]


@pytest.mark.parametrize("M,N,K", TWO + FOUR)
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_sizes_that_split(M, N, K, b_rows, out):
    run, right = product(M, N, K, b_rows, out)
    y, status = run()
    assert status == 0
    right(y)
    assert torch.equal(y, run()[0])  # the parts are added in one order


@pytest.mark.parametrize("split", [1, 2, 4])
@pytest.mark.parametrize("M,N,K", [(65, 300, 656), (300, 131, 1040), (257, 770, 528)])
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_forced_parts(tune, split, M, N, K, b_rows, out):
    tune(m.NVFP4_TUNE_STREAM_SPLIT, split)
    run, right = product(M, N, K, b_rows, out)
    y, status = run()
    assert status == 0
    right(y)


@pytest.mark.parametrize("split", [1, 2, 4])
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("stage", [1, 2])
def test_withheld_stage_is_reported(tune, split, b_rows, out, stage):
    """Every wait ends by itself, the cluster's barriers pair, and the next call is right."""
    run, right = product(300, 520, 1040, b_rows, out)
    tune(m.NVFP4_TUNE_STREAM_SPLIT, split)
    tune(m.NVFP4_TUNE_WATCHDOG_US, 20000)
    tune(m.NVFP4_TUNE_TEST_WITHHOLD_STAGE, stage)
    assert run()[1] == -7
    tune(m.NVFP4_TUNE_TEST_WITHHOLD_STAGE, 0)
    y, status = run()
    assert status == 0
    right(y)

"""Operands of the FP8 products are checked against the sizes of the call, not by their element count alone, and
no call takes a status or an output in host memory."""
import inspect

import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev, dense_case

on_gpu = pytest.mark.gpu

M, N, K, E = 8, 272, 512, 3


def dense():
    g = torch.Generator(device=dev()).manual_seed(0)
    a, sa = m.nvfp4_fp8_quantize(torch.randn(M, K, generator=g, device=dev()).bfloat16())
    b, sb = m.nvfp4_fp8_quantize(torch.randn(N, K, generator=g, device=dev()).bfloat16(), 128)
    return a, sa, b, sb


def grouped():
    a, sa, b, sb = dense()
    off = torch.tensor([0, 3, 3, M], dtype=torch.int32, device=dev())
    return a, sa, torch.stack([b] * E), torch.stack([sb] * E), off


# operand, and a tensor of as many elements whose sizes are not the call's
DENSE_WRONG = [(0, lambda t: t.view(2 * M, K // 2)), (1, lambda t: t.t().contiguous()), (2, lambda t: t.view(N * 2, K // 2)),
               (3, lambda t: t.t().contiguous())]


@on_gpu
@pytest.mark.parametrize("i,change", DENSE_WRONG)
def test_fp8_gemm_refuses_other_sizes(i, change):
    args = list(dense())
    args[i] = change(args[i])
    with pytest.raises(TypeError):
        m.nvfp4_fp8_gemm(*args, M, N, K)


@on_gpu
@pytest.mark.parametrize("i,change", DENSE_WRONG[:2] + [(2, lambda t: t.view(E, N * 2, K // 2)), (2, lambda t: t.view(N, E, K)),
                                                        (3, lambda t: t.transpose(1, 2).contiguous()),
                                                        (4, lambda t: t[:E].clone())])
def test_fp8_grouped_gemm_refuses_other_sizes(i, change):
    args = list(grouped())
    args[i] = change(args[i])
    with pytest.raises(TypeError):
        m.nvfp4_fp8_grouped_gemm(*args, E, M, N, K)


@on_gpu
def test_fp8_products_take_flat_buffers_and_more_rows():
    a, sa, b, sb = dense()
    want = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K)
    assert torch.equal(want, m.nvfp4_fp8_gemm(a.flatten(), sa.flatten(), b.flatten(), sb.flatten(), M, N, K))
    assert torch.equal(want, m.nvfp4_fp8_gemm(a.view(2, M // 2, K), sa, torch.cat([b, b]), torch.cat([sb, sb]), M, N, K))
    ga, gsa, gb, gsb, off = grouped()
    want = m.nvfp4_fp8_grouped_gemm(ga, gsa, gb, gsb, off, E, M, N, K)
    assert torch.equal(want, m.nvfp4_fp8_grouped_gemm(ga, gsa, gb.view(E * N, K), gsb.view(-1, K // 128), off, E, M, N, K))


@on_gpu
def test_fp8_products_take_split_and_merged_dimensions():
    a, sa, b, sb = dense()
    want = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K)
    y = torch.empty(2, M // 2, 2, N // 2, dtype=torch.bfloat16, device=dev())  # [batch, tokens, heads, size]
    m.nvfp4_fp8_gemm(a.view(2, M // 2, 4, K // 4), sa.view(K // 128, 2, M // 2), b.view(N, 4, K // 4), sb, M, N, K, y=y)
    assert torch.equal(want, y.view(M, N))


@pytest.mark.parametrize("have,shape,fits", [((8, 512), (8, 512), True), ((9, 512), (8, 512), True), ((4096,), (8, 512), True),
                                             ((2, 4, 512), (8, 512), True), ((8, 4, 128), (8, 512), True), ((7, 512), (8, 512), False),
                                             ((16, 256), (8, 512), False), ((8, 1024), (8, 512), False), ((512, 8), (8, 512), False),
                                             ((6, 512), (2, 3, 512), True), ((3, 2, 512), (2, 3, 512), False),
                                             ((2, 3, 4, 128), (2, 3, 512), True), ((1, 4), (4, 1), True),
                                             ((4, 128), (1, 512), True), ((1, 1024), (1, 512), False), ((0, 512), (0, 512), True), ((5,), (0, 512), True)])
def test_fits(have, shape, fits):
    assert m._fits(torch.Size(have), shape) == fits


@on_gpu
def test_sizes_that_the_library_refuses_stay_its_error():
    a, sa, b, sb = dense()
    for sizes, status in (((M, N, K + 8), -2), ((M, 0, K), -1), ((M, N, -16), -1)):
        with pytest.raises(m.NVFP4Error) as e:
            m.nvfp4_fp8_gemm(a, sa, b, sb, *sizes)
        assert e.value.status == status
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_fp8_grouped_gemm(*grouped(), 0, M, N, K)
    assert e.value.status == -1


@on_gpu
@pytest.mark.parametrize("bad", [lambda: torch.zeros(1, dtype=torch.int32), lambda: torch.zeros(1, dtype=torch.int64, device=dev()),
                                 lambda: torch.zeros(0, dtype=torch.int32, device=dev())])
def test_status_is_checked(bad):
    with pytest.raises(TypeError):
        m.nvfp4_fp8_gemm(*dense(), M, N, K, dev_status=bad())
    with pytest.raises(TypeError):
        m.nvfp4_fp8_grouped_gemm(*grouped(), E, M, N, K, dev_status=bad())
    A, B = dense_case(16, 128, 256, 3)
    with pytest.raises(TypeError):
        m.nvfp4_gemm(A.dq, A.dsf, A.dg, B.dq, B.dsf, B.dg, 16, 128, 256, dev_status=bad())


@on_gpu
def test_host_memory_is_refused():
    A, B = dense_case(16, 128, 256, 3)
    with pytest.raises(TypeError):
        m.nvfp4_gemm(A.dq, A.dsf, A.dg, B.dq, B.dsf, B.dg, 16, 128, 256, y=torch.empty(16, 128, dtype=torch.bfloat16))
    x = torch.zeros(16, 256, dtype=torch.bfloat16, device=dev())
    with pytest.raises(TypeError):
        m.nvfp4_amax(x, workspace=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(TypeError):
        m.nvfp4_quantize(x, A.dg, q_out=torch.empty(16, 128, dtype=torch.uint8))


def test_every_call_with_a_status_checks_it():
    for n in m.EXPORTS:
        if hasattr(m, n) and "dev_status" in inspect.signature(getattr(m, n)).parameters:
            assert "_status(dev_status)" in inspect.getsource(getattr(m, n))

"""Results of the dense feed-forward calls beside their operands in one buffer: what shares no element is taken and right,
what does is refused."""
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.test_gpu_gated_ffn import check_backward, check_forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 5, 300])
def test_columns_of_one_buffer(M):
    """x and h side by side in each row, and h in rows four times as far apart as it needs behind every second row of x."""
    I, K = 136, 200
    x, wg, wu, _ = make(M, I, K, torch.bfloat16, seed=M)
    buf = torch.full((M, K + I), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :K] = x
    m.nvfp4_gated_ffn(buf[:, :K], wg, wu, h=buf[:, K:])
    assert torch.equal(buf[:, :K], x)
    check_forward(x, wg, wu, "silu", buf[:, K:])
    pitch = K + I + 8
    flat = torch.full((2 * M * pitch,), 7.0, dtype=torch.bfloat16, device="cuda")
    near, far = flat[:M * pitch].view(M, pitch), flat.view(M, 2 * pitch)
    near[:, :K] = x
    m.nvfp4_gated_ffn(near[:, :K], wg, wu, h=far[:, K:K + I])
    assert torch.equal(near[:, :K], x)
    check_forward(x, wg, wu, "silu", far[:, K:K + I])


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


@pytest.mark.parametrize("M", [5, 200])
def test_refused(M):
    x, wg, wu, _ = make(M, 256, 256, torch.bfloat16)
    a, sa = m.nvfp4_int8_quantize(x)
    b, sb = m.nvfp4_int8_quantize(wg)
    over = sb.view(torch.bfloat16)[:2 * M].view(M, 2)  # two channels' results over the channels' scales
    g = torch.ones(100, device="cuda")
    kept = [t.clone() for t in (x, wg, sb, g)]
    for call in (lambda: m.nvfp4_gated_ffn(x, wg, wu, h=x), lambda: m.nvfp4_gated_ffn(x, wg, wu, h=wg[:M]),
                 lambda: m.nvfp4_int8_gemm(a, sa, b[:2], sb[:2], M, 2, 256, y=over),
                 lambda: m.nvfp4_grad_clip([g], 1.0, norm=g[3:4]), lambda: m.nvfp4_grad_clip([g], norm=g[3:4])):
        with pytest.raises(m.NVFP4Error) as e:
            call()
        assert e.value.status == -1
    assert all(torch.equal(t, k) for t, k in zip((x, wg, sb, g), kept))


def test_norm_behind_the_gradients():
    """A norm that is the next value of the gradients' buffer shares nothing with them."""
    flat = torch.full((101,), 2.0, device="cuda")
    norm = m.nvfp4_grad_clip([flat[:100]], 10.0, norm=flat[100:])
    assert norm.data_ptr() == flat[100:].data_ptr() and float(norm) == 20.0
    assert ((flat[:100] - 1).abs() < 1e-6).all()

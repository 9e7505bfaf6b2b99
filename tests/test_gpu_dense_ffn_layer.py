"""The dense feed-forward layer of examples/dense_ffn_layer.py: the gated block, its gradients, clipping, the int8 quantiser
and the int8 product together, as a training step and as serving."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import dense_ffn_layer
    return dense_ffn_layer


def act64(g, act):
    return torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")


@pytest.mark.parametrize("T,H,I,act,dtype", [(1, 64, 136, "silu", torch.bfloat16), (77, 256, 520, "gelu_tanh", torch.float16),
                                             (300, 512, 1032, "silu", torch.bfloat16)])
def test_gradients_against_autograd(ex, T, H, I, act, dtype):
    """All gradients against autograd in 64 bits. Every tensor on the way is rounded to the type at most once per
    product (h, dh, dg, du, the result), each off by half a step of its value, so norms differ by at most 5 half steps
    and the sums' 1e-4."""
    g = torch.Generator(device="cuda").manual_seed(T)
    layer = ex.DenseLayer(H, I, g, dtype, act)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    dy = (torch.randn(T, H, generator=g, device="cuda") * 0.1).to(dtype)
    y, saved = layer.forward(x, save=True)
    dx, grads = layer.gradients(x, saved, dy)
    leaves = [t.double().requires_grad_() for t in (x, *layer.weights)]
    X, G, U, D = leaves
    want = (act64(X @ G.t(), act) * (X @ U.t())) @ D.t()
    want.backward(dy.double())
    want = want.detach()
    tol = 5 * torch.finfo(dtype).eps / 2 + 1e-4
    for name, got, ref in [("y", y, want)] + [(n, a, l.grad) for n, a, l in zip(("dx", "gate", "up", "down"), [dx] + grads, leaves)]:
        assert float((got.double() - ref).norm() / ref.norm()) <= tol, name


def test_training_step_clips_and_updates(ex):
    """A step subtracts the clipped gradients: their norm, as it was before, scaled to the limit; the master weights move
    by at most lr times the limit (and the rounding of each gradient)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = ex.DenseLayer(256, 520, g)
    x = torch.randn(130, 256, generator=g, device="cuda").bfloat16()
    target = torch.randn(130, 256, generator=g, device="cuda").bfloat16()
    y, saved = layer.forward(x, save=True)
    diff = y.float() - target.float()
    _, grads = layer.gradients(x, saved, (diff / diff.numel() ** 0.5).bfloat16())
    total = sum(float((t.double() ** 2).sum()) for t in grads) ** 0.5
    before = [w.clone() for w in layer.master]
    limit = total / 3
    loss, norm = ex.train_step(layer, x, target, lr=0.5, max_norm=limit)
    assert abs(float(norm) - total) <= 1e-5 * total and torch.isfinite(loss)
    moved = [b - w for b, w in zip(before, layer.master)]
    assert abs(sum(float((t.double() ** 2).sum()) for t in moved) ** 0.5 - 0.5 * limit) <= 2.0 ** -8 * limit
    for t, gr in zip(moved, grads):  # the direction of the gradients
        assert float((t / 0.5 - gr.float() / 3).norm() / (gr.float() / 3).norm()) <= 2.0 ** -7
    assert all(torch.equal(w, v.bfloat16()) for w, v in zip(layer.weights, layer.master))


@pytest.mark.parametrize("T", [1, 40, 200])
def test_served_in_int8(ex, T):
    """Against the same arithmetic in 64 bits: the quantised operands are shared, so that only the roundings between the
    calls differ. h is rounded to 16 bits before it is quantised; a code may then lie a step (scale, amax / 127) off."""
    import moe_nvfp4_gemm_gb300 as m
    g = torch.Generator(device="cuda").manual_seed(2)
    layer = ex.DenseLayer(512, 1040, g)
    served = ex.Int8Layer(layer)
    x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
    got = served.forward(x)
    values = lambda qs: qs[0].double() * qs[1].double()[:, None]
    X = values(m.nvfp4_int8_quantize(x))
    G, U, D = (values(w) for w in served.weights)
    h = torch.nn.functional.silu(X @ G.t()) * (X @ U.t())
    want = h @ D.t()
    amax = h.abs().amax(1, keepdim=True)
    tol = (0.51 * amax / 127 + 2.0 ** -8 * h.abs()) @ D.abs().t() + 2.0 ** -8 * 1.01 * want.abs() + 1e-4 * (h.abs() @ D.abs().t())
    assert ((got.double() - want).abs() <= tol).all()


def test_int8_widths_are_multiples_of_16(ex):
    import moe_nvfp4_gemm_gb300 as m
    with pytest.raises(m.NVFP4Error) as e:  # the 16-bit layer takes multiples of 8
        ex.Int8Layer(ex.DenseLayer(512, 1032, torch.Generator(device="cuda").manual_seed(3)))
    assert e.value.status == -2


def test_example_runs(ex, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["dense_ffn_layer.py", "--tokens", "70", "--hidden", "128", "--inner", "272", "--steps", "2", "--repeat", "0"])
    ex.main()
    out = capsys.readouterr().out
    assert "int8" in out and "nan" not in out

"""A dense gated feed-forward layer: trained in 16 bits, its gradients clipped, then served in 8-bit integers.

    python examples/dense_ffn_layer.py [--tokens T] [--hidden H] [--inner I] [--steps N]

train_step():  gated block -> down projection -> gradients of all three weights and of the input -> clipped to a
               largest norm -> subtracted from fp32 master weights
Int8Layer:     the same layer with int8 weights (a scale for each output channel) and activations (for each token)
main() trains the layer to follow another one for a few steps, then serves a prompt and single tokens, and prints
the losses, the differences between the two forms and times.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_nvfp4_gemm_gb300 as m  # noqa: E402


class DenseLayer:
    """w_gate, w_up [I, H] and w_down [H, I] in 16 bits, with fp32 master copies."""

    def __init__(self, H, I, generator, dtype=torch.bfloat16, activation="silu"):
        def normal(*shape):
            return torch.randn(*shape, generator=generator, device="cuda") * shape[1] ** -0.5

        self.activation = activation
        self.master = [normal(I, H), normal(I, H), normal(H, I)]
        self.weights = [w.to(dtype) for w in self.master]

    def forward(self, x, save=False):
        w_gate, w_up, w_down = self.weights
        out = m.nvfp4_gated_ffn(x, w_gate, w_up, self.activation, save=save)
        h = out[0] if save else out
        return (h @ w_down.t(), out) if save else h @ w_down.t()

    def gradients(self, x, saved, dy):
        """(dx, [dw_gate, dw_up, dw_down]) from the gradient dy of the layer's result."""
        h, gate, up = saved
        w_gate, w_up, w_down = self.weights
        dx, dw_gate, dw_up = m.nvfp4_gated_ffn_backward(x, w_gate, w_up, gate, up, dy @ w_down, self.activation)
        return dx, [dw_gate, dw_up, dy.t() @ h]

    def update(self, grads, lr):
        for master, weight, g in zip(self.master, self.weights, grads):
            master.sub_(g.float(), alpha=lr)
            weight.copy_(master)


def train_step(layer, x, target, lr=1.0, max_norm=0.5):
    """One step on 0.5 mean((y - target)^2): (loss, gradient norm), both on the device."""
    y, saved = layer.forward(x, save=True)
    diff = y.float() - target.float()
    dy = (diff / diff.numel() ** 0.5).to(x.dtype)
    _, grads = layer.gradients(x, saved, dy)
    norm = m.nvfp4_grad_clip(grads, max_norm)
    layer.update(grads, lr)
    return 0.5 * diff.square().mean(), norm


class Int8Layer:
    """A DenseLayer's weights as int8 codes with a scale for each output channel."""

    def __init__(self, layer):
        self.activation = layer.activation
        self.weights = [m.nvfp4_int8_quantize(w) for w in layer.weights]

    def linear(self, x, at):
        q, s = m.nvfp4_int8_quantize(x)
        w, sw = self.weights[at]
        return m.nvfp4_int8_gemm(q, s, w, sw, x.shape[0], w.shape[0], w.shape[1], out_dtype=x.dtype)

    def forward(self, x):
        q, s = m.nvfp4_int8_quantize(x)  # once for both projections
        gate, up = (m.nvfp4_int8_gemm(q, s, w, sw, x.shape[0], w.shape[0], w.shape[1], out_dtype=torch.float32)
                    for w, sw in self.weights[:2])
        act = torch.nn.functional.silu(gate) if self.activation == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
        return self.linear((act * up).to(x.dtype), 2)


def reference(layer, x):
    """The layer in fp32 torch operations on its 16-bit weights."""
    w_gate, w_up, w_down = (w.float() for w in layer.weights)
    g, u = x.float() @ w_gate.t(), x.float() @ w_up.t()
    a = torch.nn.functional.silu(g) if layer.activation == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    return (a * u) @ w_down.t()


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm().clamp(min=1e-30))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2816)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--repeat", type=int, default=20, help="timed passes (0: none)")
    args = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    layer, teacher = (DenseLayer(args.hidden, args.inner, g) for _ in range(2))
    x = torch.randn(args.tokens, args.hidden, generator=g, device="cuda").bfloat16()
    target = teacher.forward(x)
    history = [train_step(layer, x, target) for _ in range(args.steps)]
    print("loss, gradient norm: " + "  ".join(f"{float(l):.4f} {float(n):.3f}" for l, n in history))
    served = Int8Layer(layer)
    for rows in (1, 64, args.tokens):
        y = served.forward(x[:rows].contiguous())
        print(f"{rows} tokens: 16 bits {relative(layer.forward(x[:rows]), reference(layer, x[:rows])):.4f}, "
              f"int8 {relative(y, reference(layer, x[:rows])):.4f} from fp32")
    if args.repeat:
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for name, f in (("training step", lambda: train_step(layer, x, target)), ("16-bit layer", lambda: layer.forward(x)),
                        ("int8 layer", lambda: served.forward(x)), ("16-bit layer, one token", lambda: layer.forward(x[:1])),
                        ("int8 layer, one token", lambda: served.forward(x[:1]))):
            for _ in range(3):
                f()
            torch.cuda.synchronize()
            a.record()
            for _ in range(args.repeat):
                f()
            b.record()
            torch.cuda.synchronize()
            print(f"{name}: {a.elapsed_time(b) / args.repeat * 1e3:.1f} us")


if __name__ == "__main__":
    main()

"""An MoE layer with FP8 experts, and one training step of its router and of an FP8 linear layer.

    python examples/moe_fp8_layer.py [--tokens T] [--experts E] [--topk K] [--hidden H] [--inner I]

forward():       router -> routed rows gathered and quantised -> grouped gate/up product -> SwiGLU
                 -> quantised -> grouped down product -> weighted sum of each token's experts
router_step():   gradient of the router's logits from the layer's gradient and the balance loss
linear_step():   y = x W^T in FP8 with both gradients
The same routing drives NVFP4 experts: forward_nvfp4_gate_up(). main() runs everything once, checks it
against torch in fp32 on the same quantised weights, and prints times.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_nvfp4_gemm_gb300 as m  # noqa: E402


class Fp8Experts:
    """E experts: gate/up weight [2 I, H] (gate rows, then up rows) and down weight [H, I], in E4M3 with
    a scale for each 128 x 128 block."""

    def __init__(self, E, H, I, generator):
        self.E, self.H, self.I = E, H, I

        def quantised(N, K):
            q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
            s = torch.empty(E, (N + 127) // 128, (K + 127) // 128, device="cuda")
            for e in range(E):
                w = torch.randn(N, K, generator=generator, device="cuda") * K ** -0.5
                q[e], s[e] = m.nvfp4_fp8_quantize(w.bfloat16(), 128)
            return q, s

        self.gate_up, self.gate_up_s = quantised(2 * I, H)
        self.down, self.down_s = quantised(H, I)


def forward(x, logits, experts, k, valid=None):
    """x bf16 [T, H], logits [T, E] -> (y bf16 [T, H], routing, expert outputs bf16 [T k, H])."""
    E, H, I = experts.E, experts.H, experts.I
    T = x.shape[0]
    r = m.nvfp4_moe_route(logits, k, renormalize=True, valid=valid)
    rows = T * k
    a, sa = m.nvfp4_fp8_quantize(x, row_token=r.row_token)
    gu = m.nvfp4_fp8_grouped_gemm(a, sa, experts.gate_up, experts.gate_up_s, r.expert_offsets, E, rows, 2 * I, H)
    gate, up = gu.float().split(I, 1)
    act = (torch.nn.functional.silu(gate) * up).bfloat16()
    # rows past the last routed one hold nothing: the row list quantises them as zeros
    kept = torch.where(r.row_token >= 0, torch.arange(rows, device="cuda", dtype=torch.int32), -1)
    h, sh = m.nvfp4_fp8_quantize(act, row_token=kept)
    out = m.nvfp4_fp8_grouped_gemm(h, sh, experts.down, experts.down_s, r.expert_offsets, E, rows, H, I)
    return combine(out, r), r, out


def combine(out, r):
    """Each token's experts' rows, weighted; empty slots (row -1) have weight 0 and read no row."""
    picked = torch.where((r.slot_row >= 0)[..., None], out[r.slot_row.clamp(min=0).long()].float(), 0.0)
    return (picked * r.topk_w[..., None]).sum(1).bfloat16()


def forward_nvfp4_gate_up(x, logits, w_gu, k):
    """The same routing in front of NVFP4 experts (all slots filled): w_gu = (codes, scales, global scales)."""
    r = m.nvfp4_moe_route(logits, k, renormalize=True)
    q, sf = m.nvfp4_quantize(x, g := m.nvfp4_amax(x)[1])
    b, sfb, gb = w_gu
    return m.nvfp4_grouped_gemm_gather(q, sf, g, b, sfb, gb, r.expert_offsets, r.row_token, b.shape[0], x.shape[0],
                                       x.shape[0] * k, b.shape[1], x.shape[1]), r


def router_step(logits, r, out, dy, coef, valid=None):
    """d logits of sum(dy * y) + coef * balance loss, y the weighted sum of the expert outputs. (The routing knows
    what it was made with; `valid`, where given, has to be that of the forward call.)"""
    picked = torch.where((r.slot_row >= 0)[..., None], out[r.slot_row.clamp(min=0).long()].float(), 0.0)
    d_w = torch.einsum("th,tkh->tk", dy.float(), picked).contiguous()
    return m.nvfp4_moe_route_backward(logits, r, d_w=d_w, d_loss=torch.full((1,), coef, device="cuda"), valid=valid)


def linear_step(x, w, dy):
    """y = x W^T, dx = dy W, dW = dy^T x (fp32): three products of two quantisations of each tensor."""
    T, K = x.shape
    N = w.shape[0]
    Tp = (T + 15) // 16 * 16
    xq, xs, xt, xts = m.nvfp4_fp8_quantize(x, transposed=True)
    wq, ws, wt, wts = m.nvfp4_fp8_quantize(w, 128, transposed=True)
    dq, ds, dt, dts = m.nvfp4_fp8_quantize(dy, transposed=True)
    y = m.nvfp4_fp8_gemm(xq, xs, wq, ws, T, N, K)
    dx = m.nvfp4_fp8_gemm(dq, ds, wt, wts, T, K, N)
    dw = m.nvfp4_fp8_gemm(dt, dts, xt, xts, N, K, Tp, b_block_rows=1, out_dtype=torch.float32)
    return y, dx, dw


def reference(x, logits, experts, k, valid=None):
    """forward() in fp32 with the quantised weights; the activations are not quantised."""
    def decoded(q, s):
        return q.float() * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]

    l = logits.float()
    if valid is not None:
        l = torch.where(valid[:, None], l, -torch.inf)
    p = torch.softmax(l, 1).nan_to_num(0.0)
    w, idx = p.topk(k, 1)
    w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    y = torch.zeros(x.shape, device="cuda")
    for e in range(experts.E):
        t, s = (idx == e).nonzero(as_tuple=True)
        gate, up = (x[t].float() @ decoded(experts.gate_up[e], experts.gate_up_s[e]).t()).split(experts.I, 1)
        o = (torch.nn.functional.silu(gate) * up) @ decoded(experts.down[e], experts.down_s[e]).t()
        y.index_add_(0, t, o * w[t, s, None])
    return y


def relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm().clamp(min=1e-30))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--repeat", type=int, default=20, help="timed passes (0: none)")
    args = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    T, E, k, H, I = args.tokens, args.experts, args.topk, args.hidden, args.inner
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    valid = torch.rand(T, generator=g, device="cuda") < 0.9  # a tenth of the tokens are padding
    dy = (torch.randn(T, H, generator=g, device="cuda") * 1e-2).bfloat16()
    experts = Fp8Experts(E, H, I, g)

    y, r, out = forward(x, logits, experts, k, valid)
    print(f"layer: {T} tokens, {E} experts, top-{k}: relative difference {relative(y, reference(x, logits, experts, k, valid)):.4f},"
          f" balance loss {float(r.balance_loss):.4f}, rows per expert {int(r.counts.min())}..{int(r.counts.max())}")
    d = router_step(logits, r, out, dy, 0.01, valid)
    print(f"router gradient: norm {float(d.norm()):.3e}, padding rows zero: {bool((d[~valid] == 0).all())}")
    w = (torch.randn(I, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    dyl = (torch.randn(T, I, generator=g, device="cuda") * 1e-2).bfloat16()
    yl, dx, dw = linear_step(x, w, dyl)
    print(f"linear: y {relative(yl, x.float() @ w.float().t()):.4f}, dx {relative(dx, dyl.float() @ w.float()):.4f}, "
          f"dW {relative(dw, dyl.float().t() @ x.float()):.4f} (relative differences from the products of the bf16 values)")
    if args.repeat:
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for name, f in (("layer forward", lambda: forward(x, logits, experts, k, valid)),
                        ("router gradient", lambda: router_step(logits, r, out, dy, 0.01, valid)),
                        ("linear step", lambda: linear_step(x, w, dyl))):
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

"""The gated feed-forward block and its gradients on the GPU against 64-bit restatements of the formulas.

Tolerances: the tensor cores add 16 products a step to an fp32 sum, each step off by at most 2^-23 of the largest
magnitude in it, so a sum over n is off by at most (n / 16 + 4) 2^-23 sum |a b|; the activation's fast
exponential and division by less than 4e-6 of the value (|p| <= 30); a rounding to the type by half a step,
finfo.eps / 2 of the value (and half the smallest subnormal number, 2^-25, in fp16)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
FAST = 4e-6


@pytest.fixture(scope="module")
def m():
    import moe_nvfp4_gemm_gb300
    return moe_nvfp4_gemm_gb300


def act64(g, act):
    """act(g) and its derivative in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = (2 / torch.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def half_step(t):
    return torch.finfo(t).eps / 2


def sums(n):
    return (n / 16 + 4) * 2.0 ** -23


def make(M, I, K, dtype, seed=0, dh_scale=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return (r(M, K).to(dtype), (r(I, K) * K ** -0.5).to(dtype), (r(I, K) * K ** -0.5).to(dtype), (r(M, I) * dh_scale).to(dtype))


def close(got, want, tol, name):
    bad = ((got.double() - want).abs() > tol + 2.0 ** -25) | ~torch.isfinite(got)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}, worst " \
                          f"{float(((got.double() - want).abs() / (tol + 2.0 ** -25)).max()):.3g} of the tolerance"


def check_forward(x, wg, wu, act, h, gate=None, up=None):
    X, G, U = x.double(), wg.double(), wu.double()
    g, u = X @ G.t(), X @ U.t()
    dg, du = (sums(x.shape[1]) * (X.abs() @ W.abs().t()) for W in (G, U))
    a, _ = act64(g, act)
    e = half_step(h.dtype)
    want = a * u
    # |act'| <= 1.13
    close(h, want, e * want.abs() * 1.01 + 1.13 * dg * (u.abs() + du) + a.abs() * du + FAST * want.abs(), "h")
    if gate is not None:
        close(gate, g, dg, "gate")
        close(up, u, du, "up")


def check_backward(x, wg, wu, gate, up, dh, act, dx, dwg, dwu):
    X, G, U, D = x.double(), wg.double(), wu.double(), dh.double()
    a, s = act64(gate.double(), act)
    dg, du = D * up.double() * s, D * a
    e = half_step(x.dtype)
    # the derivative is a sum of terms up to 1.13 |g| + 1 in size; each is off by FAST of that
    eg = e * dg.abs() * 1.01 + FAST * (D * up.double()).abs() * (1.2 + gate.double().abs()) + 2.0 ** -25
    eu = e * du.abs() * 1.01 + FAST * du.abs() + 2.0 ** -25
    M, I = gate.shape
    if dx is not None:
        want = dg @ G + du @ U
        close(dx, want, 1.01 * e * want.abs() + eg @ G.abs() + eu @ U.abs()
              + sums(2 * I) * 1.01 * (dg.abs() @ G.abs() + du.abs() @ U.abs()), "dx")
    for dw, d, ed, n in ((dwg, dg, eg, "dw_gate"), (dwu, du, eu, "dw_up")):
        if dw is not None:
            want = d.t() @ X
            close(dw, want, 1.01 * e * want.abs() + ed.t() @ X.abs() + sums(M) * 1.01 * (d.abs().t() @ X.abs()), n)


# rows: one token, tile edges and ragged ends; widths: the smallest, odd multiples of 8, past a tile; contraction
# lengths that end inside a block of 64 and that are cut into parts (few tiles, long)
SIZES = [(1, 8, 8), (1, 264, 520), (2, 128, 64), (5, 136, 72), (31, 72, 200), (33, 1000, 136), (64, 512, 1024), (65, 512, 1032),
         (127, 1296, 64), (129, 128, 1536), (255, 264, 248), (257, 392, 328), (300, 2816, 1024), (513, 520, 2056), (1031, 72, 80)]


@pytest.mark.parametrize("M,I,K", SIZES)
@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16"])
def test_forward_and_gradients(m, M, I, K, dtype):
    act = "silu" if (M + I // 8) % 2 else "gelu_tanh"
    x, wg, wu, dh = make(M, I, K, dtype, seed=M + I + K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = m.nvfp4_gated_ffn(x, wg, wu, act, dev_status=status)
    h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, act, save=True, dev_status=status)
    check_forward(x, wg, wu, act, h, gate, up)
    check_forward(x, wg, wu, act, plain)
    got = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, act, dev_status=status)
    check_backward(x, wg, wu, gate, up, dh, act, *got)
    again = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the order of the sums is fixed
    assert int(status) == 0


@pytest.mark.parametrize("M,I,K", [(8, 4096, 256), (40, 256, 4096), (2000, 64, 64)])
def test_products_of_few_tiles(m, M, I, K):
    """Contractions in parts: long ones with few tiles, in each of the three products."""
    x, wg, wu, dh = make(M, I, K, torch.bfloat16, seed=7)
    h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, "silu", save=True)
    check_forward(x, wg, wu, "silu", h, gate, up)
    check_backward(x, wg, wu, gate, up, dh, "silu", *m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, "silu"))


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
def test_wanted_gradients_alone(m, need):
    x, wg, wu, dh = make(70, 200, 136, torch.bfloat16, seed=3)
    _, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    every = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh)
    some = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, need=need)
    for a, b, n in zip(every, some, need):
        assert (b is None) == (not n)
        if n:
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_views_with_strides(m, M):
    """x a slice of wider rows, the weights the halves of one tensor with padding columns, h a slice; what lies
    beside the slice of h stays."""
    I, K = 136, 200
    g = torch.Generator(device="cuda").manual_seed(M)
    wide = torch.randn(M, K + 64, generator=g, device="cuda").bfloat16()
    both = (torch.randn(2 * I, K + 8, generator=g, device="cuda") * K ** -0.5).bfloat16()
    x, wg, wu = wide[:, 16:16 + K], both[:I, :K], both[I:, :K]
    out = torch.full((M, I + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    h = m.nvfp4_gated_ffn(x, wg, wu, h=out[:, 8:8 + I])
    assert torch.equal(h, m.nvfp4_gated_ffn(x.contiguous(), wg.contiguous(), wu.contiguous()))
    assert (out[:, :8] == 7).all() and (out[:, 8 + I:] == 7).all()
    check_forward(x, wg, wu, "silu", h)
    _, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    dwide = (torch.randn(M, I + 8, generator=g, device="cuda") * 0.05).bfloat16()
    got = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dwide[:, 8:])
    check_backward(x, wg, wu, gate, up, dwide[:, 8:], "silu", *got)


def test_no_tokens(m):
    x, wg, wu, dh = make(0, 64, 32, torch.float16)
    h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    assert h.shape == (0, 64)
    dw = [torch.full((64, 32), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    dx, a, b = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, dw_gate=dw[0], dw_up=dw[1])
    assert dx.shape == (0, 32) and (a == 0).all() and (b == 0).all()


@pytest.mark.parametrize("M", [3, 300])
def test_not_finite_rows_stay_alone(m, M):
    """A row with an infinity or NaN gives no other row another result."""
    x, wg, wu, _ = make(M, 136, 200, torch.bfloat16, seed=5)
    want = m.nvfp4_gated_ffn(x, wg, wu)
    x[1] = float("nan")
    x[2, 5] = float("inf")
    got = m.nvfp4_gated_ffn(x, wg, wu)
    keep = [r for r in range(M) if r not in (1, 2)]
    assert torch.equal(got[keep], want[keep])
    assert got[1].isnan().all() and not got[2].isfinite().all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_large_gate_values(m, act):
    """Gates far outside the activation's bend: act(g) is g or 0, the derivative 1 or 0."""
    x = torch.eye(64, device="cuda").bfloat16() * 8
    gates = torch.tensor([-3e38, -1e5, -200.0, -60.0, 60.0, 200.0, 1e5, 3e37], device="cuda")
    wg = (gates / 8)[:, None].expand(8, 64).bfloat16().contiguous()
    wu = torch.full((8, 64), 0.125, dtype=torch.bfloat16, device="cuda")
    h, gate, up = m.nvfp4_gated_ffn(x, wg, wu, act, save=True)
    assert torch.equal(h[:, 4:].float(), gate[:, 4:]) and (h[:, :4].abs() < 1e-20).all()
    dh = torch.ones_like(h)
    dx, dwg, dwu = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, act)
    assert torch.equal(dwg[4:], x.t()[:1].expand(4, 64) * 0 + 8) and (dwg[:4].abs() < 1e-20).all()
    assert torch.equal(dwu[4:].float(), gate[:1, 4:].t().expand(4, 64) * 8)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradient_against_differences(m, act):
    """Along d = dx / max |dx| the loss sum dh h changes by t (dx . d): central differences, with the rounded points
    themselves. The loss is off by at most half_step sum |dh h|; the quadratic rest is t^2-small."""
    M, I, K = 24, 64, 48
    dtype = torch.float16
    x, wg, wu, dh = make(M, I, K, dtype, seed=11, dh_scale=1.0)
    _, gate, up = m.nvfp4_gated_ffn(x, wg, wu, act, save=True)
    grads = m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, act)
    loss = lambda *a: float((m.nvfp4_gated_ffn(*a, act).double() * dh.double()).sum())
    noise = 2 * half_step(dtype) * float((m.nvfp4_gated_ffn(x, wg, wu, act).double() * dh.double()).abs().sum())
    for at in range(3):
        point = [x, wg, wu]
        d = grads[at].double() / grads[at].double().abs().max()
        t = 0.06 if at == 0 else 0.02
        hi, lo = ((point[at].double() + s * t * d).to(dtype) for s in (1, -1))
        slope = float((grads[at].double() * (hi.double() - lo.double())).sum())
        there = loss(*[hi if i == at else p for i, p in enumerate(point)])
        back = loss(*[lo if i == at else p for i, p in enumerate(point)])
        assert abs(there - back - slope) <= noise + 0.02 * abs(slope), (at, there - back, slope, noise)
        assert noise < 0.2 * abs(slope)


def test_streams_and_graphs(m):
    """Two captured graphs with their own workspaces, replayed on new inputs, give what eager calls give."""
    x, wg, wu, dh = make(130, 264, 2048, torch.bfloat16, seed=1)
    want = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    want += m.nvfp4_gated_ffn_backward(x, wg, wu, want[1], want[2], dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = m.nvfp4_gated_ffn(x, wg, wu, save=True, stream=s)
    got += m.nvfp4_gated_ffn_backward(x, wg, wu, got[1], got[2], dh, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = m.nvfp4_gated_ffn(x, wg, wu, save=True)
            o += m.nvfp4_gated_ffn_backward(x, wg, wu, o[1], o[2], dh)
        graphs.append(g)
        outs.append(o)
    x.copy_(make(130, 264, 2048, torch.bfloat16, seed=2)[0])
    want = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    want += m.nvfp4_gated_ffn_backward(x, wg, wu, want[1], want[2], dh)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, o))


def test_refusals(m):
    x, wg, wu, dh = make(4, 64, 32, torch.bfloat16)
    _, gate, up = m.nvfp4_gated_ffn(x, wg, wu, save=True)
    for bad in (dict(x=x.float()), dict(w_gate=wg.half()), dict(w_up=wu[:, :24]), dict(x=x.cpu()), dict(w_up=wu[:32]),
                dict(x=x.t().contiguous().t()), dict(x=x[:1].expand(4, 32))):
        with pytest.raises(TypeError):
            m.nvfp4_gated_ffn(**{**dict(x=x, w_gate=wg, w_up=wu), **bad})
    with pytest.raises(ValueError):
        m.nvfp4_gated_ffn(x, wg, wu, "relu")
    for a in ((x[:, :28], wg[:, :28], wu[:, :28]), (x, wg[:60], wu[:60])):  # widths that are not multiples of 8
        with pytest.raises(m.NVFP4Error) as e:
            m.nvfp4_gated_ffn(*a)
        assert e.value.status == -2
    wide = torch.zeros(4, 48, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_gated_ffn(wide[:, 4:36], wg, wu)  # rows that do not start at 16 bytes
    assert e.value.status == -3
    for bad in (dict(gate=gate[:, :56]), dict(dh=dh[:3]), dict(dx=torch.empty(4, 40, dtype=x.dtype, device="cuda")),
                dict(up=torch.empty(4, 72, device="cuda")[:, :64]), dict(gate=gate.bfloat16())):
        with pytest.raises(TypeError):
            m.nvfp4_gated_ffn_backward(**{**dict(x=x, w_gate=wg, w_up=wu, gate=gate, up=up, dh=dh), **bad})
    with pytest.raises(ValueError):
        m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, need=(True, True))
    with pytest.raises(m.NVFP4Error) as e:  # over an operand that the other product still reads
        m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, dx=x)
    assert e.value.status == -1
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_gated_ffn_backward(x, wg, wu, gate, up, dh, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -6

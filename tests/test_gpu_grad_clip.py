"""Gradient norm and clipping on the GPU against sums in 64 bits.

The norm: a thread's sum of up to 64 squares in fp32 is off by at most 64 2^-24 of itself, the rest is fp64, the
result is rounded to fp32: 64 2^-24 / 2 + 2^-24 of the norm at most (the square root halves relative errors). A scaled
value is the fp32 product with the factor, rounded to the type: half a step, and the factor's own error."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NORM_TOL = 33 * 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def m():
    import moe_nvfp4_gemm_gb300
    return moe_nvfp4_gemm_gb300


def norm64(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def check(m, grads, max_norm, out=None, in_place=False):
    before = [t.clone() for t in grads]
    want = norm64(grads)
    norm = m.nvfp4_grad_clip(grads, max_norm, out=out)
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= NORM_TOL * want
    factor = min(1.0, max_norm / (want + 1e-6))
    for t, b, r in zip(grads, before, grads if out is None else out):
        assert out is None or torch.equal(t, b)
        tol = (torch.finfo(t.dtype).eps / 2 * 1.01 + NORM_TOL + 2.0 ** -22) * (b.double() * factor).abs() + 2.0 ** -25
        assert ((r.double() - b.double() * factor).abs() <= tol).all()
    return norm


def tensors(seed, sizes, dtypes, scale=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale).to(d) for s, d in zip(sizes, dtypes)]


# around a chunk of 16,384 values, a block's groups of eight loads, and 16 bytes
SIZES = [1, 2, 7, 8, 9, 255, 2047, 2048, 4100, 16383, 16384, 16385, 32768, 70001, 300000, 0, 5]


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("max_norm", [0.5, 1e3, 0.0])
def test_sizes(m, dtype, max_norm):
    grads = tensors(1, SIZES, [dtype] * len(SIZES))
    check(m, grads, max_norm, out=[torch.full_like(t, 3.0) for t in grads])
    check(m, grads, max_norm)


def test_mixed_types_and_one_value(m):
    check(m, tensors(2, [1000, 33, 40000, 7], [torch.float32, torch.bfloat16, torch.float16, torch.bfloat16]), 0.1)
    check(m, tensors(3, [1], [torch.float32]), 1e-3)


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("at,to", [(0, 0), (1, 1), (3, 3), (1, 2), (5, 0)])
def test_any_alignment(m, dtype, at, to):
    """Views that start anywhere in a buffer; what lies around them stays."""
    n = 20011
    flat = torch.full((n + 16,), 9.0, dtype=dtype, device="cuda")
    result = torch.full((n + 16,), 9.0, dtype=dtype, device="cuda")
    g = flat[at:at + n]
    g.copy_(tensors(4, [n], [dtype])[0])
    check(m, [g], 0.3, out=[result[to:to + n]])
    check(m, [g], 0.3)
    for b, o in ((flat, at), (result, to)):
        assert (b[:o] == 9).all() and (b[o + n:] == 9).all()


@pytest.mark.parametrize("count", [64, 65, 959, 960, 961, 2000])
def test_long_lists(m, count):
    grads = tensors(count, [1 + (i * 37) % 90 for i in range(count)], [TYPES[i % 3] for i in range(count)])
    check(m, grads, 0.5)
    big = tensors(6, [200000], [torch.float32])
    check(m, grads + big, 0.5)


def test_empty_lists(m):
    assert float(m.nvfp4_grad_clip([], 1.0)) == 0
    e = torch.empty(0, device="cuda")
    assert float(m.nvfp4_grad_clip([e, e], 1.0)) == 0
    z = torch.zeros(5000, device="cuda")
    assert float(m.nvfp4_grad_clip([z], 1.0)) == 0 and (z == 0).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-25, 1e-20, 1e15, 1e19, 1e25, 1e33])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_squares_outside_fp32(m, scale, dtype):
    grads = tensors(7, [30000, 9, 3], [dtype] * 3, scale)
    want = norm64(grads)
    assert abs(float(m.nvfp4_grad_clip(grads)) - want) <= NORM_TOL * want + 2.0 ** -149
    mixed = grads + tensors(8, [100], [torch.float32], 1.0)
    want = norm64(mixed)
    assert abs(float(m.nvfp4_grad_clip(mixed)) - want) <= NORM_TOL * want


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(m, value):
    grads = tensors(9, [5000, 300], [torch.bfloat16, torch.float32])
    grads[0][777] = value
    norm = m.nvfp4_grad_clip(grads, 1.0)
    f = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
    assert not norm.isfinite().any()
    if math.isnan(value):
        assert norm.isnan().all() and all(t.isnan().all() for t in grads)
    else:  # the factor is 0
        assert float(f) == 0 and (grads[1] == 0).all() and grads[0][777].isnan()


def test_norm_alone_and_no_limit(m):
    grads = tensors(10, [5000, 300], [torch.bfloat16, torch.float32])
    before = [t.clone() for t in grads]
    a = m.nvfp4_grad_clip(grads)
    assert all(torch.equal(x, y) for x, y in zip(grads, before))
    out = [torch.zeros_like(t) for t in grads]
    b = m.nvfp4_grad_clip(grads, out=out)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(out, before))
    # the same tensor twice counts twice where nothing is written
    assert abs(float(m.nvfp4_grad_clip(grads + grads)) - math.sqrt(2) * float(a)) <= 1e-6 * float(a)


def test_repeats_bit_for_bit_and_replays(m):
    grads = tensors(11, [1 << 20, 777, 33333], [torch.bfloat16, torch.float32, torch.float16])
    out = [torch.empty_like(t) for t in grads]
    norms = [m.nvfp4_grad_clip(grads, 0.1, out=out).clone() for _ in range(3)]
    first = [t.clone() for t in out]
    assert all(torch.equal(n, norms[0]) for n in norms)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = m.nvfp4_grad_clip(grads, 0.1, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(n, norms[0]) and all(torch.equal(a, b) for a, b in zip(out, first))
    graphs = []
    for _ in range(2):
        o = [torch.empty_like(t) for t in grads]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            n = m.nvfp4_grad_clip(grads, 0.1, out=o)
        graphs.append((g, n, o))
    grads[0].mul_(3.0)
    want = m.nvfp4_grad_clip(grads, 0.1, out=out)
    for g, _, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, n, o in graphs:
        assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(o, out))


def test_refusals(m):
    g = torch.ones(64, device="cuda")
    for bad in (dict(grads=[g.double()]), dict(grads=[g.cpu()]), dict(grads=[torch.ones(8, 8, device="cuda").t()]),
                dict(out=[]), dict(out=[g.bfloat16()]), dict(out=[g[:32]]), dict(norm=torch.zeros(1, device="cuda").double())):
        with pytest.raises(TypeError):
            m.nvfp4_grad_clip(**{**dict(grads=[g], max_norm=1.0), **bad})
    two = torch.ones(128, device="cuda")
    for grads, out in (([g, g], None), ([two[:100], two[50:]], None), ([two[:64], two[64:]], [two[64:], two[:64]]),
                       ([g, two[:64]], [two[64:], two[64:]])):
        with pytest.raises(m.NVFP4Error) as e:
            m.nvfp4_grad_clip(grads, 1.0, out=out)
        assert e.value.status == -1
    for bad in (-1.0, float("nan")):
        with pytest.raises(m.NVFP4Error) as e:
            m.nvfp4_grad_clip([g], bad)
        assert e.value.status == -1
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_grad_clip([g], 1.0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -6
    assert (g == 1).all() and (two == 1).all()

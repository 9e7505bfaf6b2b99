"""8-bit integer quantiser and product on the GPU: codes, scales and fp32 results are those of the stated fp32
operations bit for bit (the sums are whole numbers, exact in 64 bits); 16-bit results are their rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import moe_nvfp4_gemm_gb300
    return moe_nvfp4_gemm_gb300


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def formula(x):
    """The quantiser's operations in fp32 (rows with amax of at least 2^-100)."""
    v = x.float()
    amax = v.abs().amax(1)
    one = torch.ones_like(amax)
    s = torch.where(amax > 0, amax / 127.0, one)
    inv = torch.where(amax > 0, 127.0 / torch.where(amax > 0, amax, one), one)
    return torch.round(v * inv[:, None]).to(torch.int8), s


@pytest.mark.parametrize("M,K", [(1, 16), (3, 240), (7, 1024), (300, 1040), (33, 8192), (1500, 272), (2, 32768), (3, 32784), (2, 80000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_quantise(m, M, K, dtype):
    r = rand(M + K)
    x = r(M, K) * torch.exp(2 * r(M, 1))
    x[M // 2] = 0
    x = x.to(dtype)
    q, s = m.nvfp4_int8_quantize(x)
    want_q, want_s = formula(x)
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    assert s[M // 2] == 1 and (q[M // 2] == 0).all()
    # a view of wider rows
    wide = torch.full((M, K + 24), float("nan"), dtype=dtype, device="cuda")
    wide[:, 8:8 + K] = x
    q2, s2 = m.nvfp4_int8_quantize(wide[:, 8:8 + K])
    assert torch.equal(q2, q) and torch.equal(s2, s)


def test_quantise_ties_and_extremes(m):
    # amax 127: scale 1, halves are ties to even
    x = torch.zeros(1, 64, device="cuda")
    x[0, :9] = torch.tensor([127, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 125.5, -127])
    q, s = m.nvfp4_int8_quantize(x.half())
    assert s.item() == 1 and q[0, :9].tolist() == [127, 0, 2, 2, 0, -2, -126, 126, -127]


def test_quantise_tiny_rows(m):
    """Down to the smallest bf16 numbers: 127 / amax would be infinite. Codes within half a step of x / scale, the
    product of the fp32 operations off by less than 2^-20 steps; scales within half of fp32's spacing there, 2^-150."""
    r = rand(1)
    x = torch.stack([r(256) * 2.0 ** -e for e in (90, 99, 101, 110, 120, 126, 130)]).bfloat16()
    x = torch.cat([x, torch.zeros(1, 256, device="cuda").bfloat16()])
    x[-1, 3] = 2.0 ** -133
    q, s = m.nvfp4_int8_quantize(x)
    amax = x.double().abs().amax(1)
    assert ((s.double() - amax / 127).abs() <= 2.0 ** -150 + 2.0 ** -24 * amax / 127).all()
    exact = x.double() * 127 / amax[:, None]
    assert ((q.double() - exact).abs() <= 0.5 + 2.0 ** -16).all()
    assert q[-1, 3] == 127


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("K", [64, 4096, 40000])
def test_quantise_not_finite(m, dtype, K):
    x = rand(2)(6, K).to(dtype)
    want = m.nvfp4_int8_quantize(x)
    x[1, 5], x[2, K - 1], x[4, 0] = float("nan"), float("inf"), -float("inf")
    q, s = m.nvfp4_int8_quantize(x)
    assert s[[1, 2, 4]].isnan().all() and (q[[1, 2, 4]] == 0).all()
    assert torch.equal(q[[0, 3, 5]], want[0][[0, 3, 5]]) and torch.equal(s[[0, 3, 5]], want[1][[0, 3, 5]])


def product(a, sa, b, sb):
    total = a.double() @ b.double().t()
    return (total.float() * sa[:, None]) * sb


def codes(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


# one token to tile edges of 64, 128 and 256; channels odd, below and past a tile; K inside a block of 128, past a
# chunk of 1,024, and long enough to be cut into parts
SIZES = [(1, 1, 16), (1, 8, 144), (2, 300, 1024), (1, 4096, 8192), (17, 1000, 1040), (64, 256, 2064), (65, 257, 4096), (77, 5003, 2064),
         (128, 520, 96), (129, 130, 528), (255, 2049, 1552), (256, 512, 8192), (300, 7, 3088), (513, 1024, 2304), (1111, 777, 272)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(m, M, N, K):
    a, b = codes(M + N, M, K), codes(K + N, N, K)
    r = rand(K)
    sa, sb = (r(M) * 1e-2).abs() + 1e-3, (r(N) * 1e-3).abs() + 1e-4
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = product(a, sa, b, sb)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        assert m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=dtype, y=y, dev_status=status) is y
        off = (y[:M] != want.to(dtype)).nonzero()
        assert off.shape[0] == 0, (dtype, off.shape[0], off[:5].tolist(), y[off[0][0], off[0][1]], want[off[0][0], off[0][1]])
        assert (y[M] == 7).all()  # the row behind the last
    assert int(status) == 0


# tiles of 256 tokens (fp16 through the workspace), whole and in two and three parts; the others above take smaller ones
@pytest.mark.parametrize("M,N,K", [(129, 12175, 496), (256, 8192, 8192), (300, 4000, 8192), (512, 2579, 8192), (513, 8200, 1040), (600, 5003, 2064),
                                   (700, 7000, 80), (1100, 5003, 512), (1111, 2300, 272), (5000, 4100, 1040)])
def test_product_of_wide_tiles(m, M, N, K):
    assert m.nvfp4_int8_gemm_workspace_bytes(M, N, K) == 2 * M * K
    test_product(m, M, N, K)


@pytest.mark.parametrize("M,N", [(3, 200), (100, 200), (300, 200), (600, 5300)])
@pytest.mark.parametrize("K", [1024, 4096, 20000])
def test_largest_sums_in_each_kernel(m, M, N, K):
    """Sums of equal signs and odd ones beside them, in the kernels of up to 8, 64, 128 and 256 tokens a tile."""
    assert (m.nvfp4_int8_gemm_workspace_bytes(M, N, K) > 0) == (N == 5300)
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    a[1], b[1] = 127, 127
    b[2, ::2], a[2, ::3], b[5], a[0, K - 1], b[0, K - 1], b[N - 1, 0] = 127, 1, codes(5, K), 1, 1, 3
    y = m.nvfp4_int8_gemm(a, torch.ones(M, device="cuda"), b, torch.ones(N, device="cuda"), M, N, K, out_dtype=torch.float32)
    assert torch.equal(y, (a.double() @ b.double().t()).float())


@pytest.mark.parametrize("M", [3, 100, 300])
@pytest.mark.parametrize("K", [1024, 4096, 20000])
def test_largest_sums(m, M, K):
    """Sums of equal signs: 1,024 products reach 2^24, the largest number up to which fp32 holds every integer; odd
    products next to them would be lost in a shorter sum."""
    N = 200
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    a[1], b[1] = 127, 127
    b[2, ::2] = 127
    a[2, ::3] = 1
    b[5] = codes(5, K)
    a[0, K - 1] = 1
    b[0, K - 1] = 1
    b[7, 0] = 3
    one = lambda n: torch.ones(n, device="cuda")
    y = m.nvfp4_int8_gemm(a, one(M), b, one(N), M, N, K, out_dtype=torch.float32)
    assert torch.equal(y, (a.double() @ b.double().t()).float())


# a few tokens take a kernel of their own, up to 8: each number of tokens; channels and K on both sides of its pieces (4
# channels, 16 bytes, steps of 512 of K), K shared by one to eight warps
@pytest.mark.parametrize("M", range(1, 10))
@pytest.mark.parametrize("N,K", [(1, 16), (3, 48), (4, 512), (5, 528), (33, 1040), (257, 4112), (2050, 6160), (29000, 1552), (30000, 512)])
def test_few_tokens(m, M, N, K):
    a, b, r = codes(M, M, K), codes(N + K, N, K), rand(M * N)
    sa, sb = r(M).abs() + 1e-3, r(N).abs() + 1e-4
    want = product(a, sa, b, sb)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=dtype, y=y)
        assert torch.equal(y[:M], want.to(dtype)) and (y[M] == 7).all()
    sa[M - 1], sb[N - 1] = float("nan"), float("inf")
    y = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32)
    assert y[M - 1].isnan().all() and torch.equal(y[:M - 1, :N - 1], want[:M - 1, :N - 1])
    assert torch.equal(y[:, N - 1].isfinite(), torch.zeros(M, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("M", [2, 7, 12])
def test_weights_past_32_bits(m, M):
    N, K, times = 1003, 8192, 540  # 4.4 GB of weights
    a, b, r = codes(M, M, K), codes(N, N, K), rand(M)
    sa, sb = r(M).abs() + 1e-3, r(N).abs() + 1e-4
    y = m.nvfp4_int8_gemm(a, sa, b.repeat(times, 1), sb.repeat(times), M, N * times, K, out_dtype=torch.float32)
    assert torch.equal(y.view(M, times, N), product(a, sa, b, sb)[:, None].expand(M, times, N))


def test_few_tokens_in_a_graph(m):
    """Quantise and multiply, captured and replayed with other tokens: what the call reads is of this replay."""
    r = rand(3)
    x, w = r(4, 2048).bfloat16(), r(3000, 2048).bfloat16()
    b, sb = m.nvfp4_int8_quantize(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.nvfp4_int8_gemm(*m.nvfp4_int8_quantize(x), b, sb, 4, 3000, 2048)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = [m.nvfp4_int8_gemm(*m.nvfp4_int8_quantize(x), b, sb, 4, 3000, 2048, out_dtype=torch.float32) for _ in range(3)]
    for _ in range(3):
        x.copy_(r(4, 2048))
        g.replay()
        q, s = formula(x)
        want = product(q, s, b, sb)
        assert all(torch.equal(t, want) for t in y)


def test_longest_sum(m):
    K = 131056
    a, b = (torch.full((n, K), -128, dtype=torch.int8, device="cuda") for n in (2, 3))
    b[1] = 127
    one = torch.ones(3, device="cuda")
    y = m.nvfp4_int8_gemm(a, one[:2].contiguous(), b, one, 2, 3, K, out_dtype=torch.float32)
    assert torch.equal(y, (a.double() @ b.double().t()).float())


def test_scales_not_finite_stay_in_place(m):
    M, N, K = 70, 300, 256
    a, b = codes(1, M, K), codes(2, N, K)
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    want = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32)
    sa[3], sb[299] = float("nan"), float("nan")
    y = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32)
    assert y[3].isnan().all() and y[:, 299].isnan().all()
    rows = [i for i in range(M) if i != 3]
    assert torch.equal(y[rows][:, :299], want[rows][:, :299])


def test_layer_against_the_values(m):
    """Quantise and multiply: each operand is off by half a step of its row's scale."""
    M, N, K = 130, 264, 768
    r = rand(4)
    x, w = r(M, K).bfloat16(), (r(N, K) * 0.05).bfloat16()
    (a, sa), (b, sb) = m.nvfp4_int8_quantize(x), m.nvfp4_int8_quantize(w)
    y = m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32)
    X, W = x.double(), w.double()
    ex, ew = 0.5001 * sa.double()[:, None], 0.5001 * sb.double()[:, None]
    tol = ex * W.abs().sum(1)[None, :] + X.abs().sum(1)[:, None] * ew.t() + K * ex * ew.t()
    assert ((y.double() - X @ W.t()).abs() <= tol).all()


@pytest.mark.parametrize("M", [5, 90, 300])
def test_streams_and_graphs(m, M):
    N, K = 400, 2048
    x, w = rand(1)(M, K).bfloat16(), rand(2)(N, K).bfloat16()
    b, sb = m.nvfp4_int8_quantize(w)

    def layer(**kw):
        a, sa = m.nvfp4_int8_quantize(x, **kw)
        return m.nvfp4_int8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32, **kw)

    want = layer()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want, got)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer()
        graphs.append((g, out))
    x.copy_(rand(3)(M, K).bfloat16())
    want = layer()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)


def test_refusals(m):
    a, b = codes(1, 4, 32), codes(2, 8, 32)
    sa, sb = torch.ones(4, device="cuda"), torch.ones(8, device="cuda")
    ok = dict(a=a, sa=sa, b=b, sb=sb, M=4, N=8, K=32)
    for bad in (dict(a=a.float()), dict(a=a.cpu()), dict(b=b.t()), dict(sa=sa.double()), dict(sb=sb[:7]), dict(M=5), dict(N=9),
                dict(out_dtype=torch.int32), dict(y=torch.empty(4, 8, device="cuda"))):
        with pytest.raises(TypeError):
            m.nvfp4_int8_gemm(**{**ok, **bad})
    for K, status in ((24, -2), (131072, -2), (0, -1)):
        with pytest.raises(m.NVFP4Error) as e:
            m.nvfp4_int8_gemm(**{**ok, "K": K})
        assert e.value.status == status
    assert m.nvfp4_int8_gemm(a[:0], sa[:0], b, sb, 0, 8, 32).shape == (0, 8)
    big, wide = codes(3, 1025, 32), codes(4, 8192, 32)
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_int8_gemm(big, torch.ones(1025, device="cuda"), wide, torch.ones(8192, device="cuda"), 1025, 8192, 32, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -6
    x = torch.zeros(4, 32, device="cuda").bfloat16()
    for bad in (x.float(), x.cpu(), x.t(), x[0]):
        with pytest.raises(TypeError):
            m.nvfp4_int8_quantize(bad)
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_int8_quantize(x[:, :24])
    assert e.value.status == -2
    assert m.nvfp4_int8_quantize(x[:0])[0].shape == (0, 32)
    q, s = m.nvfp4_int8_quantize(x[:, :0])  # rows without values are rows of zeros
    assert q.shape == (4, 0) and (s == 1).all()
    assert math.isfinite(float(m.nvfp4_int8_quantize(x)[1][0]))

"""GPU checks of the FP8 block-128 quantiser and products against 64-bit restatements.

The quantiser is bit-exact (its recipe is IEEE fp32 steps, restated here in numpy). The products
meet the library's GEMM bound, |y - y_ref| <= 4e-3 |y_ref| + 1e-5 sum_k |a_k b_k| in bf16 (2^-9
relative for the output's rounding, fp32 sums of exact products), and 1e-5 sum_k |a_k b_k| in fp32.
"""
import numpy as np
import pytest
import torch

import moe_nvfp4_gemm_gb300 as m
from tests.helpers import dev

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def blocks(n):
    return (n + 127) // 128


def acts(M, K, seed, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=dev()) * scale
    x *= torch.where(torch.rand(M, K, generator=g, device=dev()) < 1e-2, 20.0, 1.0)
    return x.bfloat16()


def ref_quantize(x, block_rows):
    """numpy fp32: codes (as float32 values) and scales in the library's layouts."""
    x = x.float().cpu().numpy()
    M, K = x.shape
    R = M if block_rows == 1 else blocks(M) * 128
    p = np.zeros((R, blocks(K) * 128), np.float32)
    p[:M, :K] = x
    v = p.reshape(R // block_rows, block_rows, blocks(K), 128)
    amax = np.abs(v).max((1, 3))
    s = np.where(amax == 0, np.float32(1), amax / np.float32(448)).astype(np.float32)
    q = (v / s[:, None, :, None]).reshape(R, -1)[:M, :K]
    t = torch.from_numpy(np.clip(q, -448, 448)).to(FP8)
    return t, (s.T.copy() if block_rows == 1 else s)


def same_codes(got, want):
    assert got.dtype == FP8 and tuple(got.shape) == tuple(want.shape)
    assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


SHAPES = [(1, 16), (1, 128), (2, 144), (16, 256), (127, 128), (128, 128), (129, 400), (300, 1040), (257, 2048), (40, 6144)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(M, K, block_rows):
    x = acts(M, K, M + K)
    x[0, :16] = 0.0
    q, s = m.nvfp4_fp8_quantize(x, block_rows)
    wq, ws = ref_quantize(x, block_rows)
    same_codes(q, wq)
    assert np.array_equal(s.cpu().numpy(), ws)


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_transposed(M, K, block_rows):
    x = acts(M, K, M * 3 + K)
    q, s, qt, st = m.nvfp4_fp8_quantize(x, block_rows, transposed=True)
    wq, ws = ref_quantize(x, block_rows)
    same_codes(q, wq)
    assert np.array_equal(s.cpu().numpy(), ws)
    xt = torch.zeros(K, (M + 15) // 16 * 16, dtype=torch.bfloat16, device=dev())
    xt[:, :M] = x.t()
    wqt, wst = ref_quantize(xt, block_rows)
    same_codes(qt, wqt)
    assert np.array_equal(st.cpu().numpy(), wst)


def test_quantize_zeros_signs_and_extremes():
    x = torch.zeros(256, 256, dtype=torch.bfloat16, device=dev())
    x[3] = -0.0
    x[5, 7] = 3.3e38                 # block scale above the fast division's range
    x[6, ::3] = 1e-38                # and far below it
    x[7, 1::2] = -9.2e-41            # bf16 subnormals
    x[8, :] = torch.linspace(-1, 1, 256).bfloat16().to(dev())
    x[9, 0], x[9, 1] = 448.0, 1e-9
    for br in (1, 128):
        q, s, qt, st = m.nvfp4_fp8_quantize(x, br, transposed=True)
        wq, ws = ref_quantize(x, br)
        same_codes(q, wq)
        assert np.array_equal(s.cpu().numpy(), ws)
        wqt, wst = ref_quantize(x.t().contiguous(), br)
        same_codes(qt, wqt)
        assert np.array_equal(st.cpu().numpy(), wst)


def test_quantize_every_quotient_near_a_tie():
    """All bf16 significands over all bf16 block maxima's significands: every way to sit beside a tie."""
    sig = torch.arange(128, 256, dtype=torch.float32)
    x = torch.empty(128 * 16, 128, dtype=torch.float32)
    for e in range(16):
        for i in range(128):
            x[e * 128 + i] = sig * 2.0 ** -e  # the row's other values
            x[e * 128 + i, 0] = (128 + i) * 2.0   # the block's maximum
    x = x.bfloat16().to(dev())
    q, s = m.nvfp4_fp8_quantize(x)
    wq, ws = ref_quantize(x, 1)
    same_codes(q, wq)


@pytest.mark.parametrize("rows,M,K", [(1, 1, 16), (7, 3, 256), (512, 64, 400), (1000, 333, 2048)])
def test_quantize_gather(rows, M, K):
    x = acts(M, K, rows)
    g = torch.Generator(device=dev()).manual_seed(rows)
    idx = torch.randint(-1, M + 2, (rows,), generator=g, device=dev(), dtype=torch.int32)  # some outside [0, M)
    q, s = m.nvfp4_fp8_quantize(x, row_token=idx)
    inside = (idx >= 0) & (idx < M)
    xg = torch.where(inside[:, None], x[idx.long().clamp(0, M - 1)], torch.zeros((), dtype=torch.bfloat16, device=dev()))
    wq, ws = ref_quantize(xg, 1)
    same_codes(q, wq)
    assert np.array_equal(s.cpu().numpy(), ws)


def test_quantize_no_rows():
    q, s, qt, st = m.nvfp4_fp8_quantize(torch.empty(0, 256, dtype=torch.bfloat16, device=dev()), transposed=True)
    assert q.shape == (0, 256) and s.shape == (2, 0) and qt.shape == (256, 0) and st.shape == (0, 256)


# ---- products -----------------------------------------------------------------------------------


def decode(q, s, block_rows):
    v = q.double()
    rows, K = v.shape
    if block_rows == 1:
        return v * s.double().t().repeat_interleave(128, 1)[:, :K]
    return v * s.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :K]


def check(y, A, B):
    ref = A @ B.t()
    mag = A.abs() @ B.abs().t()
    err = (y.double() - ref).abs()
    bound = 1e-5 * mag + (4e-3 * ref.abs() if y.dtype == torch.bfloat16 else 0.0)
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), y[bad][:5].tolist(), ref[bad][:5].tolist())


GEMM_SHAPES = [(1, 1, 16), (1, 128, 128), (1, 8192, 2048), (2, 100, 144), (15, 257, 272), (16, 512, 1024), (17, 384, 640),
               (33, 1000, 2064), (64, 130, 4096), (77, 503, 1040), (127, 129, 384), (128, 256, 512), (129, 257, 528),
               (200, 640, 4112), (256, 256, 128), (300, 777, 256), (512, 1024, 1536), (1000, 333, 2000), (1025, 2050, 640)]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm(M, N, K, b_rows, out):
    a, sa = m.nvfp4_fp8_quantize(acts(M, K, M + K))
    b, sb = m.nvfp4_fp8_quantize(acts(N, K, N + K + 1, 0.02), b_rows)
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    guard = torch.full((M * N + 64,), 7.0, dtype=out, device=dev())
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows, out_dtype=out, y=guard[:M * N].view(M, N),
                         dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(y, decode(a, sa, 1), decode(b, sb, b_rows))
    assert (guard[M * N:] == 7.0).all()  # nothing past the output


@pytest.mark.parametrize("M,N,K", [(33, 10000, 144), (64, 9984, 2064), (65, 257, 400), (100, 12000, 1040), (128, 8, 16),
                                   (129, 1000, 272), (300, 2500, 528), (77, 9995, 3088)])
def test_gemm_tokens_on_the_narrow_side(M, N, K):
    """Dense sizes that take token tiles of up to 128 rows, and the same product in 256 x 256 tiles."""
    a, sa = m.nvfp4_fp8_quantize(acts(M, K, M + K))
    b, sb = m.nvfp4_fp8_quantize(acts(N, K, N, 0.02), 128)
    A, B = decode(a, sa, 1), decode(b, sb, 128)
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, dev_status=st)
    check(y, A, B)
    assert torch.equal(y, m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K))
    try:
        m.nvfp4_tune(m.NVFP4_TUNE_STREAM_MAX_M, -1)
        check(m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, dev_status=st), A, B)
    finally:
        m.nvfp4_tune(m.NVFP4_TUNE_STREAM_MAX_M, 0)
    assert st.item() == 0


@pytest.mark.parametrize("M,N,K", [(9, 260, 1536), (16, 384, 2064), (20, 8200, 1680), (32, 1000, 4112), (32, 9000, 400)])
def test_gemm_few_rows(M, N, K):
    a, sa = m.nvfp4_fp8_quantize(acts(M, K, M + K))
    b, sb = m.nvfp4_fp8_quantize(acts(N, K, N, 0.02), 128)
    check(m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K), decode(a, sa, 1), decode(b, sb, 128))


@pytest.mark.parametrize("M", [1, 5, 16, 31, 48, 100, 128, 160, 300])
def test_gemm_repeats_and_scales_apply_per_block(M):
    """Block scales that differ by powers of two between neighbours, ones codes: the result is a closed form."""
    N, K = 520, 1296
    kb = blocks(K)
    a = torch.ones(M, K, device=dev()).to(FP8)
    b = torch.ones(N, K, device=dev()).to(FP8)
    g = torch.Generator(device=dev()).manual_seed(M)
    sa = torch.exp2(torch.randint(-3, 4, (kb, M), generator=g, device=dev()).float())
    sb = torch.exp2(torch.randint(-3, 4, (blocks(N), kb), generator=g, device=dev()).float())
    lens = torch.full((kb,), 128.0, device=dev(), dtype=torch.float64)
    lens[-1] = K - 128 * (kb - 1)
    want = torch.einsum("cm,nc,c->mn", sa.double(), sb.double(), lens).repeat_interleave(128, 1)[:, :N]
    y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, out_dtype=torch.float32)
    assert torch.equal(y.double(), want)  # every sum is exact in fp32
    sb1 = torch.exp2(torch.randint(-3, 4, (kb, N), generator=g, device=dev()).float())
    y = m.nvfp4_fp8_gemm(a, sa, b, sb1, M, N, K, b_block_rows=1, out_dtype=torch.float32)
    assert torch.equal(y.double(), torch.einsum("cm,cn,c->mn", sa.double(), sb1.double(), lens))


@pytest.mark.parametrize("T,N,K", [(100, 256, 384), (257, 640, 512), (1, 144, 272)])
def test_linear_layer_gradients(T, N, K):
    """y = x W^T, dx = dy W, dW = dy^T x on quantised operands: each against the 64-bit product of the
    same codes, and against the exact gradient (the change of sum(dy * y) with x and W, which are
    linear) within what rounding an operand to E4M3 can do: 2^-4 of each value plus half the
    smallest step, 2^-10 of its block's scale."""
    x, dy = acts(T, K, 1), acts(T, N, 2, 0.1)
    w = acts(N, K, 3, 0.02)
    xq, xs, xqt, xst = m.nvfp4_fp8_quantize(x, transposed=True)
    dq, ds, dqt, dst = m.nvfp4_fp8_quantize(dy, transposed=True)
    wq, ws, wqt, wst = m.nvfp4_fp8_quantize(w, 128, transposed=True)
    Tp, Np = (T + 15) // 16 * 16, (N + 15) // 16 * 16
    assert Np == N  # N is the contraction length of dx

    def against(y, q1, s1, b1, q2, s2, b2, X1, X2):
        A, B = decode(q1, s1, b1), decode(q2, s2, b2)
        check(y, A, B)
        e1 = 2.0 ** -4 * X1.abs() + 2.0 ** -10 * decode(torch.ones_like(q1, dtype=torch.float32).to(FP8), s1, b1)[:, :X1.shape[1]]
        e2 = 2.0 ** -4 * X2.abs() + 2.0 ** -10 * decode(torch.ones_like(q2, dtype=torch.float32).to(FP8), s2, b2)[:, :X2.shape[1]]
        true = X1 @ X2.t()
        bound = e1 @ X2.abs().t() + X1.abs() @ e2.t() + e1 @ e2.t()
        out = 4e-3 * true.abs() + 4e-3 * bound + 1e-5 * (A.abs() @ B.abs().t())
        assert ((y.double() - true).abs() <= bound + out).all()

    X, W, D = x.double(), w.double(), dy.double()
    y = m.nvfp4_fp8_gemm(xq, xs, wq, ws, T, N, K)
    against(y, xq, xs, 1, wq, ws, 128, X, W)
    dx = m.nvfp4_fp8_gemm(dq, ds, wqt, wst, T, K, N)
    against(dx, dq, ds, 1, wqt, wst, 128, D, W.t())
    dw = m.nvfp4_fp8_gemm(dqt, dst, xqt, xst, N, K, Tp, b_block_rows=1, out_dtype=torch.float32)
    against(dw, dqt, dst, 1, xqt, xst, 1, D.t(), X.t())


def grouped_case(counts, N, K, seed, tail=0):
    E = len(counts)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    rows = int(off[-1]) + tail
    a, sa = m.nvfp4_fp8_quantize(acts(rows, K, seed))
    b = torch.empty(E, N, K, dtype=FP8, device=dev())
    sb = torch.empty(E, blocks(N), blocks(K), device=dev())
    for e in range(E):
        b[e], sb[e] = m.nvfp4_fp8_quantize(acts(N, K, seed * 1000 + e, 0.02), 128)
    if tail:  # what lies past the routed rows is anything
        a.view(torch.uint8)[rows - tail:] = 0x7F  # NaN codes
        sa[:, rows - tail:] = torch.nan
    return off, rows, a, sa, b, sb


@pytest.mark.parametrize("counts", [[1], [0, 0, 3], [5, 0, 16, 17, 1, 0, 128], [129, 0, 300, 1], [64] * 9, [1000, 3, 0, 257],
                                    [0, 0, 0, 513]])
@pytest.mark.parametrize("N,K", [(128, 128), (520, 1040), (257, 400)])
def test_grouped(counts, N, K):
    off, rows, a, sa, b, sb = grouped_case(counts, N, K, len(counts) + N, tail=3)
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=dev())
    m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, off.to(dev()), len(counts), rows, N, K, y=y, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for e in range(len(counts)):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            check(y[r], decode(a[r], sa[:, r].contiguous(), 1), decode(b[e], sb[e], 128))
    assert (y[int(off[-1]):] == 7.0).all()


@pytest.mark.parametrize("K", [16, 256, 272, 1024, 1152, 2192])
@pytest.mark.parametrize("N", [8, 131, 520])
def test_grouped_tokens_on_the_narrow_side(N, K):
    """Experts around the edges of a token tile (32, 64, 128 rows), odd and even numbers of blocks of K."""
    counts = [1, 33, 0, 64, 65, 127, 128, 129]
    off, rows, a, sa, b, sb = grouped_case(counts, N, K, N + K, tail=5)
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=dev())
    m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, off.to(dev()), len(counts), rows, N, K, y=y, dev_status=st)
    again = m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, off.to(dev()), len(counts), rows, N, K)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert torch.equal(again[:int(off[-1])], y[:int(off[-1])])
    for e in range(len(counts)):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            check(y[r], decode(a[r], sa[:, r].contiguous(), 1), decode(b[e], sb[e], 128))
    assert (y[int(off[-1]):] == 7.0).all()


def test_grouped_many_experts_of_few_rows():
    E, N, K = 80, 1160, 400
    counts = [int(v) for v in np.random.default_rng(5).poisson(3, E)]
    off, rows, a, sa, b, sb = grouped_case(counts, N, K, 6, tail=2)
    y = m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, off.to(dev()), E, rows, N, K)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            check(y[r], decode(a[r], sa[:, r].contiguous(), 1), decode(b[e], sb[e], 128))


@pytest.mark.parametrize("M,N,K", [(2600, 5200, 384), (1100, 9000, 144)])
@pytest.mark.parametrize("b_rows", [128, 1])
def test_gemm_more_tiles_than_ctas(M, N, K, b_rows):
    a, sa = m.nvfp4_fp8_quantize(acts(M, K, 1))
    b, sb = m.nvfp4_fp8_quantize(acts(N, K, 2, 0.02), b_rows)
    check(m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, b_block_rows=b_rows), decode(a, sa, 1), decode(b, sb, b_rows))


@pytest.mark.parametrize("mean", [6, 30, 60, 130, 600])
def test_grouped_more_items_than_ctas(mean):
    """Every kernel form of the grouped product (by rows per expert) with several items per CTA."""
    E, N, K = 24, 1160, 528
    g = np.random.default_rng(mean)
    counts = [int(v) for v in g.poisson(mean, E)]
    counts[3] = 0
    counts[7] = 2 * mean + 33  # more rows than a tile
    off, rows, a, sa, b, sb = grouped_case(counts, N, K, mean, tail=2)
    y = m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, off.to(dev()), E, rows, N, K)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            check(y[r], decode(a[r], sa[:, r].contiguous(), 1), decode(b[e], sb[e], 128))


def test_withheld_stage_is_reported_and_the_next_call_is_right():
    """The pipeline waits are bounded: a stage that never arrives ends in a status, not a hang."""
    cases = [(7, 520, 1024, 0), (7, 520, 1024, 1), (300, 520, 1024, 0)]  # streaming, split along K; tiles
    try:
        for M, N, K, split in cases:
            a, sa = m.nvfp4_fp8_quantize(acts(M, K, 1))
            b, sb = m.nvfp4_fp8_quantize(acts(N, K, 2, 0.02), 128)
            m.nvfp4_tune(m.NVFP4_TUNE_STREAM_SPLIT, split)
            m.nvfp4_tune(m.NVFP4_TUNE_WATCHDOG_US, 20000)
            m.nvfp4_tune(m.NVFP4_TUNE_TEST_WITHHOLD_STAGE, 2)
            st = torch.zeros(1, dtype=torch.int32, device=dev())
            m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, dev_status=st)
            torch.cuda.synchronize()
            assert st.item() == -7
            m.nvfp4_tune(m.NVFP4_TUNE_TEST_WITHHOLD_STAGE, 0)
            st.zero_()
            y = m.nvfp4_fp8_gemm(a, sa, b, sb, M, N, K, dev_status=st)
            assert st.item() == 0
            check(y, decode(a, sa, 1), decode(b, sb, 128))
        off, rows, a, sa, b, sb = grouped_case([5, 9, 200], 260, 512, 3)
        m.nvfp4_tune(m.NVFP4_TUNE_TEST_WITHHOLD_STAGE, 1)
        st = torch.zeros(1, dtype=torch.int32, device=dev())
        m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, off.to(dev()), 3, rows, 260, 512, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == -7
    finally:
        for key in (m.NVFP4_TUNE_STREAM_SPLIT, m.NVFP4_TUNE_WATCHDOG_US, m.NVFP4_TUNE_TEST_WITHHOLD_STAGE):
            m.nvfp4_tune(key, 0)


@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [1, 2, 3, 8], [0, 2, 4, 9], [0, -1, 4, 8]])
def test_grouped_bad_offsets_are_reported(bad):
    off, rows, a, sa, b, sb = grouped_case([2, 3, 3], 128, 256, 5)
    y = torch.full((rows, 128), 7.0, dtype=torch.bfloat16, device=dev())
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, torch.tensor(bad, dtype=torch.int32, device=dev()), 3, rows, 128, 256, y=y,
                             dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == -8 and (y == 7.0).all()


def test_grouped_moe_decode_shape():
    """256 experts, 512 tokens x 8: sampled experts of the routed product."""
    E, N, K, T = 256, 4096, 6144, 512
    g = torch.Generator(device=dev()).manual_seed(1)
    logits = torch.randn(T, E, generator=g, device=dev())
    r = m.nvfp4_moe_route(logits, 8, renormalize=True)
    a, sa = m.nvfp4_fp8_quantize(acts(T, K, 4), row_token=r.row_token)
    b = torch.randint(0, 256, (E, N, K), generator=g, device=dev(), dtype=torch.uint8)
    b[(b & 0x7F) == 0x7F] = 0  # no NaN codes
    sb = torch.rand(E, blocks(N), blocks(K), generator=g, device=dev()) * 1e-3
    y = m.nvfp4_fp8_grouped_gemm(a, sa, b, sb, r.expert_offsets, E, T * 8, N, K)
    off = r.expert_offsets.tolist()
    for e in (0, 1, 100, 255):
        s = slice(off[e], off[e + 1])
        check(y[s], decode(a[s], sa[:, s].contiguous(), 1), decode(b[e].view(FP8), sb[e], 128))


def test_products_in_a_graph_on_another_stream():
    a, sa = m.nvfp4_fp8_quantize(acts(9, 512, 1))
    b, sb = m.nvfp4_fp8_quantize(acts(700, 512, 2), 128)
    y0 = m.nvfp4_fp8_gemm(a, sa, b, sb, 9, 700, 512)
    off, rows, ga, gsa, gb, gsb = grouped_case([3, 0, 40], 256, 512, 3)
    off = off.to(dev())
    z0 = m.nvfp4_fp8_grouped_gemm(ga, gsa, gb, gsb, off, 3, rows, 256, 512)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            y1 = m.nvfp4_fp8_gemm(a, sa, b, sb, 9, 700, 512)
            z1 = m.nvfp4_fp8_grouped_gemm(ga, gsa, gb, gsb, off, 3, rows, 256, 512)
        for _ in range(3):
            g.replay()
    st.synchronize()
    assert torch.equal(y0, y1) and torch.equal(z0, z1)


# ---- refusals -----------------------------------------------------------------------------------


def test_refusals():
    x = acts(8, 256, 1)
    q, s = m.nvfp4_fp8_quantize(x)
    w, ws = m.nvfp4_fp8_quantize(acts(16, 256, 2), 128)
    for bad in (x.float(), x.t(), x.cpu(), x[0]):
        with pytest.raises(TypeError):
            m.nvfp4_fp8_quantize(bad)
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_fp8_quantize(acts(8, 24, 1))
    assert e.value.status == -2
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_fp8_quantize(x, 64)
    assert e.value.status == -1
    for args in ((q.float(), s, w, ws), (q, s.double(), w, ws), (q, s, w.t(), ws), (q, s, w, ws.cpu())):
        with pytest.raises(TypeError):
            m.nvfp4_fp8_gemm(*args, 8, 16, 256)
    with pytest.raises(TypeError):
        m.nvfp4_fp8_gemm(q, s, w, ws, 9, 16, 256)       # a holds fewer rows
    with pytest.raises(TypeError):
        m.nvfp4_fp8_gemm(q, s, w, ws, 8, 16, 256, out_dtype=torch.float16)
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_fp8_gemm(q, s, w, ws, 8, 16, 248)
    assert e.value.status == -2
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_fp8_gemm(q, s, w, ws, 8, 16, 256, b_block_rows=64)
    assert e.value.status == -1
    off = torch.tensor([0, 8], dtype=torch.int32, device=dev())
    with pytest.raises(m.NVFP4Error) as e:
        m.nvfp4_fp8_grouped_gemm(q, s, w.view(1, 16, 256), ws.view(1, 1, 2), off, 1, 8, 16, 256,
                                 workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    assert e.value.status == -6
    with pytest.raises(TypeError):
        m.nvfp4_fp8_grouped_gemm(q, s, w, ws, off.long(), 1, 8, 16, 256)

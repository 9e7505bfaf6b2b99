"""CPU checks of what may share memory in the dense feed-forward calls: every result and workspace over every operand and
every other result is refused before the device is touched. (Calls that are let through are in
test_gpu_dense_ffn_overlap.py, on memory that exists; here they end at a workspace that is too small.)"""
import ctypes

import pytest

P = ctypes.c_void_p
APART = 1 << 28  # bytes between two operands


@pytest.fixture(scope="module")
def lib():
    from moe_nvfp4_gemm_gb300 import build
    build.build()
    import moe_nvfp4_gemm_gb300 as m
    return m.lib()


def place(names):
    """An address of its own for each name."""
    return {n: 4096 + (i + 1) * APART for i, n in enumerate(names.split())}


def backward(lib, M, I, K, wsb, ldx=None, lddh=None, **over):
    a = {**place("x wg wu gate up dh dx dwg dwu ws"), **over}
    return lib.nvfp4_gated_ffn_backward(P(a["x"]), ldx or K, P(a["wg"]), K, P(a["wu"]), K, P(a["gate"]), P(a["up"]), P(a["dh"]), lddh or I,
                                        0, 0, P(a["dx"]), P(a["dwg"]), P(a["dwu"]), M, I, K, P(a["ws"]), wsb, None, None)


def test_gradients_and_the_parts_in_the_workspace(lib):
    """Few tiles: the workspace holds dg and du, 4 M I bytes, and behind them the fp32 sums of the products' parts."""
    M, I, K = 8, 4096, 256
    need = lib.nvfp4_gated_ffn_backward_workspace_bytes(M, I, K)
    parts = 4 * M * I
    assert need >= parts + 2 * 256 * 256 * 4
    ws = place("x wg wu gate up dh dx dwg dwu ws")["ws"]
    for at in (ws, ws + parts, ws + parts + 65536):
        for name in ("dx", "dwg", "dwu", "x", "wg", "wu", "gate", "up", "dh"):
            assert backward(lib, M, I, K, need, **{name: at}) == -1, (name, at - ws)
    for name in ("dx", "dwg", "dwu", "x", "wg", "wu", "gate", "up", "dh"):  # behind the workspace: let through
        assert backward(lib, M, I, K, 0, **{name: ws + need + 256}) == -6, name


def test_gradients_between_rows_that_lie_apart(lib):
    """A result in the gap between two rows of an operand shares nothing with it."""
    M, I, K, ld = 2, 64, 256, 4096
    x = place("x")["x"]
    assert backward(lib, M, I, K, 0, ldx=ld, dx=x + 2 * K) == -6            # dx takes 1,024 of the 7,680 bytes of the gap
    assert backward(lib, M, I, K, 0, ldx=ld, dx=x + 2 * ld - 1024) == -6    # up to the second row
    assert backward(lib, M, I, K, 0, ldx=ld, dx=x + 2 * ld - 1008) == -1 and backward(lib, M, I, K, 0, ldx=ld, dx=x + 2 * K - 16) == -1
    assert backward(lib, M, I, K, 0, ldx=ld, dx=x + 2 * ld + 2 * K - 16) == -1 and backward(lib, M, I, K, 0, ldx=ld, dx=x + 2 * ld + 2 * K) == -6
    assert backward(lib, M, I, K, 0, lddh=ld, dwg=place("x wg wu gate up dh")["dh"] + 128) == -1  # 32,768 bytes: over the second row


def forward(lib, M, I, K, wsb=1 << 27, ldx=None, ldh=None, save=True, **over):
    a = {**place("x wg wu h gate up ws"), **over}
    gate, up = (a["gate"], a["up"]) if save else (0, 0)
    return lib.nvfp4_gated_ffn(P(a["x"]), ldx or K, P(a["wg"]), K, P(a["wu"]), K, 0, 0, P(a["h"]), ldh or I, P(gate), P(up), M, I, K,
                               P(a["ws"]), wsb, None, None)


# streamed, in whole tiles, in parts
@pytest.mark.parametrize("M,I,K", [(5, 256, 256), (300, 256, 256), (256, 256, 8192)])
def test_forward(lib, M, I, K):
    at = place("x wg wu h gate up ws")
    row = 2 * K
    for name, size in (("x", M * row), ("wg", I * row), ("wu", I * row), ("gate", 4 * M * I), ("up", 4 * M * I)):
        assert forward(lib, M, I, K, h=at[name]) == -1, name
        assert forward(lib, M, I, K, h=at[name] + size - 16) == -1, name
        assert forward(lib, M, I, K, h=at[name] - 2 * M * I + 16) == -1, name
    for name, size in (("x", M * row), ("wg", I * row), ("wu", I * row), ("h", 2 * M * I), ("up", 4 * M * I)):
        assert forward(lib, M, I, K, gate=at[name]) == -1 and forward(lib, M, I, K, gate=at[name] + size - 32) == -1, name
    for name in ("x", "wg", "wu", "h", "gate"):
        assert forward(lib, M, I, K, up=at[name]) == -1, name
    assert forward(lib, M, I, K, save=False, h=at["x"]) == -1
    if lib.nvfp4_gated_ffn_workspace_bytes(M, I, K):
        need = lib.nvfp4_gated_ffn_workspace_bytes(M, I, K)
        for name in ("x", "wg", "wu", "h", "gate", "up"):
            assert forward(lib, M, I, K, ws=at[name]) == -1 and forward(lib, M, I, K, ws=at[name] - need + 16) == -1, name


@pytest.mark.parametrize("M", [5, 300])
def test_forward_rows_that_lie_apart(lib, M):
    """h and x as columns of one buffer, eight columns too near; and with strides of their own, where some rows meet."""
    I, K, ld = 128, 256, 512
    x = place("x")["x"]
    assert forward(lib, M, I, K, ldx=ld, ldh=ld, h=x + 2 * (K - 8)) == -1            # over the end of each row of x
    assert forward(lib, M, I, K, ldx=ld, ldh=ld, h=x + 2 * (ld - I + 8)) == -1       # over the start of the next row
    assert forward(lib, M, I, K, ldx=ld, ldh=ld, h=x + 2 * (ld * (M - 1) + K - 8)) == -1  # one row alone meets the last of x
    assert forward(lib, M, I, K, ldx=ld, ldh=ld, h=x - 2 * (ld * (M - 1) + I - 8)) == -1  # the last of h meets the first of x
    # rows of h 520 apart: the fourth ends eight columns into the next row of x
    assert forward(lib, M, I, K, ldx=ld, ldh=520, h=x + 2 * 368) == -1
    # rows of h twice as far apart as those of x
    assert forward(lib, M, I, K, ldx=ld, ldh=2 * ld, h=x + 2 * (K - 8)) == -1


@pytest.mark.parametrize("M,N,K", [(4, 512, 256), (40, 512, 256), (1025, 8192, 256)])
def test_int8_product(lib, M, N, K):
    at = place("a sa b sb y ws")
    need = lib.nvfp4_int8_gemm_workspace_bytes(M, N, K)

    def call(kind=1, **over):
        a = {**at, **over}
        return lib.nvfp4_int8_gemm(P(a["a"]), P(a["sa"]), P(a["b"]), P(a["sb"]), P(a["y"]), kind, M, N, K, P(a["ws"]), need, None, None)
    for name, size in (("a", M * K), ("sa", 4 * M), ("b", N * K), ("sb", 4 * N)):
        assert call(y=at[name]) == -1 and call(y=at[name] + (size - 1) // 16 * 16) == -1, name
        assert call(y=at[name] - 4 * M * N + 16) == -1 and call(kind=0, y=at[name] - 2 * M * N + 16) == -1, name
        if need:
            assert call(ws=at[name]) == -1 and call(ws=at[name] - need + 16) == -1, name
    if need:
        assert call(ws=at["y"]) == -1


def test_int8_quantiser(lib):
    M, K, ld = 8, 256, 1024
    at = place("x q s")

    def call(ldx=K, **over):
        a = {**at, **over}
        return lib.nvfp4_int8_quantize(P(a["x"]), ldx, 0, M, K, P(a["q"]), P(a["s"]), None)
    assert call(q=at["x"]) == -1 and call(q=at["x"] + 2 * M * K - 16) == -1 and call(q=at["x"] - M * K + 16) == -1
    assert call(s=at["x"]) == -1 and call(s=at["x"] + 2 * M * K - 4) == -1
    assert call(s=at["q"]) == -1 and call(q=at["s"]) == -1 and call(s=at["q"] + M * K - 4) == -1
    assert call(ldx=ld, q=at["x"] + 2 * K) == -1 and call(ldx=ld, s=at["x"] + 2 * ld - 4) == -1  # over the second row of x


@pytest.mark.parametrize("limit", [1.0, float("inf")])
@pytest.mark.parametrize("scaled", [False, True])
def test_clipping(lib, limit, scaled):
    """The norm and the workspace over a gradient, a result or each other."""
    src = [(1 << 24) + i * 65536 for i in range(70)]
    dst = [(1 << 25) + i * 65536 for i in range(70)]
    n = len(src)
    need = lib.nvfp4_grad_clip_workspace_bytes(n)

    def call(norm=1 << 20, ws=1 << 21):
        return lib.nvfp4_grad_clip((P * n)(*src), (P * n)(*dst) if scaled else None, (ctypes.c_int64 * n)(*[1000] * n),
                                   (ctypes.c_int32 * n)(*[i % 3 for i in range(n)]), n, limit, P(norm), P(ws), need, None)
    for i in (0, 33, 69):
        size = (2, 4, 2)[i % 3] * 1000
        for at in (src, dst) if scaled else (src,):
            assert call(norm=at[i]) == -1 and call(norm=at[i] + size - 4) == -1
            assert call(ws=at[i]) == -1 and call(ws=at[i] + (size - 1) // 16 * 16) == -1 and call(ws=at[i] - need + 16) == -1
    assert call(norm=1 << 21) == -1 and call(norm=(1 << 21) + need - 4) == -1

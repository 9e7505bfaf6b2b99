"""CPU checks of the gated block's, the int8 operators' and clipping's entry points: arguments rejected before the device is
touched, and the workspace sizes."""
import ctypes
import inspect
import os
import re

import pytest

P = ctypes.c_void_p
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    from moe_nvfp4_gemm_gb300 import build
    build.build()
    import moe_nvfp4_gemm_gb300 as m
    return m.lib()


def test_every_declared_symbol_is_exported(lib):
    import moe_nvfp4_gemm_gb300 as m
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nvfp4_ffn.h")
    src = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(nvfp4_[a-z0-9_]+)\s*\(", src)))
    assert sorted(m.EXPORTS_FFN) == names and all(hasattr(lib, n) for n in names) and all(hasattr(m, n) for n in names)


def test_every_call_with_a_stream_runs_on_it(monkeypatch):
    import moe_nvfp4_gemm_gb300 as m
    monkeypatch.setattr(m, "_on_stream", lambda stream, fn, args: (stream, fn, args))
    names = [n for n in m.EXPORTS_FFN if not n.endswith("_workspace_bytes")]
    assert len(names) == 5
    for n in names:
        fn = getattr(m, n)
        given = {p: i for i, p in enumerate(inspect.signature(fn).parameters)}
        assert fn(**given) == (given["stream"], fn, given)  # before anything is looked at or allocated
        assert "dev_status" not in given or "_status(dev_status)" in inspect.getsource(fn)


def test_gated_host_validation(lib):
    def call(x=64, ldx=256, wg=64, ldg=256, wu=64, ldu=256, kind=0, act=0, h=64, ldh=128, gate=0, up=0, M=300, I=128, K=256, ws=64,
             wsb=1 << 40):
        return lib.nvfp4_gated_ffn(P(x), ldx, P(wg), ldg, P(wu), ldu, kind, act, P(h), ldh, P(gate), P(up), M, I, K, P(ws), wsb,
                                   None, None)
    assert call(M=0) == 0
    assert call(M=-1) == -1 and call(I=0, ldh=8) == -1 and call(K=0) == -1 and call(kind=1) == -1 and call(act=2) == -1
    assert call(K=252) == -2 and call(I=124) == -2 and call(M=(1 << 30) + 1) == -2 and call(I=(1 << 24) + 8, ldh=1 << 25) == -2
    assert call(ldx=248) == -1 and call(ldg=255) == -1 and call(ldh=120) == -1 and call(ldx=260) == -2 and call(ldu=1 << 38) == -2
    assert call(x=0) == -1 and call(wu=0) == -1 and call(h=0) == -1 and call(gate=64) == -1 and call(up=64) == -1
    assert call(x=72) == -3 and call(wg=8) == -3 and call(h=24) == -3 and call(gate=16, up=32) == -3 and call(ws=8) == -3


def test_gated_workspaces(lib):
    assert lib.nvfp4_gated_ffn_workspace_bytes(1, 4096, 4096) == 0            # streamed
    assert lib.nvfp4_gated_ffn_workspace_bytes(4096, 14336, 8192) == 0        # more tiles than pairs
    need = lib.nvfp4_gated_ffn_workspace_bytes(256, 256, 8192)                # two tiles, 128 blocks: parts
    assert need > 0 and need % (2 * 256 * 256 * 4) == 0
    def call(ws, wsb):
        return lib.nvfp4_gated_ffn(P(64), 8192, P(64), 8192, P(64), 8192, 0, 0, P(64), 256, None, None, 256, 256, 8192, P(ws), wsb,
                                   None, None)
    assert call(0, need) == -6 and call(64, need - 1) == -6
    for M, I, K in ((0, 64, 64), (-1, 64, 64), (4, 60, 64), (4, 64, 0)):
        assert lib.nvfp4_gated_ffn_workspace_bytes(M, I, K) == 0 and lib.nvfp4_gated_ffn_backward_workspace_bytes(M, I, K) == 0
    assert lib.nvfp4_gated_ffn_backward_workspace_bytes(5, 64, 64) >= 5 * 64 * 4


def test_gated_backward_host_validation(lib):
    need = lib.nvfp4_gated_ffn_backward_workspace_bytes(300, 128, 256)
    apart = 1 << 24  # bytes between two operands
    def call(x=64, ldx=256, wg=64 + apart, wu=64 + 2 * apart, gate=64 + 3 * apart, up=64 + 4 * apart, dh=64 + 5 * apart, lddh=128, kind=2,
             act=1, dx=64 + 6 * apart, dwg=64 + 7 * apart, dwu=64 + 8 * apart, M=300, I=128, K=256, ws=256 + 9 * apart, wsb=need):
        return lib.nvfp4_gated_ffn_backward(P(x), ldx, P(wg), 256, P(wu), 256, P(gate), P(up), P(dh), lddh, kind, act, P(dx), P(dwg),
                                            P(dwu), M, I, K, P(ws), wsb, None, None)
    assert call(dx=0, dwg=0, dwu=0) == 0 and call(M=0, dwg=0, dwu=0) == 0     # nothing to do
    assert call(M=-1) == -1 and call(kind=1) == -1 and call(lddh=120) == -1 and call(K=250) == -2
    assert call(gate=0) == -1 and call(dh=0) == -1 and call(x=0) == -1 and call(wg=0) == -1
    assert call(dh=72) == -3 and call(dx=8) == -3 and call(ws=128) == -3
    assert call(ws=0) == -6 and call(wsb=need - 1) == -6
    # results over an operand, another result or the workspace: by a byte, or entirely
    assert call(dx=64) == -1 and call(dx=64 + 300 * 512 - 16) == -1 and call(dx=64 + 300 * 512, wsb=0) == -6
    assert call(dwg=64 + 8 * apart) == -1 and call(dwu=64 + apart) == -1 and call(ws=256 + 5 * apart) == -1
    assert call(dx=64 + 3 * apart + 300 * 128 * 4 - 16) == -1


def test_int8_host_validation(lib):
    def quantise(x=16, ldx=64, kind=0, M=4, K=64, q=16, s=16):
        return lib.nvfp4_int8_quantize(P(x), ldx, kind, M, K, P(q), P(s), None)
    assert quantise(M=0) == 0 and quantise(K=0, s=0) == -1
    assert quantise(M=-1) == -1 and quantise(kind=1) == -1 and quantise(ldx=56) == -1 and quantise(K=56) == -2 and quantise(ldx=68) == -2
    assert quantise(x=0) == -1 and quantise(s=0) == -1 and quantise(x=8) == -3 and quantise(q=8) == -3 and quantise(s=18) == -3

    def gemm(a=16, sa=16, b=16, y=16, kind=0, M=4, N=100, K=256, ws=16, wsb=1 << 30):
        return lib.nvfp4_int8_gemm(P(a), P(sa), P(b), P(16), P(y), kind, M, N, K, P(ws), wsb, None, None)
    assert gemm(M=0) == 0
    assert gemm(M=-1) == -1 and gemm(N=0) == -1 and gemm(kind=3) == -1 and gemm(a=0) == -1 and gemm(y=0) == -1
    assert gemm(K=100) == -2 and gemm(K=131072) == -2 and gemm(M=(1 << 30) + 1) == -2
    assert gemm(a=24) == -3 and gemm(y=24) == -3 and gemm(sa=18) == -3 and gemm(ws=8) == -3
    assert lib.nvfp4_int8_gemm_workspace_bytes(128, 64, 256) == 0 and lib.nvfp4_int8_gemm_workspace_bytes(1025, 8192, 256) == 1025 * 512
    assert gemm(M=1025, N=8192, ws=0) == -6 and gemm(M=1025, N=8192, wsb=1025 * 512 - 1) == -6


def test_clip_host_validation(lib):
    one = lib.nvfp4_grad_clip_workspace_bytes(1)
    assert one == lib.nvfp4_grad_clip_workspace_bytes(0) == lib.nvfp4_grad_clip_workspace_bytes(960) and one % 16 == 0
    assert lib.nvfp4_grad_clip_workspace_bytes(961) == 2 * one and lib.nvfp4_grad_clip_workspace_bytes(-1) == 0

    def call(grads=((64, 8, 1),), out=None, limit=1.0, norm=16, ws=16, wsb=1 << 20, count=None):
        n = len(grads)
        src = (P * n)(*[g[0] for g in grads])
        to = None if out is None else (P * n)(*out)
        return lib.nvfp4_grad_clip(src, to, (ctypes.c_int64 * n)(*[g[1] for g in grads]), (ctypes.c_int32 * n)(*[g[2] for g in grads]),
                                   n if count is None else count, limit, P(norm), P(ws), wsb, None)
    assert call(limit=-1.0) == -1 and call(limit=float("nan")) == -1 and call(norm=0) == -1 and call(count=-1) == -1
    assert call(grads=((0, 8, 1),)) == -1 and call(grads=((64, -1, 1),)) == -1 and call(grads=((64, 8, 3),)) == -1
    assert call(out=(0,)) == -1 and call(count=(1 << 24) + 1) == -2 and call(grads=((64, 1 << 41, 1),)) == -2
    assert call(grads=((66, 8, 1),)) == -3 and call(grads=((65, 8, 0),)) == -3 and call(out=(66,)) == -3 and call(norm=18) == -3 and call(ws=8) == -3
    assert call(ws=0) == -6 and call(wsb=one - 1) == -6
    # shared memory: the same gradient twice, an overlap of one value, a result over another gradient
    assert call(grads=((64, 8, 1), (64, 8, 1))) == -1 and call(grads=((64, 8, 1), (92, 8, 1))) == -1
    assert call(grads=((64, 8, 1), (128, 8, 1)), out=(128, 256)) == -1 and call(grads=((64, 8, 1), (128, 8, 1)), out=(256, 284)) == -1
    many = tuple((4096 + 64 * i, 16, 1) for i in range(100))
    assert call(grads=many + ((4096 + 64 * 50 + 60, 1, 1),)) == -1

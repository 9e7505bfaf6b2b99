"""CPU checks of the router's and the FP8 operators' entry points (arguments rejected before the
device is touched) and of the arithmetic that the FP8 quantiser replaces a division with."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from moe_nvfp4_gemm_gb300 import build
    build.build()
    import moe_nvfp4_gemm_gb300 as m
    return m.lib()


def test_route_host_validation(lib):
    def call(T=4, E=16, k=2, kind=1, logits=16, idx=16, counts=16, ws=16, wsb=1 << 20, mean=16):
        return lib.nvfp4_moe_route(P(logits), kind, None, T, E, k, 0, P(idx), P(16), P(16), P(counts), P(16), P(16), P(mean),
                                   P(16), P(16), P(ws), wsb, None)
    assert call(T=-1) == -1 and call(E=0) == -1 and call(k=0) == -1 and call(k=17) == -1 and call(kind=2) == -1
    assert call(E=1025) == -2 and call(E=64, k=33) == -2 and call(T=1 << 31) == -2 and call(T=(1 << 30) + 1, k=2) == -2
    assert call(logits=0) == -1 and call(idx=0) == -1 and call(counts=0) == -1 and call(mean=0) == -1
    assert call(logits=18) == -3 and call(idx=18) == -3 and call(counts=17) == -3
    assert call(kind=0, logits=17) == -3
    assert call(ws=0) == -6 and call(wsb=lib.nvfp4_moe_route_workspace_bytes(4, 16) - 1) == -6 and call(ws=24) == -3
    assert lib.nvfp4_moe_route_workspace_bytes(0, 16) == 0 and lib.nvfp4_moe_route_workspace_bytes(10, 2000) == 0
    one, many = (lib.nvfp4_moe_route_workspace_bytes(t, 256) for t in (1, 1 << 20))
    assert one == (2 * 256 + 1) * 4 and many == 304 * one


def test_route_backward_host_validation(lib):
    def call(T=4, E=16, k=2, logits=16, idx=16, d=16, dw=16):
        return lib.nvfp4_moe_route_backward(P(logits), 1, None, T, E, k, 0, P(idx), P(16), P(16), P(16), P(dw), P(16), P(d),
                                            None)
    assert call(T=0) == 0                      # nothing to do
    assert call(k=17) == -1 and call(E=1025) == -2
    assert call(logits=0) == -1 and call(idx=0) == -1 and call(d=0) == -1
    assert call(logits=18) == -3 and call(d=18) == -3 and call(dw=18) == -3


def test_fp8_quantize_host_validation(lib):
    def call(M_x=8, K=256, br=1, rt=0, M=8, x=16, q=16, s=16, qt=0, st=0):
        return lib.nvfp4_fp8_quantize(P(x), M_x, K, br, P(rt), M, P(q), P(s), P(qt), P(st), None)
    assert call(M=0, M_x=0) == 0
    assert call(M_x=-1) == -1 and call(br=64) == -1 and call(M=9) == -1       # M without a row list
    assert call(K=24) == -2 and call(M_x=1 << 31, M=1 << 31) == -2
    assert call(x=0) == -1 and call(q=0, s=0) == -1 and call(s=0) == -1 and call(qt=16) == -1
    assert call(x=8) == -3 and call(q=24) == -3 and call(s=18) == -3 and call(qt=16, st=8) == -3 and call(rt=18) == -3


def test_fp8_gemm_host_validation(lib):
    def call(M=4, N=100, K=256, br=128, kind=0, a=16, y=16, sa=16):
        return lib.nvfp4_fp8_gemm(P(a), P(sa), P(16), P(16), br, P(y), kind, M, N, K, None, None)
    assert call(M=0) == 0
    assert call(M=-1) == -1 and call(N=0) == -1 and call(br=2) == -1 and call(kind=2) == -1
    assert call(K=100) == -2 and call(M=(1 << 30) + 1) == -2
    assert call(a=0) == -1 and call(y=0) == -1
    assert call(a=24) == -3 and call(y=24) == -3 and call(sa=18) == -3


def test_fp8_grouped_host_validation(lib):
    need = lib.nvfp4_fp8_grouped_gemm_workspace_bytes(4, 100, 128, 256)
    def call(E=4, M=100, N=128, K=256, off=16, ws=256, wsb=need, a=16):
        return lib.nvfp4_fp8_grouped_gemm(P(a), P(16), P(16), P(16), P(off), E, M, N, K, P(16), P(ws), wsb, None, None)
    assert need > 0 and lib.nvfp4_fp8_grouped_gemm_workspace_bytes(0, 100, 128, 256) == 0
    assert call(E=0) == -1 and call(M=0) == 0 and call(off=0) == -1 and call(a=0) == -1
    assert call(K=200) == -2 and call(E=16385) == -2 and call(E=16384, N=1 << 17) == -2
    assert call(ws=0) == -6 and call(wsb=need - 1) == -6 and call(ws=272) == -3 and call(a=24) == -3


def test_two_part_reciprocal_rounds_as_the_division():
    """RN(x hi + RN(x lo)) == RN(x / s), s = RN(amax / 448), for all 8-bit significands of x <= amax and
    every exponent that reaches a code; the steps are those of the quantiser's fast path."""
    f32 = np.float32

    def nearest(v, exact):  # the float nearest to `exact`, ties to even, from an approximation
        cand = [np.nextafter(v, f32(0)), v, np.nextafter(v, f32(np.inf))]
        return min(cand, key=lambda c: (abs(Fraction(float(c)) - exact), int(c.view(np.uint32)) & 1))

    sig = np.arange(128, 256, dtype=np.float64)
    for A in range(128, 256):
        amax = f32(2 * A)
        s = nearest(f32(2 * A / 448.0), Fraction(2 * A, 448))
        inv = 1 / Fraction(float(s))
        hi = f32(1.0 / float(s))
        if Fraction(float(hi)) > inv:
            hi = np.nextafter(hi, f32(0))                            # rounded down
        rest = 1 - Fraction(float(s)) * Fraction(float(hi))
        assert Fraction(float(f32(float(rest)))) == rest             # the fma's remainder is exact
        lo = f32(float(f32(float(rest))) * float(hi))
        assert lo >= 0
        x = np.concatenate([sig * 2.0 ** (1 - e) for e in range(24)])
        x = x[x <= float(amax)]
        # x hi has at most 32 bits and RN(x lo) 24, at most 2^-23 of it: their sum fits the wider
        # type's significand or is rounded there far from a middle, then once to fp32
        t = (x.astype(np.longdouble) * np.longdouble(lo)).astype(f32)
        got = (x.astype(np.longdouble) * np.longdouble(hi) + t.astype(np.longdouble)).astype(f32)
        want = (x.astype(np.longdouble) / np.longdouble(s)).astype(f32)
        assert np.array_equal(got, want), A

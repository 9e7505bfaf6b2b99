// bf16 -> E4M3 codes with one fp32 scale for each block of 128 elements, in the forms that the
// FP8 product reads: 1 x 128 blocks along K (activations, gradients), 128 x 128 blocks (weights),
// and the same for the transpose (the operands of the products' gradients).
//
//   s = amax_block / 448 (1 for a block of zeros);  code = E4M3_rn_sat(x / s).
// A NaN does not count in amax and has a NaN code, so that it reaches the products through its own value
// alone; a block of nothing but NaN and zeros has scale 1. An infinity makes its block's scale infinite.
// Both divisions are IEEE round-to-nearest; the block scale is held in fp32 because the product
// applies it to fp32 sums (no rounding of the scale is needed).
#include <stdint.h>

#include <type_traits>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

constexpr int kFp8QuantThreads = 256;  // 16 groups of 8 rows x 16 groups of 8 columns

// 1 / s as an unevaluated sum hi + lo, hi rounded down and lo >= 0 the rounded rest (its remainder
// 1 - s hi is exact): hi + lo is within 2^-46 of 1 / s.
struct Reciprocal {
  float hi, lo;
};
DEVI Reciprocal fp8_reciprocal(float s) {
  Reciprocal y;
  y.hi = __frcp_rd(s);
  y.lo = __fmul_rn(__fmaf_rn(-s, y.hi, 1.0f), y.hi);
  return y;
}

// Eight E4M3 codes of v / s (element j in byte j), element pair j divided by s[j] (two scales).
// FAST: RN(x hi + RN(x lo)) is RN(x / s) for a bf16 x and s = RN(amax / 448) of a bf16 amax >= |x|:
// the sum is within 2^-46 of x / s, and no such quotient lies that close to the middle of two
// floats without being rounded alike (checked for all pairs of significands and all exponents that
// reach a code). x lo has x's sign, so that a zero keeps its own.
template <bool FAST>
DEVI uint2 e4m3_codes8(const uint4& w, const float2 (&s)[4], const float2 (&hi)[4], const float2 (&lo)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint16_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float xl = bf16lo(u[j]), xh = bf16hi(u[j]);
    float a, b;
    if (FAST) {
      const uint64_t xx = f2(xl, xh);
      f2_split(f2_fma(xx, f2(hi[j].x, hi[j].y), f2_mul(xx, f2(lo[j].x, lo[j].y))), a, b);
    } else {
      a = __fdiv_rn(xl, s[j].x);
      b = __fdiv_rn(xh, s[j].y);
    }
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[j]) : "f"(b), "f"(a));
  }
  return make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
}

// max(|a|, |b|) of two bf16 pairs; the sign bits of the result are to be ignored.
DEVI uint32_t maxabs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
DEVI uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Columns c0 .. c3 of four rows' code words (byte = column) as words (byte = row).
DEVI void transpose4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3, uint32_t (&c)[4]) {
  const uint32_t t0 = __byte_perm(r0, r1, 0x5140), t1 = __byte_perm(r2, r3, 0x5140);
  const uint32_t t2 = __byte_perm(r0, r1, 0x7362), t3 = __byte_perm(r2, r3, 0x7362);
  c[0] = __byte_perm(t0, t1, 0x5410);
  c[1] = __byte_perm(t0, t1, 0x7632);
  c[2] = __byte_perm(t2, t3, 0x5410);
  c[3] = __byte_perm(t2, t3, 0x7632);
}

// amax: the block's maximum but for NaN, NaN where it holds nothing else
DEVI float fp8_block_scale(float amax) { return amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f; }

// Scales for which the two-part reciprocal holds: hi, lo, the products that matter (quotients from
// 2^-11 on) and lo's remainder all stay clear of underflow; smaller quotients have code 0 anyway.
DEVI bool fp8_fast(float s) { return s >= 8.077935669463161e-28f && s <= 1.8446744073709552e19f; }  // 2^-90, 2^64

// One CTA = one 128 x 128 tile of x; thread (ty, tx) holds rows ty*8 .. +7, columns tx*8 .. +7
// (eight 16-byte loads in flight, a warp reads two 256-byte runs per load).
//   SQUARE: one scale for the tile, otherwise one for each row (q) and each column (qt).
// A row's maximum meets in its 16 lanes by recursive halving (each lane ends with the row tx / 2),
// so that a warp computes its 16 rows' scales (an IEEE division and a reciprocal, ~40 instructions)
// once, not once per row; the tile's 128 column scales are computed by one thread each.
// Bound by memory in the form without a transpose (4099 x 8192 13.1 us where x is in L2; 67 MB read and
// 35 written would take 15 from HBM), by instruction issue with it (25.9 us against 20.1 for its 136 MB)
// and for gathered rows (4096 x 6144 10.6 us, 32 MB: 4.8).
// qt goes through shared memory as bytes [column][row]; rows >= M and columns >= K read as 0, so
// the padding columns of qt (up to the next multiple of 16 rows) are written 0.
template <bool SQUARE, bool TRANSPOSED>
__global__ void __launch_bounds__(kFp8QuantThreads, TRANSPOSED ? 4 : 5) k_fp8_quantize(const Fp8QuantArgs a) {
  __shared__ __align__(16) uint8_t tile[TRANSPOSED ? 128 * 128 : 16];
  __shared__ __align__(16) uint32_t colmax[TRANSPOSED || SQUARE ? 8 : 1][64];  // per warp: |x| maxima of column pairs
  __shared__ __align__(16) float colscale[3][TRANSPOSED && !SQUARE ? 128 : 1];  // scale, its reciprocal's parts
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
  const int kbs = static_cast<int>((a.K + 127) / 128);
  const int64_t mb = blockIdx.x / kbs;
  const int kb = static_cast<int>(blockIdx.x % kbs);
  const int64_t m0 = mb * 128, k0 = static_cast<int64_t>(kb) * 128;
  const int64_t col = k0 + tx * 8;
  const bool col_ok = col < a.K;  // K is a multiple of 16: a group of 8 columns is whole
  uint4 v[8];
  const int64_t r0 = m0 + ty * 8;
  if (a.row_token) {
    int32_t src[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) src[i] = r0 + i < a.M ? __ldg(a.row_token + r0 + i) : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (col_ok && src[i] >= 0 && src[i] < a.M_x) v[i] = __ldg(reinterpret_cast<const uint4*>(a.x + src[i] * a.K + col));
    }
  } else {
    const uint16_t* x = a.x + r0 * a.K + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (col_ok && r0 + i < a.M) v[i] = __ldg(reinterpret_cast<const uint4*>(x));
      x += a.K;
    }
  }
  uint32_t rm[8], cm[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    rm[i] = maxabs_bf16x2(maxabs_bf16x2(u[0], u[1]), maxabs_bf16x2(u[2], u[3])) & 0x7FFF7FFFu;
    if (TRANSPOSED || SQUARE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) cm[j] = i == 0 ? u[j] : maxabs_bf16x2(cm[j], u[j]);
    }
  }
  float rs = 1.0f;  // SQUARE: the tile's scale, otherwise that of row ty*8 + tx/2
  if (!SQUARE) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {  // lanes 2 o apart exchange the halves of their rows
      const bool up = (tx & (2 * o)) != 0;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const uint32_t give = up ? rm[i] : rm[i + o], keep = up ? rm[i + o] : rm[i];
        rm[i] = max_bf16x2(keep, __shfl_xor_sync(0xffffffffu, give, 2 * o));
      }
    }
    rm[0] = max_bf16x2(rm[0], __shfl_xor_sync(0xffffffffu, rm[0], 1));
    rs = fp8_block_scale(fmaxf(bf16lo(rm[0]), bf16hi(rm[0])));
    const int64_t r = m0 + ty * 8 + (tx >> 1);
    if (a.q && (tx & 1) == 0 && r < a.M) a.s[static_cast<int64_t>(kb) * a.M + r] = rs;
  }
  if (TRANSPOSED || SQUARE) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      cm[j] = maxabs_bf16x2(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16)) & 0x7FFF7FFFu;
    if (lane < 16) *reinterpret_cast<uint4*>(&colmax[warp][tx * 4]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    __syncthreads();
  }
  if (SQUARE) {
    uint32_t m2 = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m2 = max_bf16x2(m2, max_bf16x2(colmax[w][lane], colmax[w][lane + 32]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m2 = max_bf16x2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    rs = fp8_block_scale(fmaxf(bf16lo(m2), bf16hi(m2)));
    if (tid == 0) {
      const int64_t mbs = (a.M + 127) / 128;
      if (a.q) a.s[mb * kbs + kb] = rs;
      if (TRANSPOSED) a.st[kb * mbs + mb] = rs;
    }
  } else if (TRANSPOSED) {
    if (tid < 64) {  // column pair tid
      uint32_t m2 = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) m2 = max_bf16x2(m2, colmax[w][tid]);
      const float s0 = fp8_block_scale(bf16lo(m2)), s1 = fp8_block_scale(bf16hi(m2));
      *reinterpret_cast<float2*>(&colscale[0][2 * tid]) = make_float2(s0, s1);
      const Reciprocal y0 = fp8_reciprocal(s0), y1 = fp8_reciprocal(s1);
      *reinterpret_cast<float2*>(&colscale[1][2 * tid]) = make_float2(y0.hi, y1.hi);
      *reinterpret_cast<float2*>(&colscale[2][2 * tid]) = make_float2(y0.lo, y1.lo);
      if (k0 + 2 * tid < a.K) *reinterpret_cast<float2*>(a.st + mb * a.K + k0 + 2 * tid) = make_float2(s0, s1);
    }
    __syncthreads();
  }
  uint2 codes[8];
  if (a.q || SQUARE) {
    const Reciprocal ry = fp8_reciprocal(rs);
    uint8_t* q = a.q ? a.q + r0 * a.K + col : nullptr;
    const int rows = a.q && col_ok ? static_cast<int>(min(int64_t(8), a.M - r0)) : 0;
    auto code_rows = [&](auto fast) {
      constexpr bool FAST = decltype(fast)::value;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        auto of_row = [&](float x) {
          const float f = SQUARE ? x : __shfl_sync(0xffffffffu, x, (lane & 16) + 2 * i);
          return make_float2(f, f);
        };
        const float2 s = FAST ? make_float2(0.0f, 0.0f) : of_row(rs);
        const float2 hi = FAST ? of_row(ry.hi) : s, lo = FAST ? of_row(ry.lo) : s;
        const float2 ss[4] = {s, s, s, s}, hh[4] = {hi, hi, hi, hi}, ll[4] = {lo, lo, lo, lo};
        codes[i] = e4m3_codes8<FAST>(v[i], ss, hh, ll);
        if (i < rows) *reinterpret_cast<uint2*>(q) = codes[i];
        q += a.K;
      }
    };
    if (__all_sync(0xffffffffu, fp8_fast(rs)))
      code_rows(std::true_type());
    else
      code_rows(std::false_type());
  }
  if (TRANSPOSED) {
    if (!SQUARE) {
      float2 cs[4], hi[4], lo[4];
      bool fast = true;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 s4 = *reinterpret_cast<const float4*>(&colscale[0][tx * 8 + 2 * j]);
        const float4 h4 = *reinterpret_cast<const float4*>(&colscale[1][tx * 8 + 2 * j]);
        const float4 l4 = *reinterpret_cast<const float4*>(&colscale[2][tx * 8 + 2 * j]);
        cs[j] = make_float2(s4.x, s4.y), cs[j + 1] = make_float2(s4.z, s4.w);
        hi[j] = make_float2(h4.x, h4.y), hi[j + 1] = make_float2(h4.z, h4.w);
        lo[j] = make_float2(l4.x, l4.y), lo[j + 1] = make_float2(l4.z, l4.w);
        fast = fast && fp8_fast(s4.x) && fp8_fast(s4.y) && fp8_fast(s4.z) && fp8_fast(s4.w);
      }
      fast = __all_sync(0xffffffffu, fast);
      if (fast) {
#pragma unroll
        for (int i = 0; i < 8; ++i) codes[i] = e4m3_codes8<true>(v[i], cs, hi, lo);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) codes[i] = e4m3_codes8<false>(v[i], cs, hi, lo);
      }
    }
    // 8 x 8 byte transpose: column tx*8 + j gets rows ty*8 .. +7 as one 8-byte unit, unit ty
    // stored at ty ^ tx so that a warp's 32 units of one j cover all banks
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8], top[4], bot[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = h == 0 ? codes[i].x : codes[i].y;
      transpose4(w[0], w[1], w[2], w[3], top);
      transpose4(w[4], w[5], w[6], w[7], bot);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(tile + (tx * 8 + h * 4 + j) * 128 + ((ty ^ tx) << 3)) = make_uint2(top[j], bot[j]);
    }
    __syncthreads();
    const int64_t ldt = (a.M + 15) / 16 * 16;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int c = p * 32 + (tid >> 3), u = tid & 7;  // output row (column of x), 16-byte unit
      const int cx = c >> 3;
      uint4 w = *reinterpret_cast<const uint4*>(tile + c * 128 + (((2 * u) ^ (cx & ~1)) << 3));
      if (cx & 1) w = make_uint4(w.z, w.w, w.x, w.y);
      if (k0 + c < a.K && m0 + u * 16 < ldt) *reinterpret_cast<uint4*>(a.qt + (k0 + c) * ldt + m0 + u * 16) = w;
    }
  }
}

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int block_rows, cudaStream_t st) {
  const int64_t grid = ((a.M + 127) / 128) * ((a.K + 127) / 128);
  const dim3 g(static_cast<unsigned>(grid));
  if (block_rows == 128) {
    if (a.qt)
      k_fp8_quantize<true, true><<<g, kFp8QuantThreads, 0, st>>>(a);
    else
      k_fp8_quantize<true, false><<<g, kFp8QuantThreads, 0, st>>>(a);
  } else {
    if (a.qt)
      k_fp8_quantize<false, true><<<g, kFp8QuantThreads, 0, st>>>(a);
    else
      k_fp8_quantize<false, false><<<g, kFp8QuantThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4

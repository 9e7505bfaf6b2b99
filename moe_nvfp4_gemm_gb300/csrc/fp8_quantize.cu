// bf16 -> E4M3 codes with one fp32 scale for each block of 128 elements, in the forms that the
// FP8 product reads: 1 x 128 blocks along K (activations, gradients), 128 x 128 blocks (weights),
// and the same for the transpose (the operands of the products' gradients).
//
//   s = amax_block / 448 (1 for a block of zeros);  code = E4M3_rn_sat(x / s).
// Both divisions are IEEE round-to-nearest; the block scale is held in fp32 because the product
// applies it to fp32 sums (no rounding of the scale is needed).
#include <stdint.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

constexpr int kFp8QuantThreads = 256;  // 16 groups of 8 rows x 16 groups of 8 columns

// Eight E4M3 codes of v / s (element j in byte j), for s with y = RN(1 / s).
DEVI uint2 e4m3_codes8(const uint4& w, const float (&s)[8], const float (&y)[8], bool fast) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint16_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = bf16lo(u[j]), hi = bf16hi(u[j]);
    float a, b;
    if (fast) {
      // x / s correctly rounded by the two fma corrections of div_rn_by, two elements at a time
      const uint64_t xx = f2(lo, hi), yy = f2(y[2 * j], y[2 * j + 1]), nd = f2(-s[2 * j], -s[2 * j + 1]);
      const uint64_t q0 = f2_mul(xx, yy);
      const uint64_t q1 = f2_fma(f2_fma(q0, nd, xx), yy, q0);
      f2_split(f2_fma(f2_fma(q1, nd, xx), yy, q1), a, b);
      a = with_sign_of(a, lo);
      b = with_sign_of(b, hi);
    } else {
      a = __fdiv_rn(lo, s[2 * j]);
      b = __fdiv_rn(hi, s[2 * j + 1]);
    }
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[j]) : "f"(b), "f"(a));
  }
  return make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
}

DEVI float fp8_block_scale(float amax) { return amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f); }

// Where the corrections are exact or cannot change a code: with 2^-90 <= s <= 1e30, an element
// of magnitude >= 2^-102 has an exact remainder (see div_rn_by), and a smaller one a quotient
// below 2^-12, less than half the smallest code's 2^-9: its code is 0 (with x's sign) either way.
DEVI bool fp8_fast(float s) { return s >= 8.077935669463161e-28f && s <= 1e30f; }

// One CTA = one 128 x 128 tile of x; thread (ty, tx) holds rows ty*8 .. +7, columns tx*8 .. +7
// (eight 16-byte loads in flight, a warp reads two 256-byte runs per load).
//   SQUARE: one scale for the tile, otherwise one for each row (q) and each column (qt).
// qt goes through shared memory as bytes [column][row]; rows >= M and columns >= K read as 0, so
// the padding columns of qt (up to the next multiple of 16 rows) are written 0.
template <bool SQUARE, bool TRANSPOSED>
__global__ void __launch_bounds__(kFp8QuantThreads) k_fp8_quantize(const Fp8QuantArgs a) {
  __shared__ __align__(16) uint8_t tile[TRANSPOSED ? 128 * 128 : 16];
  __shared__ __align__(16) uint32_t colmax[8][64];  // per warp: |x| maxima of column pairs
  __shared__ float rowscale[128];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
  const int kbs = static_cast<int>((a.K + 127) / 128);
  const int64_t mb = blockIdx.x / kbs;
  const int kb = static_cast<int>(blockIdx.x % kbs);
  const int64_t m0 = mb * 128, k0 = static_cast<int64_t>(kb) * 128;
  const int64_t col = k0 + tx * 8;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = m0 + ty * 8 + i;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < a.M && col < a.K) {  // K is a multiple of 16: a group of 8 columns is whole
      int64_t src = r;
      if (a.row_token) src = __ldg(a.row_token + r);
      if (src >= 0 && src < a.M_x) v[i] = __ldg(reinterpret_cast<const uint4*>(a.x + src * a.K + col));
    }
  }
  float rs[8];  // SQUARE: the tile's scale in rs[0]
  uint32_t cm[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu, v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu};
    uint32_t m2 = u[0];
#pragma unroll
    for (int j = 1; j < 4; ++j) asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(u[j]));
    if (TRANSPOSED || SQUARE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) asm("max.bf16x2 %0, %0, %1;" : "+r"(cm[j]) : "r"(u[j]));
    }
    if (!SQUARE) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const uint32_t w = __shfl_xor_sync(0xffffffffu, m2, o);
        asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(w));
      }
      rs[i] = fp8_block_scale(fmaxf(bf16lo(m2), bf16hi(m2)));
      if (tx == 0) rowscale[ty * 8 + i] = rs[i];
    }
  }
  float cs[8];
  if (TRANSPOSED || SQUARE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = __shfl_xor_sync(0xffffffffu, cm[j], 16);
      asm("max.bf16x2 %0, %0, %1;" : "+r"(cm[j]) : "r"(w));
    }
    if (lane < 16) *reinterpret_cast<uint4*>(&colmax[warp][tx * 4]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
  }
  __syncthreads();
  if (SQUARE) {
    uint32_t m2 = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(colmax[w][lane]));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(colmax[w][lane + 32]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint32_t w = __shfl_xor_sync(0xffffffffu, m2, o);
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(w));
    }
    rs[0] = fp8_block_scale(fmaxf(bf16lo(m2), bf16hi(m2)));
    if (tid == 0) {
      const int64_t mbs = (a.M + 127) / 128;
      if (a.q) a.s[mb * kbs + kb] = rs[0];
      if (TRANSPOSED) a.st[kb * mbs + mb] = rs[0];
    }
  } else {
    if (a.q && tid < 128 && m0 + tid < a.M) a.s[static_cast<int64_t>(kb) * a.M + m0 + tid] = rowscale[tid];
    if (TRANSPOSED) {
      uint32_t m2[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint4 c = *reinterpret_cast<const uint4*>(&colmax[w][tx * 4]);
        asm("max.bf16x2 %0, %0, %1;" : "+r"(m2[0]) : "r"(c.x));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(m2[1]) : "r"(c.y));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(m2[2]) : "r"(c.z));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(m2[3]) : "r"(c.w));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cs[2 * j] = fp8_block_scale(bf16lo(m2[j]));
        cs[2 * j + 1] = fp8_block_scale(bf16hi(m2[j]));
      }
      if (ty == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < a.K) a.st[mb * a.K + col + j] = cs[j];
      }
    }
  }
  uint2 codes[8];
  if (a.q || SQUARE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = SQUARE ? rs[0] : rs[i];
      const float y = __frcp_rn(s);
      const float ss[8] = {s, s, s, s, s, s, s, s}, yy[8] = {y, y, y, y, y, y, y, y};
      codes[i] = e4m3_codes8(v[i], ss, yy, fp8_fast(s));
      const int64_t r = m0 + ty * 8 + i;
      if (a.q && r < a.M && col < a.K) *reinterpret_cast<uint2*>(a.q + r * a.K + col) = codes[i];
    }
  }
  if (TRANSPOSED) {
    if (!SQUARE) {
      float y[8];
      bool fast = true;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = __frcp_rn(cs[j]);
        fast = fast && fp8_fast(cs[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) codes[i] = e4m3_codes8(v[i], cs, y, fast);
    }
    // 8 x 8 byte transpose: column tx*8 + j gets rows ty*8 .. +7 as one 8-byte unit, unit ty
    // stored at ty ^ tx so that a warp's 32 units of one j cover all banks
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t half = j < 4 ? codes[i].x : codes[i].y;
        w[i >> 2] |= ((half >> (8 * (j & 3))) & 0xFFu) << (8 * (i & 3));
      }
      *reinterpret_cast<uint2*>(tile + (tx * 8 + j) * 128 + ((ty ^ tx) << 3)) = make_uint2(w[0], w[1]);
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

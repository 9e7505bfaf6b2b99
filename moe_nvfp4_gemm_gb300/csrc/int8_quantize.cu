// Rows of 16-bit values to 8-bit integers with a scale for each row:
//   s = amax (1/127) (1 for a row of zeros),  code = rn(x (127 (1/amax))), ties to even: one division a row,
// every step, 1/127 and 1/amax too, one IEEE fp32 operation. Rows with an infinity or NaN: codes 0 and scale NaN, so that all
// that is made of them is NaN.
//
// Bound by memory (3 bytes a value): a CTA takes a row and holds it in registers, 32 values a thread, between
// the maximum and the codes; rows of more than 32,768 values are read twice, from L2 the second time. 4,099 rows of
// 8,192 take 14.0 us, the bytes 14.9 (a part of them stays in L2 between runs).
// Codes without a conversion instruction: x inv + 1.5 2^23 has the rounded integer in its low byte.
#include <stdint.h>

#include "ffn.cuh"
#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kVec = 4;  // 16-byte groups of a row a thread holds

// The larger magnitude of each half; a NaN stays one.
template <bool HALF>
DEVI uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  b &= 0x7FFF7FFFu;
  if (HALF)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool HALF>
DEVI uint32_t group_max(uint4 v, uint32_t m) {
  m = max_abs2<HALF>(m, v.x);
  m = max_abs2<HALF>(m, v.y);
  m = max_abs2<HALF>(m, v.z);
  return max_abs2<HALF>(m, v.w);
}

// Codes of eight values; `up` (a power of two) keeps 1 / amax in range for tiny rows.
template <bool HALF>
DEVI uint2 group_codes(uint4 v, float up, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t inv2 = f2(inv, inv);
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    f2_split(f2_mul(f2(unpack16<HALF>(w[j], 0) * up, unpack16<HALF>(w[j], 1) * up), inv2), lo, hi);
    c[2 * j] = __float_as_uint(__fadd_rn(lo, 12582912.0f));
    c[2 * j + 1] = __float_as_uint(__fadd_rn(hi, 12582912.0f));
  }
  uint2 r;
  r.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return r;
}

template <bool HALF, bool LONG>
__global__ void __launch_bounds__(1024) k_int8_quantize(const __grid_constant__ Int8QuantArgs p) {
  __shared__ uint32_t top[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int threads = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = static_cast<int>(p.K / 8);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const uint4* src = reinterpret_cast<const uint4*>(p.x + row * p.ldx);
    uint4 v[kVec];
    uint32_t m = 0;
    if (!LONG) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int g = threadIdx.x + j * threads;
        v[j] = g < groups ? src[g] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) m = group_max<HALF>(v[j], m);
    } else {
      for (int g = threadIdx.x; g < groups; g += threads) m = group_max<HALF>(src[g], m);
    }
    // magnitudes order as integers, NaN above infinity
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if (threads > 32) {
      // two buffers: a warp that writes one again has passed the barrier behind which all have read it
      if (lane == 0) top[parity][warp] = m;
      __syncthreads();
      m = __reduce_max_sync(0xffffffffu, lane < threads / 32 ? top[parity][lane] : 0u);
      parity ^= 1;
    }
    const float amax = unpack16<HALF>(m, 0);
    const bool finite = amax <= 3.4e38f;
    float scale = amax == 0.0f ? 1.0f : amax * (1.0f / 127.0f), up = 1.0f;
    if (!finite) scale = __int_as_float(0x7FFFFFFF);
    if (amax < 0x1p-100f) up = 0x1p100f;
    // not finite: codes 0 (every value is replaced below)
    const float inv = amax == 0.0f ? 1.0f : 127.0f * (1.0f / (amax * up));
    if (threadIdx.x == 0) p.s[row] = scale;
    uint2* dst = reinterpret_cast<uint2*>(p.q + row * p.K);
    if (!LONG) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int g = threadIdx.x + j * threads;
        if (g < groups) dst[g] = finite ? group_codes<HALF>(v[j], up, inv) : make_uint2(0, 0);
      }
    } else {
      for (int g = threadIdx.x; g < groups; g += threads)
        dst[g] = finite ? group_codes<HALF>(src[g], up, inv) : make_uint2(0, 0);
    }
  }
}

}  // namespace

cudaError_t launch_int8_quantize(const Int8QuantArgs& p, int sms, cudaStream_t st) {
  const bool is_long = p.K > 1024 * kVec * 8;
  int threads = is_long ? 1024 : static_cast<int>((p.K / 8 + kVec * 32 - 1) / (kVec * 32)) * 32;
  if (threads == 0) threads = 32;  // rows without values: scale 1
  const int64_t resident = static_cast<int64_t>(sms) * (2048 / threads < 32 ? 2048 / threads : 32) * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.M < resident ? p.M : resident));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = p.half ? (is_long ? k_int8_quantize<true, true> : k_int8_quantize<true, false>)
                       : (is_long ? k_int8_quantize<false, true> : k_int8_quantize<false, false>);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace nvfp4

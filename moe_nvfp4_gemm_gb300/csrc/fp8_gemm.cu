// FP8 block-scaled products: y[m, n] = sum_c sa[c, m] sb(c, n) sum_{k in block c} a[m, k] b[n, k],
// a, b E4M3, c running over blocks of 128 of K, sb one scale per 128 rows of b or per row.
#include <stdint.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

// Grouped: 0 = offsets[0] <= ... <= offsets[E] <= M; the verdict goes to *ok for the product.
__global__ void __launch_bounds__(256) k_fp8_check_offsets(const int32_t* __restrict__ offsets, int E, int64_t M,
                                                           int32_t* ok, int32_t* status) {
  bool good = offsets[0] == 0 && offsets[E] <= M;
  for (int e = threadIdx.x; e < E; e += 256) good = good && offsets[e] <= offsets[e + 1];
  good = __syncthreads_and(good) != 0;
  if (threadIdx.x == 0) {
    *ok = good;
    if (!good) report_status(status, kStatusBadOffsets);
  }
}

// One CTA per 64 x 64 tile of y (grouped: of one expert's rows), 4 x 4 outputs per thread; each
// 128-block's sum in fp32, then scaled into the fp32 result.
__global__ void __launch_bounds__(256) k_fp8_gemm(const Fp8GemmArgs p) {
  __shared__ float as[32][65], bs[32][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int e = blockIdx.z;
  const int64_t N = p.N, K = p.K;
  if (p.offsets && *p.ok == 0) return;
  const int64_t r_begin = p.offsets ? p.offsets[e] : 0, r_end = p.offsets ? p.offsets[e + 1] : p.M;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64;
  const uint8_t* b = p.b + e * N * K;
  const int64_t kbs = (K + 127) / 128;
  const float* sb = p.sb + e * ((N + 127) / 128) * kbs;
  for (int64_t m0 = r_begin + static_cast<int64_t>(blockIdx.y) * 64; m0 < r_end; m0 += static_cast<int64_t>(gridDim.y) * 64) {
    float acc[4][4] = {};
    for (int64_t c = 0; c < kbs; ++c) {
      float part[4][4] = {};
      for (int64_t k0 = c * 128; k0 < min(K, c * 128 + 128); k0 += 32) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * 32; i += 256) {
          const int r = i >> 5, kk = i & 31;
          as[kk][r] = (m0 + r < r_end && k0 + kk < K) ? e4m3_decode(p.a[(m0 + r) * K + k0 + kk]) : 0.0f;
          bs[kk][r] = (n0 + r < N && k0 + kk < K) ? e4m3_decode(b[(n0 + r) * K + k0 + kk]) : 0.0f;
        }
        __syncthreads();
        for (int kk = 0; kk < 32; ++kk)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[i][j] += as[kk][ty * 4 + i] * bs[kk][tx * 4 + j];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
          if (m < r_end && n < N)
            acc[i][j] += part[i][j] * (p.sa[c * p.M + m] * (p.b_rows == 1 ? sb[c * N + n] : sb[(n >> 7) * kbs + c]));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m < r_end && n < N) {
          if (p.f32)
            static_cast<float*>(p.y)[m * N + n] = acc[i][j];
          else
            static_cast<uint16_t*>(p.y)[m * N + n] = static_cast<uint16_t>(pack_bf16x2(acc[i][j], 0.0f) & 0xFFFFu);
        }
      }
  }
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& p, int E, cudaStream_t st) {
  if (p.offsets) k_fp8_check_offsets<<<1, 256, 0, st>>>(p.offsets, E, p.M, p.ok, p.status);
  const int64_t mt = (p.M + 63) / 64;
  dim3 grid(static_cast<unsigned>((p.N + 63) / 64), static_cast<unsigned>(E > 1 ? (mt / E + 1) : (mt < 65535 ? mt : 65535)),
            static_cast<unsigned>(E));
  k_fp8_gemm<<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4

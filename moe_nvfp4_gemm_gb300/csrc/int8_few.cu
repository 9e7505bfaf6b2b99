// Product of 8-bit integers for a few tokens, sums in 32-bit integers on the ordinary cores:
//   y[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k],  M <= 8.
//
// Bound by the weights' bytes with up to four tokens, given whole rounds of CTAs (28,672 x 8,192, 35 us of bytes: one 35.8 us, two 38.4,
// four 39.6; 8,192 x 8,192, 9.9: one 11.0, two 11.6; in tiles of the tensor cores, which convert every weight, 17.1). With five to
// eight the tokens' reads from L1 and the products count, two CTAs an SM (28,672 channels: 48). Three and more tokens
// do not split K at 8,192 channels: 256 CTAs put two on 104 SMs and one on 48, and the call takes as long as two on each would
// (four tokens 16.5 us; 9,728 channels, exactly two an SM, 17.6; 14,592, three, 21.4 of 17.6). A warp takes four channels, a lane 16 bytes of each at every 512 of K, with two such steps under
// way (a step is asked for as soon as the one two before it is summed): 16 to 32 warps and 64 to 128 KB an SM. The
// tokens' bytes, the same for all warps, stay in L1. Products of four bytes add to 32 bits (dp4a).
// Few channels: `split` warps of a CTA take a channel's steps in turn and add their sums through shared memory (whole
// numbers: any order gives the same).
#include <stdint.h>

#include "ffn.cuh"
#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kRows = 4, kSteps = 2, kWarps = kInt8FewRows / kRows;

// weights pass once: they do not displace the tokens in L1
DEVI int4 load_weights(const int8_t* p) {
  int4 v;
  asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int MT>
__global__ void __launch_bounds__(32 * kWarps, int8_few_resident(MT)) k_int8_few(const __grid_constant__ Int8FewArgs p) {
  __shared__ int part[kWarps][kRows * MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split, rows = kWarps / split * kRows;  // channels of the CTA
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * rows;
  const int M = static_cast<int>(p.M), K = static_cast<int>(p.K);
  griddep_wait();
  griddep_launch_dependents();

  const int64_t first = n0 + warp / split * kRows;
  const int last = first + kRows <= p.N ? kRows - 1 : (first < p.N ? static_cast<int>(p.N - 1 - first) : 0);
  const int8_t* w = p.b + (first < p.N ? first : p.N - 1) * p.K;
  int row_at[kRows];  // channels past the last: read again, not stored
#pragma unroll
  for (int r = 0; r < kRows; ++r) row_at[r] = min(r, last) * K;
  int sum[kRows][MT];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) sum[r][m] = 0;

  const int stride = 512 * split;
  int4 v[kSteps][kRows];
  int base = warp % split * 512;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    if (base + s * stride < K) {
      const int k = min(base + s * stride + lane * 16, K - 16);  // past the end: any weights, the tokens are 0
#pragma unroll
      for (int r = 0; r < kRows; ++r) v[s][r] = load_weights(w + row_at[r] + k);
    }
  for (; base < K; base += kSteps * stride) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (base + s * stride >= K) break;
      const int k = base + s * stride + lane * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        int4 x = make_int4(0, 0, 0, 0);
        if (k < K) x = *reinterpret_cast<const int4*>(p.a + min(m, M - 1) * K + k);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          sum[r][m] = __dp4a(v[s][r].w, x.w, __dp4a(v[s][r].z, x.z, __dp4a(v[s][r].y, x.y, __dp4a(v[s][r].x, x.x, sum[r][m]))));
      }
      const int next = base + (kSteps + s) * stride;
      if (next < K) {
        const int kn = min(next + lane * 16, K - 16);
#pragma unroll
        for (int r = 0; r < kRows; ++r) v[s][r] = load_weights(w + row_at[r] + kn);
      }
    }
  }

  int mine = 0;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int total = __reduce_add_sync(0xffffffffu, sum[r][m]);
      if (lane == r * MT + m) mine = total;
    }
  if (lane < kRows * MT) part[warp][lane] = mine;
  __syncthreads();
  const int row = threadIdx.x % rows, m = threadIdx.x / rows;
  const int64_t n = n0 + row;
  if (m >= M || n >= p.N) return;  // rows * MT is at most the CTA's threads
  int total = 0;
  for (int s = 0; s < split; ++s) total += part[row / kRows * split + s][row % kRows * MT + m];
  const float y = static_cast<float>(total) * p.sa[m] * p.sb[n];
  const int64_t at = static_cast<int64_t>(m) * p.N + n;
  if (p.out == kInt8OutF32)
    static_cast<float*>(p.y)[at] = y;
  else if (p.out == kInt8OutF16)
    static_cast<uint16_t*>(p.y)[at] = static_cast<uint16_t>(pack16<true>(y, 0.0f));
  else
    static_cast<uint16_t*>(p.y)[at] = static_cast<uint16_t>(pack16<false>(y, 0.0f));
}

}  // namespace

cudaError_t launch_int8_few(const Int8FewArgs& p, cudaStream_t st) {
  const int64_t rows = kWarps / p.split * kRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + rows - 1) / rows));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = p.M == 1 ? k_int8_few<1> : (p.M == 2 ? k_int8_few<2> : (p.M <= 4 ? k_int8_few<4> : k_int8_few<8>));
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace nvfp4

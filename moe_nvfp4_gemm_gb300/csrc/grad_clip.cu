// Norm over a list of gradients and clipping to a largest norm:
//   norm = sqrt(sum over all values of g^2),  f = min(1, max_norm / (norm + 1e-6)),  out = g f.
//
// Bound by memory: the gradients are read for the norm and, since every value needs the whole norm, once
// more for the scaling, and written once. The list travels in the kernels' parameters (no copy to the
// device, so that a captured graph carries it); it is cut into chunks of 16,384 values, which a fixed grid
// walks in strides, so that the order of the sums, and with it every bit of the result, depends on the sizes
// and types alone, wherever the gradients lie. The second kernel walks the chunks backwards: the last ones read are still
// in L2. Lists of up to 16 chunks take one launch: a cluster of eight CTAs, whose sums meet in distributed shared memory.
// (0.8 billion bf16 values: norm 230 us, scaling 495 us, the bytes of both passes at 6.7 TB/s.)
//
// Squares: a thread adds those of a chunk (up to 64) in fp32 and joins chunks in fp64. Where that fp32 sum is
// infinite (|g| > 2^63) or so small that squares fell below fp32's range, the thread's values are added
// again in fp64: the norm is right for every finite input (and infinite or NaN for the others). One beyond fp32's largest number
// is written as infinity, but the factor comes from its fp64 value.
#include <stdint.h>

#include "ffn.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kClipChunk;

template <int N>
struct ClipTable {
  ClipEntry e[N];
  int count;      // entries
  int chunks;     // chunks of all of them
  int slot0;      // first kernel: its first partial sum; second: 0 in the launch that writes the norm
  int slots;      // partial sums of all launches
  double* partial;
  float* norm;
  float max_norm;
  int scale;      // second kernel: scale, or the norm alone
};

// Entry that chunk c belongs to: the last one whose first chunk is <= c.
template <int N>
DEVI int clip_entry(const ClipTable<N>& t, int c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

DEVI float clip_value(const void* p, int64_t i, int type) {
  if (type == kClipF32) return static_cast<const float*>(p)[i];
  const uint32_t w = static_cast<const uint16_t*>(p)[i];
  return type == kClipF16 ? unpack16<true>(w, 0) : unpack16<false>(w, 0);
}

// The values [i0, i1) of a chunk as: single values up to the first 16-byte boundary, 16-byte groups, single
// values behind the last. Returns the groups' first value and count.
DEVI void clip_ranges(const void* p, int64_t i0, int64_t i1, int size, int64_t& v0, int& groups) {
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) + i0 * size) & 15u);
  const int64_t head = off ? (16 - off) / size : 0;
  v0 = i0 + head < i1 ? i0 + head : i1;
  groups = static_cast<int>((i1 - v0) * size / 16);
}

DEVI double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) total += sh[w];
  return total;
}

template <int TYPE>
DEVI void add_squares(uint4 v, float& s0, float& s1, uint32_t& any) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    any |= w[j];
    if (TYPE == kClipF32) {
      const float a = __uint_as_float(w[j]);
      (j & 1 ? s1 : s0) = fmaf(a, a, j & 1 ? s1 : s0);
    } else {
      const float a = unpack16<TYPE == kClipF16>(w[j], 0), b = unpack16<TYPE == kClipF16>(w[j], 1);
      s0 = fmaf(a, a, s0);
      s1 = fmaf(b, b, s1);
    }
  }
}

// How a gradient's groups of 16 bytes lie: at 16-byte boundaries, at those of words, or half a word behind them.
enum { kClipGroups, kClipWords, kClipHalves };

// This thread's squares of the values [i0, i1) of a chunk, of n in all. Which values a thread takes, and in which order, goes by
// their place in the chunk alone, so that the sums are the same wherever the gradient lies. Groups that do not start at a
// 16-byte boundary are read by words (the first finds the line, the others are in L1), five of them where they start
// half a word behind one; where one of the five ends outside the gradient, by half words.
// (0.8 billion bf16 values: 238 us at 16-byte boundaries, 247 at words, 272 half a word behind; groups put together
// from two 16-byte loads 303. A list of 30,000 values off the boundary takes 4.5 us, on it 4.2.)
template <int TYPE, int AT>
DEVI double chunk_squares(const void* p, int64_t i0, int64_t i1, int64_t n) {
  constexpr int SIZE = TYPE == kClipF32 ? 4 : 2, PER = 16 / SIZE;
  const int groups = static_cast<int>(i1 - i0) / PER;
  const int64_t tail = i0 + static_cast<int64_t>(groups) * PER;
  float s0 = 0.0f, s1 = 0.0f;
  uint32_t any = 0;
  const uintptr_t start = reinterpret_cast<uintptr_t>(p) + i0 * SIZE;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(AT == kClipHalves ? start - 2 : start);
  auto inside = [&](int g) {
    if (AT == kClipGroups) return reinterpret_cast<const uint4*>(start)[g];
    const uint32_t* q = words + 4 * g;
    const uint32_t w0 = q[0], w1 = q[1], w2 = q[2], w3 = q[3];
    if (AT == kClipWords) return make_uint4(w0, w1, w2, w3);
    const uint32_t w4 = q[4];
    return make_uint4(__funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16), __funnelshift_r(w2, w3, 16), __funnelshift_r(w3, w4, 16));
  };
  // groups whose five words all lie inside
  const int g0 = AT == kClipHalves && i0 == 0 ? 1 : 0, g1 = AT == kClipHalves && i1 == n && tail == n ? groups - 1 : groups;
  auto group = [&](int g) {
    if (AT != kClipHalves || (g >= g0 && g < g1)) return inside(g);
    uint32_t w[4];
    const uint16_t* half = reinterpret_cast<const uint16_t*>(start) + g * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = half[2 * j] | static_cast<uint32_t>(half[2 * j + 1]) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  constexpr int DEEP = AT == kClipHalves ? 4 : 8;
  int g = threadIdx.x;
  for (; g + (DEEP - 1) * kThreads < groups; g += DEEP * kThreads) {
    uint4 v[DEEP];
    if (AT != kClipHalves || (g >= g0 && g + (DEEP - 1) * kThreads < g1)) {  // no branch between the loads
#pragma unroll
      for (int j = 0; j < DEEP; ++j) v[j] = inside(g + j * kThreads);
    } else {
#pragma unroll
      for (int j = 0; j < DEEP; ++j) v[j] = group(g + j * kThreads);
    }
#pragma unroll
    for (int j = 0; j < DEEP; ++j) add_squares<TYPE>(v[j], s0, s1, any);
  }
  for (; g < groups; g += kThreads) add_squares<TYPE>(group(g), s0, s1, any);
  const int64_t behind = tail + threadIdx.x;  // at most 7 values: a thread each
  const bool has_behind = behind < i1;
  if (has_behind) {
    const float a = clip_value(p, behind, TYPE);
    s1 = fmaf(a, a, s1);
    any |= __float_as_uint(a);
  }
  const float s = s0 + s1;
  if ((s >= 0x1p-90f && s <= 0x1p127f) || (any & (TYPE == kClipF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return s;
  double d = 0.0;
  for (int q = threadIdx.x; q < groups; q += kThreads)
    for (int j = 0; j < PER; ++j) {
      const double a = clip_value(p, i0 + static_cast<int64_t>(q) * PER + j, TYPE);
      d += a * a;
    }
  if (has_behind) {
    const double a = clip_value(p, behind, TYPE);
    d += a * a;
  }
  return d;
}

// (calls of their own, so that their registers do not crowd the usual case)
template <int TYPE, int AT>
__device__ __noinline__ double chunk_squares_off(const void* p, int64_t i0, int64_t i1, int64_t n) {
  return chunk_squares<TYPE, AT>(p, i0, i1, n);
}

template <int TYPE>
DEVI double chunk_squares(const ClipEntry& e, int64_t i0, int64_t i1) {
  const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(e.src)) & 15u;
  if (at == 0) return chunk_squares<TYPE, kClipGroups>(e.src, i0, i1, e.numel);
  if (TYPE == kClipF32 || (at & 2) == 0) return chunk_squares_off<TYPE, kClipWords>(e.src, i0, i1, e.numel);
  return chunk_squares_off<TYPE, TYPE == kClipF32 ? kClipWords : kClipHalves>(e.src, i0, i1, e.numel);
}

// Squares of the chunks first, first + step, ... of this thread.
template <int N>
DEVI double list_squares(const ClipTable<N>& t, int first, int step) {
  double sum = 0.0;
  for (int c = first; c < t.chunks; c += step) {
    const ClipEntry& e = t.e[clip_entry(t, c)];
    const int64_t i0 = static_cast<int64_t>(c - e.first) * kChunk;
    const int64_t i1 = i0 + kChunk < e.numel ? i0 + kChunk : e.numel;
    if (e.type == kClipF32)
      sum += chunk_squares<kClipF32>(e, i0, i1);
    else if (e.type == kClipF16)
      sum += chunk_squares<kClipF16>(e, i0, i1);
    else
      sum += chunk_squares<kClipBf16>(e, i0, i1);
  }
  return sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_clip_norm(const __grid_constant__ ClipTable<N> t) {
  __shared__ double sh[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const double sum = block_sum(list_squares(t, blockIdx.x, gridDim.x), sh);
  if (threadIdx.x == 0) t.partial[t.slot0 + blockIdx.x] = sum;
}

// The factor min(1, max_norm / (norm + 1e-6)) as first * second; first is 1 but for factors below fp32's normal numbers, where
// it is a power of two that keeps both the second and all products whose result counts in range (a result of 2^-149 has
// a value of at least 2^-23 with a factor below 2^-126, of 2^41 with one below 2^-190). The norm that no fp32 number holds
// makes the fp32 quotient 0 and comes here in fp64.
struct ClipFactor {
  float first, second;
};

DEVI ClipFactor clip_factor(double norm64, float max_norm) {
  if (max_norm == __int_as_float(0x7F800000)) return {1.0f, 1.0f};
  const float q = max_norm / (static_cast<float>(norm64) + 1e-6f);
  if (q < 0x1p-126f && norm64 <= 0x1p1000) {  // an infinite norm's factor is 0
    const double d = max_norm / (norm64 + 1e-6);
    const float first = d < 0x1p-190 ? 0x1p-126f : (d < 0x1p-126 ? 0x1p-64f : 1.0f);
    return {first, static_cast<float>(d / first)};
  }
  return {1.0f, q > 1.0f ? 1.0f : q};  // NaN stays
}

DEVI float clip_scaled(float v, ClipFactor f) { return v * f.first * f.second; }

template <int TYPE>
DEVI uint4 scaled(uint4 v, ClipFactor f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = TYPE == kClipF32 ? __float_as_uint(clip_scaled(__uint_as_float(w[j]), f))
                            : pack16<TYPE == kClipF16>(clip_scaled(unpack16<TYPE == kClipF16>(w[j], 0), f),
                                                       clip_scaled(unpack16<TYPE == kClipF16>(w[j], 1), f));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int TYPE>
DEVI void scale_single(const void* p, void* out, int64_t i, ClipFactor f) {
  const float v = clip_scaled(clip_value(p, i, TYPE), f);
  if (TYPE == kClipF32)
    static_cast<float*>(out)[i] = v;
  else
    static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(pack16<TYPE == kClipF16>(v, 0.0f) & 0xFFFFu);
}

template <int TYPE>
DEVI void scale_chunk(const void* p, void* out, int64_t i0, int64_t i1, ClipFactor f) {
  constexpr int SIZE = TYPE == kClipF32 ? 4 : 2, PER = 16 / SIZE;
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15u) != 0) {
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) scale_single<TYPE>(p, out, i, f);
    return;
  }
  int64_t v0;
  int groups;
  clip_ranges(p, i0, i1, SIZE, v0, groups);
  const int64_t tail = v0 + static_cast<int64_t>(groups) * PER;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + v0 * SIZE);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + v0 * SIZE);
  constexpr int DEEP = 8;
  int g = threadIdx.x;
  for (; g + (DEEP - 1) * kThreads < groups; g += DEEP * kThreads) {
    uint4 v[DEEP];
#pragma unroll
    for (int j = 0; j < DEEP; ++j) v[j] = src[g + j * kThreads];
#pragma unroll
    for (int j = 0; j < DEEP; ++j) dst[g + j * kThreads] = scaled<TYPE>(v[j], f);
  }
  for (; g < groups; g += kThreads) dst[g] = scaled<TYPE>(src[g], f);
  if (i0 + threadIdx.x < v0) scale_single<TYPE>(p, out, i0 + threadIdx.x, f);
  if (tail + threadIdx.x < i1) scale_single<TYPE>(p, out, tail + threadIdx.x, f);
}

// The chunks of the list times min(1, max_norm / (norm + 1e-6)), 1 without a limit, the last ones first.
template <int N>
DEVI void list_scale(const ClipTable<N>& t, double norm, int first, int step) {
  const ClipFactor f = clip_factor(norm, t.max_norm);
  for (int c = t.chunks - 1 - first; c >= 0; c -= step) {
    const ClipEntry& e = t.e[clip_entry(t, c)];
    if (f.first * f.second == 1.0f && e.src == e.dst) continue;  // nothing changes
    const int64_t i0 = static_cast<int64_t>(c - e.first) * kChunk;
    const int64_t i1 = i0 + kChunk < e.numel ? i0 + kChunk : e.numel;
    if (e.type == kClipF32)
      scale_chunk<kClipF32>(e.src, e.dst, i0, i1, f);
    else if (e.type == kClipF16)
      scale_chunk<kClipF16>(e.src, e.dst, i0, i1, f);
    else
      scale_chunk<kClipBf16>(e.src, e.dst, i0, i1, f);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_clip_scale(const __grid_constant__ ClipTable<N> t) {
  __shared__ double sh[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  double sum = 0.0;
  for (int i = threadIdx.x; i < t.slots; i += kThreads) sum += t.partial[i];
  const double norm = sqrt(block_sum(sum, sh));
  if (blockIdx.x == 0 && threadIdx.x == 0 && t.slot0 == 0) *t.norm = static_cast<float>(norm);
  if (t.scale) list_scale(t, norm, blockIdx.x, gridDim.x);
}

// The whole list in one cluster.
template <int N>
__global__ void __launch_bounds__(kThreads) k_clip_cluster(const __grid_constant__ ClipTable<N> t) {
  __shared__ double sh[kThreads / 32], mine;
  griddep_wait();
  griddep_launch_dependents();
  const int rank = static_cast<int>(cluster_ctarank());
  const double sum = block_sum(list_squares(t, rank, kClipCluster), sh);
  if (threadIdx.x == 0) mine = sum;
  cluster_sync();
  double total = 0.0;
#pragma unroll
  for (int r = 0; r < kClipCluster; ++r) total += ld_shared_cluster_f64(mapa_shared(smem_u32(&mine), r));
  const double norm = sqrt(total);
  if (rank == 0 && threadIdx.x == 0) *t.norm = static_cast<float>(norm);
  if (t.scale) list_scale(t, norm, rank, kClipCluster);
  cluster_sync();  // no CTA leaves while another may still read its sum
}

template <typename Kernel, typename Table>
cudaError_t launch_clip(Kernel kernel, int grid, int cluster, cudaStream_t st, const Table& t) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, t);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// One kernel for the entries of a group.
template <int N>
cudaError_t run_group(const ClipArgs& a, const ClipGroup& g, ClipStep step, cudaStream_t st) {
  static_assert(sizeof(ClipTable<N>) <= 32764, "kernel parameters");
  ClipTable<N> t;
  t.count = 0;
  t.chunks = 0;
  for (int i = g.first; i < g.end; ++i) {
    ClipEntry e;
    if (!clip_list_entry(a, i, e)) continue;
    e.first = t.chunks;
    t.chunks += static_cast<int>((e.numel + kChunk - 1) / kChunk);
    t.e[t.count++] = e;
  }
  t.slot0 = g.slot0;
  t.slots = a.slots;
  t.partial = a.partial;
  t.norm = a.norm;
  t.max_norm = a.max_norm;
  t.scale = a.scale;
  if (step == kClipAll) return launch_clip(k_clip_cluster<N>, kClipCluster, kClipCluster, st, t);
  if (step == kClipScale) return launch_clip(k_clip_scale<N>, a.scale && g.grid > 0 ? g.grid : 1, 1, st, t);
  return launch_clip(k_clip_norm<N>, g.grid, 1, st, t);
}

}  // namespace

cudaError_t launch_clip_group(const ClipArgs& a, const ClipGroup& g, ClipStep step, cudaStream_t st) {
  const int n = g.end - g.first;  // short lists in a short table: the parameters are copied with every launch
  if (n <= 16) return run_group<16>(a, g, step, st);
  if (n <= 128) return run_group<128>(a, g, step, st);
  return run_group<kClipGroup>(a, g, step, st);
}

}  // namespace nvfp4

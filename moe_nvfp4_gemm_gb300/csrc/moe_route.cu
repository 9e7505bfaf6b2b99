// MoE router: softmax over the experts, top-k selection, per-expert counts, rows sorted by
// expert, the load-balance loss, and the gradient of the logits.
//
// For token t with logits l_te (e < E), routed when it is valid and some l_te > -inf:
//   p_te = exp(l_te - max) / sum;  the k largest l_te are selected, ties to the lowest expert,
//   an expert at -inf never (its slot holds -1 and weight 0);
//   w_ts = p at the selected experts, optionally divided by their sum.
// With n routed tokens, c_e selections of expert e and P_e = (1/n) sum_t p_te:
//   balance loss L = E sum_e (c_e / (n k)) P_e.
// A NaN is never selected and no maximum, but a valid token with one is routed like any other (also when it has
// nothing else above -inf): its p, its weights, the means, the loss and the gradient of its row are NaN, so
// that a router that has diverged shows.
// A routed row's place is offsets[e] + the number of earlier (token, slot) pairs that chose e,
// in (token, slot) order, so the order does not depend on how the work was split. Counts are
// integers and every floating sum runs in a fixed order: results repeat bit for bit.
#include <stdint.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

constexpr int kPlaceThreads = 256;
constexpr int kPlaceWarps = kPlaceThreads / 32;
constexpr float kLog2E = 1.4426950408889634f;

DEVI float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order-preserving map of fp32 (no NaN) onto uint32; 0 is below every float's key.
DEVI uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and +0 tie
  return u ^ ((u & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}
DEVI float key_value(uint32_t key) { return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu)); }
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;
constexpr int kCandSlots = 34;  // 32 candidates, read in pairs; 16-byte rows

// 1 / x to within a unit in the last place
DEVI float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of exp(v - max)
DEVI float route_arg(float v, float mx) { return (v - mx) * kLog2E; }

// Whether a valid token is routed: some logit above -inf (mx, the largest but for NaN, is), or NaN.
template <int VPL>
DEVI bool row_routed(const float (&v)[VPL], float mx) {
  if (mx > __uint_as_float(0xFF800000u)) return true;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < VPL; ++j) nan = nan || v[j] != v[j];
  return __any_sync(0xffffffffu, nan);
}

DEVI float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One row's logits: lane holds experts lane * VPL + j; experts >= E read as -inf.
template <int VPL, bool BF16>
DEVI void load_row(const void* logits, int64_t row, int E, bool vec, int lane, float (&v)[VPL]) {
  if (vec) {  // E == 32 * VPL, rows aligned to a lane's bytes
    if (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(logits) + row * E + lane * VPL;
      if constexpr (VPL >= 8) {
#pragma unroll
        for (int j = 0; j < VPL; j += 8) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + j));
          v[j] = bf16lo(w.x), v[j + 1] = bf16hi(w.x), v[j + 2] = bf16lo(w.y), v[j + 3] = bf16hi(w.y);
          v[j + 4] = bf16lo(w.z), v[j + 5] = bf16hi(w.z), v[j + 6] = bf16lo(w.w), v[j + 7] = bf16hi(w.w);
        }
      } else if constexpr (VPL >= 2) {
#pragma unroll
        for (int j = 0; j < VPL; j += 2) {
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p + j));
          v[j] = bf16lo(w), v[j + 1] = bf16hi(w);
        }
      } else {
        v[0] = __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
      }
    } else {
      const float* p = static_cast<const float*>(logits) + row * E + lane * VPL;
      if constexpr (VPL >= 4) {
#pragma unroll
        for (int j = 0; j < VPL; j += 4) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(p + j));
          v[j] = w.x, v[j + 1] = w.y, v[j + 2] = w.z, v[j + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) v[j] = __ldg(p + j);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = lane * VPL + j;
      v[j] = __uint_as_float(0xFF800000u);
      if (e < E)
        v[j] = BF16 ? __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(logits) + row * E + e)) << 16)
                    : __ldg(static_cast<const float*>(logits) + row * E + e);
    }
  }
}

// Warps per CTA of the routing kernels: 16, but 8 for more than 256 experts (registers, and the
// per-warp sums of p in shared memory).
template <int VPL>
struct RouteCfg {
  static constexpr int WARPS = VPL <= 8 ? 16 : 8;
  static constexpr int THREADS = 32 * WARPS;
};

// The k largest of a warp's 32 * VPL logits (lane holds experts lane * VPL + j), ties to the lower
// expert: a lane gets a slot and, where that is below k, its expert (-1: none above -inf is left for
// it) and logit; every slot below k is some lane's. `lane_max` is the largest of this lane's logits that are
// not NaN (-inf without one).
//
// The k-th largest of the 32 lane maxima bounds the k-th largest logit from below, so the selected
// experts are among the few (typically k and one or two) that reach it. Those candidates are
// compacted into `cand`, a lane takes one each and counts the ones that precede it, which is its
// slot: less than half the instructions of k rounds of a maximum over all. With more than 32
// candidates (many equal logits) the rounds are run.
template <int VPL>
DEVI void warp_top_k(const float (&v)[VPL], float lane_max, int k, uint64_t* cand, int& out_idx, float& out_val,
                     int& out_slot) {
  const int lane = threadIdx.x & 31;
  uint32_t bound = 0, left = order_key(lane_max);
#pragma unroll 2
  for (int s = 0; s < k; ++s) {  // equal maxima leave together: the bound is then lower, and still one
    bound = __reduce_max_sync(0xffffffffu, left);
    if (left == bound) left = 0;
  }
  bound = max(bound, kKeyNegInf + 1);
  const float least = key_value(bound);
  int n = 0;
  uint32_t at[VPL];  // where this lane's logit j goes
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const uint32_t in = __ballot_sync(0xffffffffu, v[j] >= least);
    at[j] = n + __popc(in & ((1u << lane) - 1u));
    n += __popc(in);
  }
  out_idx = -1;
  out_val = 0.0f;
  out_slot = lane;
  if (n <= 32) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (v[j] >= least) cand[at[j]] = static_cast<uint64_t>(__float_as_uint(v[j])) << 32 | static_cast<uint32_t>(lane * VPL + j);
    __syncwarp();
    // the key in the high half, the complement of the expert in the low half: one comparison orders both
    uint64_t mine = 0;
    if (lane < n) {
      const uint64_t c = cand[lane];
      mine = static_cast<uint64_t>(order_key(__uint_as_float(static_cast<uint32_t>(c >> 32)))) << 32 |
             static_cast<uint32_t>(~static_cast<uint32_t>(c));
    }
    if (lane <= n) cand[lane] = mine;  // and a 0 behind the last: the count below goes in pairs
    __syncwarp();
    int rank = 0;
    for (int i = 0; i < n; i += 2) {
      const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(cand + i);
      rank += c.x > mine;
      rank += c.y > mine;
    }
    if (lane < n) {
      out_slot = rank;
      if (rank < k) {
        out_val = key_value(static_cast<uint32_t>(mine >> 32));
        out_idx = static_cast<int>(~static_cast<uint32_t>(mine));
      }
    }
    __syncwarp();
    return;
  }
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) key[j] = v[j] >= least ? order_key(v[j]) : 0u;
  for (int s = 0; s < k; ++s) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) m = max(m, key[j]);
    const uint32_t best = __reduce_max_sync(0xffffffffu, m);
    if (best == 0u) break;
    const int w = __ffs(__ballot_sync(0xffffffffu, m == best)) - 1;
    int pos = -1;
    if (lane == w) {
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j)
        if (key[j] == best) pos = j;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j == pos) key[j] = 0;
    }
    pos = __shfl_sync(0xffffffffu, pos, w);
    if (lane == s) {
      out_idx = w * VPL + pos;
      out_val = key_value(best);
    }
  }
}

// The CTA's tokens [t0, t1): selection and weights to global memory; the per-expert
// selection counts (and at [E] the routed tokens) to hist, the sums of p to psum (per-warp
// slices, added in warp order). Ends with a CTA barrier. One warp per token.
template <int VPL, bool BF16>
DEVI void route_rows(const RouteArgs& a, int64_t t0, int64_t t1, int32_t* hist, float* psum, uint64_t* cand) {
  constexpr int WARPS = RouteCfg<VPL>::WARPS, THREADS = RouteCfg<VPL>::THREADS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  for (int e = threadIdx.x; e <= E; e += THREADS) hist[e] = 0;
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) acc[j] = 0.0f;
  int routed = 0;
  for (int64_t t = t0 + warp; t < t1; t += WARPS) {
    float v[VPL];
    float lane_max = __uint_as_float(0xFF800000u), mx = lane_max;
    bool on = false;
    if (!a.valid || __ldg(a.valid + t) != 0) {
      load_row<VPL, BF16>(a.logits, t, E, a.vec, lane, v);
#pragma unroll
      for (int j = 0; j < VPL; ++j) lane_max = fmaxf(lane_max, v[j]);
      mx = key_value(__reduce_max_sync(0xffffffffu, order_key(lane_max)));
      on = row_routed<VPL>(v, mx);
    }
    int my_idx = -1, my_slot = lane;
    float my_w = 0.0f;
    if (on) {
      float my_v;
      warp_top_k<VPL>(v, lane_max, k, cand + warp * kCandSlots, my_idx, my_v, my_slot);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        v[j] = ex2(route_arg(v[j], mx));
        sum += v[j];
      }
      const float inv = rcp(warp_sum(sum));
#pragma unroll
      for (int j = 0; j < VPL; ++j) acc[j] = fmaf(v[j], inv, acc[j]);
      ++routed;
      const float es = my_idx >= 0 ? ex2(route_arg(my_v, mx)) : 0.0f;
      // inv is at most 1, or NaN: then the renormalised weights are, whichever expert's logit it came from
      my_w = es * (a.renorm ? rcp(fmaf(inv, 0.0f, warp_sum(es))) : inv);
      if (my_idx >= 0) atomicAdd(&hist[my_idx], 1);
    }
    if (my_slot < k) {
      a.topk_idx[t * k + my_slot] = my_idx;
      a.topk_w[t * k + my_slot] = my_w;
    }
  }
  if (lane == 0) atomicAdd(&hist[E], routed);
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (lane * VPL + j < E) psum[warp * E + lane * VPL + j] = acc[j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += THREADS) {
    float s = 0.0f;
    for (int w = 0; w < WARPS; ++w) s += psum[w * E + e];
    psum[e] = s;
  }
  __syncthreads();
}

// Exclusive scan of counts[E] into offs[E + 1] (shared memory); all threads of the CTA.
DEVI void scan_counts(const int32_t* counts, int E, int32_t* offs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int c = e0 + lane < E ? counts[e0 + lane] : 0;
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      if (e0 + lane < E) offs[e0 + lane] = base + s - c;
      base += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) offs[E] = base;
  }
  __syncthreads();
}

// Rows of the CTA's tokens: base[e] (shared) is the first row of expert e that this CTA
// fills. Each warp owns a contiguous range of the (token, slot) pairs: its selections per expert
// are counted first, then 32 pairs at a time take their places: the pairs of one expert in the
// step find one another (match), and count the ones before them. wcnt: [WARPS][E] in shared
// memory.
template <int WARPS>
DEVI void place_rows(const RouteArgs& a, int64_t t0, int64_t t1, const int32_t* base, int32_t* wcnt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  for (int i = threadIdx.x; i < WARPS * E; i += 32 * WARPS) wcnt[i] = 0;
  __syncthreads();
  const int64_t per = ((t1 - t0) * k + WARPS - 1) / WARPS;
  const int64_t p0 = min(t1 * k, t0 * k + warp * per), p1 = min(t1 * k, p0 + per);
  int32_t* mine = wcnt + warp * E;
  for (int64_t i = p0 + lane; i < p1; i += 32) {
    const int e = a.topk_idx[i];
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 32 * WARPS) {
    int s = base[e];
    for (int w = 0; w < WARPS; ++w) {
      const int c = wcnt[w * E + e];
      wcnt[w * E + e] = s;
      s += c;
    }
  }
  __syncthreads();
  const uint32_t below = (1u << lane) - 1u;
  for (int64_t i0 = p0; i0 < p1; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < p1 ? a.topk_idx[i] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    int row = -1;
    if (e >= 0) row = mine[e] + __popc(same & below);
    __syncwarp();
    if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
    __syncwarp();
    if (e >= 0) a.row_token[row] = static_cast<int32_t>(i / k);
    if (i < p1) a.slot_row[i] = row;
  }
}

// Writes what one CTA writes for all: offsets and the balance loss (n routed tokens).
DEVI void finish_route(const RouteArgs& a, const int32_t* counts, const float* mean, int n, const int32_t* offs) {
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.expert_offsets[e] = offs[e];
  if (threadIdx.x < 32) {
    float s = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += 32) s += static_cast<float>(counts[e]) * mean[e];
    s = warp_sum(s);
    if (threadIdx.x == 0)
      a.loss[0] = n > 0 ? static_cast<float>(a.E) * s / (static_cast<float>(n) * static_cast<float>(a.k)) : 0.0f;
  }
}

DEVI void route_chunk(const RouteArgs& a, int64_t& t0, int64_t& t1) {
  const int64_t per = (a.T + gridDim.x - 1) / gridDim.x;
  t0 = min(a.T, static_cast<int64_t>(blockIdx.x) * per);
  t1 = min(a.T, t0 + per);
}

// Stage 1: every CTA routes its tokens; counts and sums of p per CTA to the workspace. 65,536 tokens x 256
// fp32, top-8: 36 us of the call's 47 (stages 2 and 3: 8.5 and 13 alone, cold, and partly under one
// another's launches). Bound by instruction issue (~410 a row, 68 % of the slots), not by its 67 MB
// (10 us): a warp is half idle only in the selection's exchanges, and requesting the next row ahead
// gained nothing.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(RouteCfg<VPL>::THREADS) k_moe_route(const RouteArgs a) {
  extern __shared__ __align__(16) uint64_t sh64[];
  uint64_t* cand = sh64;  // [WARPS][kCandSlots]
  int32_t* hist = reinterpret_cast<int32_t*>(cand + RouteCfg<VPL>::WARPS * kCandSlots);  // [E + 1]
  float* psum = reinterpret_cast<float*>(hist + a.E + 1);                          // [WARPS][E]
  griddep_launch_dependents();
  int64_t t0, t1;
  route_chunk(a, t0, t1);
  route_rows<VPL, BF16>(a, t0, t1, hist, psum, cand);
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x)
    a.ws_hist[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + e] = hist[e];
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.ws_psum[static_cast<int64_t>(blockIdx.x) * a.E + e] = psum[e];
}

// Stage 2: one CTA per 32 experts. ws_hist becomes each CTA's exclusive prefix; totals to
// counts, means of p to mean_prob. Warps own contiguous runs of the `blocks` rows (at most
// kScanRun each, all loaded at once). Reads what stage 1 wrote, which may still run when this kernel
// starts: plain loads behind the dependency wait.
constexpr int kScanWarps = 32;
constexpr int kScanRun = (kRouteBlocks + kScanWarps - 1) / kScanWarps;
__global__ void __launch_bounds__(kScanWarps * 32) k_moe_scan(const RouteArgs a, int blocks) {
  __shared__ int32_t part[kScanWarps][32];
  __shared__ float fpart[kScanWarps][32];
  __shared__ int32_t npart[kScanWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, e = blockIdx.x * 32 + lane;
  const int per = (blocks + kScanWarps - 1) / kScanWarps;
  const int b0 = min(blocks, warp * per), b1 = min(blocks, b0 + per);
  int32_t h[kScanRun];
  float s = 0.0f;
  int c = 0, n = 0;
#pragma unroll
  for (int i = 0; i < kScanRun; ++i) {
    h[i] = (e < E && b0 + i < b1) ? a.ws_hist[static_cast<int64_t>(b0 + i) * (E + 1) + e] : 0;
    if (e < E && b0 + i < b1) s += a.ws_psum[static_cast<int64_t>(b0 + i) * E + e];
    c += h[i];
  }
  if (b0 + lane < b1) n = a.ws_hist[static_cast<int64_t>(b0 + lane) * (E + 1) + E];
  n = __reduce_add_sync(0xffffffffu, n);
  part[warp][lane] = c;
  fpart[warp][lane] = s;
  if (lane == 0) npart[warp] = n;
  __syncthreads();
  int before = 0, total = 0;
  n = 0;
  s = 0.0f;
  for (int w = 0; w < kScanWarps; ++w) {
    const int v = part[w][lane];
    if (w < warp) before += v;
    total += v;
    s += fpart[w][lane];
    n += npart[w];
  }
  if (e < E) {
#pragma unroll
    for (int i = 0; i < kScanRun; ++i)
      if (b0 + i < b1) {
        a.ws_hist[static_cast<int64_t>(b0 + i) * (E + 1) + e] = before;
        before += h[i];
      }
    if (warp == 0) {
      a.counts[e] = total;
      a.mean_prob[e] = n > 0 ? s / static_cast<float>(n) : 0.0f;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.routed_tokens[0] = n;
}

// Stage 3: every CTA places its tokens' rows. Bound by the latency of its few dependent steps.
__global__ void __launch_bounds__(kPlaceThreads) k_moe_place(const RouteArgs a) {
  extern __shared__ int32_t sh[];
  int32_t* offs = sh;                // [E + 1]
  int32_t* base = offs + a.E + 1;    // [E]
  int32_t* wcnt = base + a.E;        // [kPlaceWarps][E]
  griddep_wait();
  scan_counts(a.counts, a.E, offs);
  for (int e = threadIdx.x; e < a.E; e += kPlaceThreads)
    base[e] = offs[e] + a.ws_hist[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + e];
  int64_t t0, t1;
  route_chunk(a, t0, t1);
  place_rows<kPlaceWarps>(a, t0, t1, base, wcnt);
  // rows that no selection fills
  for (int64_t r = offs[a.E] + static_cast<int64_t>(blockIdx.x) * kPlaceThreads + threadIdx.x; r < a.T * a.k;
       r += static_cast<int64_t>(gridDim.x) * kPlaceThreads)
    a.row_token[r] = -1;
  if (blockIdx.x == 0) finish_route(a, a.counts, a.mean_prob, a.routed_tokens[0], offs);
}

// All stages in one CTA, for few tokens: no workspace, one launch.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(RouteCfg<VPL>::THREADS) k_moe_route_one(const RouteArgs a) {
  constexpr int WARPS = RouteCfg<VPL>::WARPS;
  extern __shared__ __align__(16) uint64_t sh64[];
  uint64_t* cand = sh64;                                      // [WARPS][kCandSlots]
  int32_t* hist = reinterpret_cast<int32_t*>(cand + WARPS * kCandSlots);  // [E + 1]
  int32_t* offs = hist + a.E + 1;                             // [E + 1]
  float* psum = reinterpret_cast<float*>(offs + a.E + 1);     // [WARPS][E], then the means
  route_rows<VPL, BF16>(a, 0, a.T, hist, psum, cand);
  scan_counts(hist, a.E, offs);
  const int n = hist[a.E];
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    psum[e] = n > 0 ? psum[e] / static_cast<float>(n) : 0.0f;
    a.mean_prob[e] = psum[e];
    a.counts[e] = hist[e];
  }
  if (threadIdx.x == 0) a.routed_tokens[0] = n;
  __syncthreads();
  finish_route(a, hist, psum, n, offs);
  for (int64_t r = offs[a.E] + threadIdx.x; r < a.T * a.k; r += blockDim.x) a.row_token[r] = -1;
  __syncthreads();  // psum's memory is reused
  place_rows<WARPS>(a, 0, a.T, offs, reinterpret_cast<int32_t*>(psum));
}

// ---- gradient of the logits ------------------------------------------------------------------
//
// G_te = dL E c_e / (k n^2) from the balance loss (its counts carry no gradient): d l_te gets
// p_te (G_te - sum_i p_ti G_ti). The weights' gradients dw_ts add at the selected experts
// w_s dw_s and, when the weights are plain probabilities, -p_te sum_s w_s dw_s everywhere (it joins
// the sum above); renormalised weights are a softmax over the selected logits alone, which add
// w_s (dw_s - sum_r w_r dw_r) there. Unrouted tokens get zeros.
//
// Bound by memory and its latency: 65,536 x 256 fp32 in 29 us (its 140 MB: 21 us). With a.vec the rows
// come by cp.async, kBwdAhead rows ahead of their use (each lane copies and reads back its own bytes,
// so no lane waits for another); with plain loads 39 us. Four CTAs on an SM (64 registers) take 1 us
// less than three.
constexpr int kBwdThreads = 256;
constexpr int kBwdWarps = kBwdThreads / 32;
constexpr int kBwdAhead = 4;
// Whether a lane's share of a row is whole 16-byte pieces, and a ring of rows fits beside others.
template <int VPL, bool BF16>
constexpr bool kBwdRing = VPL <= 8 && VPL * (BF16 ? 2 : 4) % 16 == 0;
__host__ __device__ constexpr int bwd_slot_bytes(int vpl, bool bf16) {  // logits, then selection, dw, w
  return 32 * vpl * (bf16 ? 2 : 4) + 3 * 128;
}
template <int VPL, bool BF16>
__global__ void __launch_bounds__(kBwdThreads, VPL <= 8 ? 4 : 1) k_moe_route_bwd(const RouteBwdArgs a) {
  extern __shared__ __align__(16) float shf[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  float* spot = shf + warp * (32 * VPL);  // this warp's sparse part of the row, zero between rows
#pragma unroll
  for (int j = 0; j < VPL; ++j) spot[lane * VPL + j] = 0.0f;
  __syncwarp();
  constexpr int SLOT = bwd_slot_bytes(VPL, BF16), LANE_BYTES = VPL * (BF16 ? 2 : 4);
  uint8_t* ring = reinterpret_cast<uint8_t*>(shf + kBwdWarps * 32 * VPL) + warp * kBwdAhead * SLOT;
  const float n = static_cast<float>(a.routed_tokens[0]);
  const float scale = (a.d_loss && n > 0.0f) ? __ldg(a.d_loss) * static_cast<float>(E) / (static_cast<float>(k) * n * n) : 0.0f;
  float g[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane * VPL + j;
    g[j] = e < E ? scale * static_cast<float>(__ldg(a.counts + e)) : 0.0f;
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kBwdWarps;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kBwdWarps + warp;
  const bool ringed = kBwdRing<VPL, BF16> && a.vec;
  auto request = [&](int64_t t, int slot) {
    if constexpr (kBwdRing<VPL, BF16>) {
      if (t < a.T) {
        uint8_t* d = ring + slot * SLOT;
        const uint8_t* src = static_cast<const uint8_t*>(a.logits) + t * (32 * LANE_BYTES) + lane * LANE_BYTES;
#pragma unroll
        for (int i = 0; i < LANE_BYTES; i += 16) cp_async16(d + lane * LANE_BYTES + i, src + i);
        if (a.d_w && lane < k) {
          uint8_t* x = d + 32 * LANE_BYTES + lane * 4;
          cp_async4(x, a.topk_idx + t * k + lane);
          cp_async4(x + 128, a.d_w + t * k + lane);
          cp_async4(x + 256, a.topk_w + t * k + lane);
        }
      }
      cp_async_commit();
    }
  };
  if (ringed)
    for (int i = 0; i < kBwdAhead - 1; ++i) request(first + i * stride, i);
  int slot = 0;
  for (int64_t t = first; t < a.T; t += stride) {
    float v[VPL], d[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) d[j] = 0.0f;
    float mx = __uint_as_float(0xFF800000u), slot_dw = 0.0f, slot_w = 0.0f;
    int slot_idx = -1;
    const bool valid = !a.valid || __ldg(a.valid + t) != 0;
    bool on = false;
    if (ringed) {
      if constexpr (kBwdRing<VPL, BF16>) {
        request(t + (kBwdAhead - 1) * stride, (slot + kBwdAhead - 1) & (kBwdAhead - 1));
        cp_async_wait<kBwdAhead - 1>();
        const uint8_t* r = ring + slot * SLOT;
#pragma unroll
        for (int i = 0; i < LANE_BYTES; i += 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(r + lane * LANE_BYTES + i);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (BF16)
              v[i / 2 + 2 * j] = bf16lo(u[j]), v[i / 2 + 2 * j + 1] = bf16hi(u[j]);
            else
              v[i / 4 + j] = __uint_as_float(u[j]);
          }
        }
        if (a.d_w && lane < k) {
          const uint8_t* x = r + 32 * LANE_BYTES + lane * 4;
          slot_idx = *reinterpret_cast<const int32_t*>(x);
          slot_dw = *reinterpret_cast<const float*>(x + 128);
          slot_w = *reinterpret_cast<const float*>(x + 256);
        }
        slot = (slot + 1) & (kBwdAhead - 1);
      }
    } else {
      if (valid) load_row<VPL, BF16>(a.logits, t, E, a.vec, lane, v);
      if (a.d_w && lane < k) {
        slot_idx = __ldg(a.topk_idx + t * k + lane);
        slot_dw = __ldg(a.d_w + t * k + lane);
        slot_w = __ldg(a.topk_w + t * k + lane);
      }
    }
    if (valid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) mx = fmaxf(mx, v[j]);
      mx = key_value(__reduce_max_sync(0xffffffffu, order_key(mx)));
      on = row_routed<VPL>(v, mx);
    }
    if (on) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        v[j] = ex2((v[j] - mx) * kLog2E);
        sum += v[j];
      }
      const float inv = rcp(warp_sum(sum));
      int idx = -1;
      float dot = 0.0f;
      if (a.d_w) {
        if (slot_idx >= 0 && slot_idx < E) idx = slot_idx;
        float add = idx >= 0 ? slot_w * slot_dw : 0.0f;
        if (a.renorm)
          add -= (idx >= 0 ? slot_w : 0.0f) * warp_sum(add);
        else
          dot = add;
        if (idx >= 0) spot[idx] = add;
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        v[j] *= inv;
        dot = fmaf(v[j], g[j], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = fmaf(v[j], g[j] - dot, spot[lane * VPL + j]);
      __syncwarp();
      if (idx >= 0) spot[idx] = 0.0f;
      __syncwarp();
    }
    if (a.vec) {
      if (BF16) {
        uint16_t* o = static_cast<uint16_t*>(a.d_logits) + t * E + lane * VPL;
        if constexpr (VPL >= 8) {
#pragma unroll
          for (int j = 0; j < VPL; j += 8)
            *reinterpret_cast<uint4*>(o + j) = make_uint4(pack_bf16x2(d[j], d[j + 1]), pack_bf16x2(d[j + 2], d[j + 3]),
                                                          pack_bf16x2(d[j + 4], d[j + 5]), pack_bf16x2(d[j + 6], d[j + 7]));
        } else if constexpr (VPL >= 2) {
#pragma unroll
          for (int j = 0; j < VPL; j += 2) *reinterpret_cast<uint32_t*>(o + j) = pack_bf16x2(d[j], d[j + 1]);
        } else {
          o[0] = static_cast<uint16_t>(pack_bf16x2(d[0], 0.0f) & 0xFFFFu);
        }
      } else {
        float* o = static_cast<float*>(a.d_logits) + t * E + lane * VPL;
        if constexpr (VPL >= 4) {
#pragma unroll
          for (int j = 0; j < VPL; j += 4) *reinterpret_cast<float4*>(o + j) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < VPL; ++j) o[j] = d[j];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int e = lane * VPL + j;
        if (e < E) {
          if (BF16)
            static_cast<uint16_t*>(a.d_logits)[t * E + e] = static_cast<uint16_t>(pack_bf16x2(d[j], 0.0f) & 0xFFFFu);
          else
            static_cast<float*>(a.d_logits)[t * E + e] = d[j];
        }
      }
    }
  }
}

// ---- host launchers ----------------------------------------------------------------------------

// Values per lane: the smallest power of two that covers E (E <= 1024).
static int route_vpl(int E) {
  int v = 1;
  while (v * 32 < E) v <<= 1;
  return v;
}

static bool route_vec(const void* p, int E, int bf16) {
  const int v = route_vpl(E);
  const int lane_bytes = v * (bf16 ? 2 : 4) < 16 ? v * (bf16 ? 2 : 4) : 16;
  return E == 32 * v && reinterpret_cast<uintptr_t>(p) % lane_bytes == 0;
}

#define ROUTE_DISPATCH(call)                                      \
  switch (route_vpl(a.E) * 2 + (a.bf16 ? 1 : 0)) {                \
    case 2: call(1, false); break;                                \
    case 3: call(1, true); break;                                 \
    case 4: call(2, false); break;                                \
    case 5: call(2, true); break;                                 \
    case 8: call(4, false); break;                                \
    case 9: call(4, true); break;                                 \
    case 16: call(8, false); break;                               \
    case 17: call(8, true); break;                                \
    case 32: call(16, false); break;                              \
    case 33: call(16, true); break;                               \
    case 64: call(32, false); break;                              \
    default: call(32, true); break;                               \
  }

// Tokens up to which one CTA does all the stages in one launch. One CTA / three kernels, us:
//   tokens          16          32          48          64          96
//   8 experts    4.1 /  9.7  5.0 /  9.7  5.9 /  9.7  6.8 /  9.6  8.5 /  9.5
//   64           4.6 / 10.2  6.1 / 10.1  7.0 /  9.6  8.1 /  9.7 10.8 /  9.9
//   256          5.8 / 11.1  7.5 / 10.8  9.0 / 10.9 10.5 / 10.8 13.9 / 11.2
//   1024        18.4 / 20.4 23.8 / 19.9
static int route_one_tokens(int E) { return route_vpl(E) <= 8 ? 64 : 16; }

static int route_warps(int E) { return route_vpl(E) <= 8 ? 16 : 8; }

int route_blocks(int64_t T, int E) {
  const int64_t b = (T + route_warps(E) - 1) / route_warps(E);
  return static_cast<int>(b < kRouteBlocks ? b : kRouteBlocks);
}

cudaError_t launch_moe_route(RouteArgs a, cudaStream_t st, int* launches) {
  a.vec = route_vec(a.logits, a.E, a.bf16);
  const int E = a.E, warps = route_warps(E), threads = 32 * warps;
  if (a.T <= route_one_tokens(E)) {
    const int smem = warps * kCandSlots * 8 + (2 * (E + 1) + warps * E) * 4;
    *launches = 1;
#define CALL(V, B) k_moe_route_one<V, B><<<1, threads, smem, st>>>(a)
    ROUTE_DISPATCH(CALL)
#undef CALL
    return cudaGetLastError();
  }
  const int blocks = route_blocks(a.T, E);
  const int smem = warps * kCandSlots * 8 + (E + 1 + warps * E) * 4;
  *launches = 3;
#define CALL(V, B) k_moe_route<V, B><<<blocks, threads, smem, st>>>(a)
  ROUTE_DISPATCH(CALL)
#undef CALL
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the later stages' launches overlap the stage before; each waits for it before reading
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((E + 31) / 32);
  cfg.blockDim = dim3(kScanWarps * 32);
  e = cudaLaunchKernelEx(&cfg, k_moe_scan, a, blocks);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kPlaceThreads);
  cfg.dynamicSmemBytes = (2 * E + 1 + kPlaceWarps * E) * 4;
  return cudaLaunchKernelEx(&cfg, k_moe_place, a);
}

cudaError_t launch_moe_route_bwd(RouteBwdArgs a, int sms, cudaStream_t st) {
  a.vec = route_vec(a.logits, a.E, a.bf16) && route_vec(a.d_logits, a.E, a.bf16);
  const int64_t want = (a.T + kBwdWarps - 1) / kBwdWarps;
  const int grid = static_cast<int>(want < 8 * sms ? want : 8 * sms);
  const int vpl = route_vpl(a.E);
  const bool ring = a.vec && vpl <= 8 && vpl * (a.bf16 ? 2 : 4) % 16 == 0;
  const int smem = kBwdWarps * (32 * vpl * 4 + (ring ? kBwdAhead * bwd_slot_bytes(vpl, a.bf16 != 0) : 0));
#define CALL(V, B)                                                                              \
  {                                                                                             \
    const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(k_moe_route_bwd<V, B>)); \
    if (e != cudaSuccess) return e;                                                             \
    k_moe_route_bwd<V, B><<<grid, kBwdThreads, smem, st>>>(a);                                  \
  }
  ROUTE_DISPATCH(CALL)
#undef CALL
  return cudaGetLastError();
}

}  // namespace nvfp4

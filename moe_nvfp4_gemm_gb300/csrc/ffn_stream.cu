// Forward pass of the 16-bit gated feed-forward block for few tokens: h = act(x Wg^T) * (x Wu^T). The same sums as
// ffn_tile.cu with the operands exchanged: 64 gate and 64 up rows on the MMA's 128-lane side, the tokens
// (padded to 16) on its N side, so that no token is padded to a tile of 256.
//
// Bound by reading the weights, each once, in 64-column blocks by TMA; the tokens come from L2. A CTA
// takes one tile of 64 columns of h. Two CTAs share an SM, so that all tiles of a layer of up to 19,456 columns are in
// flight at once and the uneven rest of a division by 152 costs nothing: an SM with two tiles draws twice the bandwidth. The tensor core sums all of K in TMEM; the four epilogue warps put
// the sums into shared memory, where gate and up of a column, which lie in different lanes, meet.
// One token of 14,336 x 8,192: 72 us, 6.5 TB/s; 128 tokens 78.
// Few tiles: S CTAs of a cluster sum a part of K each, and each reads all parts' sums of its share of the tokens
// through distributed shared memory.
#include <stdint.h>

#include "ffn.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

template <int NT>
struct FfnStreamCfg {
  // warps 0-3: weights' producer, MMA issuer, tokens' producer, idle; warps 4-7: epilogue
  static constexpr int THREADS = 256;
  static constexpr int CTAS = 2;  // per SM
  static constexpr int W_BYTES = 128 * 128, X_BYTES = NT * 128;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int STAGES = (113 * 1024 - 1024 - 512) / STAGE_BYTES;
  static_assert(STAGES * STAGE_BYTES >= NT * 512, "the sums take the ring's place");
};

template <int NT, bool HALF>
__global__ void __launch_bounds__(FfnStreamCfg<NT>::THREADS, FfnStreamCfg<NT>::CTAS)
    k_ffn_stream(const __grid_constant__ FfnStreamMaps maps, const __grid_constant__ FfnStreamArgs p) {
  using C = FfnStreamCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int STAGES = C::STAGES;
  // the sums, [token][128], take the ring's place (every stage has been consumed by then)
  float* sums = reinterpret_cast<float*>(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;  // all sums are complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  const int M = p.M, S = p.split;
  const int tile = blockIdx.x / S, rank = static_cast<int>(blockIdx.x) - tile * S;
  const int n0 = tile * 64;
  const int m_own = (M + S - 1) / S;  // tokens per owner
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / S);
  const int mine = min(m_own, M - rank * m_own);
  if (threadIdx.x == 0) {
    prefetch_tmap(&maps.w[0]);
    prefetch_tmap(&maps.w[1]);
    prefetch_tmap(&maps.x);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);  // the weight warp and the token warp
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // this CTA's first weight blocks into L2 while the previous kernel may still run
    for (int kb = kb0; kb < min(kb1, kb0 + p.l2_prefetch); ++kb) {
      tma_prefetch_2d(&maps.w[0], kb * 64, n0);
      tma_prefetch_2d(&maps.w[1], kb * 64, n0);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, NT);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp >= 4) {
    const int q = warp & 3;
    const bool ok = mbar_wait_warp(done, 0, abort_flag, wd);
    tc_fence_after();
    // lane: weight row 32 q + lane; columns: tokens
#pragma unroll
    for (int c = 0; c < NT / 32; ++c) {
      if (c * 32 >= M || !ok) break;
      uint32_t r[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 32, r);
      tmem_ld_wait32(r);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int t = c * 32 + j;
        if (t < M) sums[t * 128 + q * 32 + lane] = __uint_as_float(r[j]);
      }
    }
  } else if (warp == 0 || warp == 2) {
    // warp 0 requests every stage's weight rows, warp 2 its token rows
    const uint64_t pol = warp == 0 ? policy_evict_first() : policy_evict_last();
    const int boxes = (M + 31) >> 5;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    uint32_t used = 0, phases = 0;  // per stage: requested at all, phase of the last request
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(&empty[s], ph ^ 1, abort_flag, wd)) break;
      uint8_t* st = smem + s * C::STAGE_BYTES;
      if (warp == 0) {
        // test hook: the first CTA withholds a stage's expect-tx arrival and weight loads
        const bool withheld = blockIdx.x == 0 && ++issued == p.drop_stage;
        if (!withheld && elect_one()) {
          mbar_arrive_expect_tx(&full[s], C::W_BYTES);
          tma_load_2d(st, &maps.w[0], &full[s], kb * 64, n0, pol);
          tma_load_2d(st + C::W_BYTES / 2, &maps.w[1], &full[s], kb * 64, n0, pol);
        }
      } else if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], boxes * 4096);
        for (int j = 0; j < boxes; ++j)
          tma_load_2d(st + C::W_BYTES + j * 4096, &maps.x, &full[s], kb * 64, j * 32, pol);
      }
      __syncwarp();
      used |= 1u << s;
      phases = (phases & ~(1u << s)) | ph << s;
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    if (warp == 0) griddep_launch_dependents();
    // this warp's copies in flight land before the CTA leaves
    for (int j = 0; j < STAGES; ++j)
      if (used >> j & 1) {
        volatile int32_t dummy = 0;
        mbar_wait_warp(&full[j], phases >> j & 1, &dummy, wd);
      }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16(128, ((M + 15) >> 4) * 16, !HALF);
    int s = 0;
    uint32_t ph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(&full[s], ph, abort_flag, wd)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t addr = smem_u32(smem + s * C::STAGE_BYTES);
        const uint64_t wdesc = desc_sw128(addr), xdesc = desc_sw128(addr + C::W_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) tc_mma_f16(tmem, wdesc + 2 * kk, xdesc + 2 * kk, idesc, kb != kb0 || kk != 0);
        tc_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    // also after an abort: completes when all MMAs issued so far are done
    if (elect_one()) tc_commit(done);
    __syncwarp();
    volatile int32_t dummy = 0;
    mbar_wait_warp(done, 0, &dummy, wd);
  }

  tc_fence_before();
  __syncwarp();
  // all sums are in place; also after an abort, so that the cluster's barriers pair
  if (S > 1)
    cluster_sync();
  else
    __syncthreads();
  if (!*abort_flag) {
    // A thread: two columns of h; a warp: every eighth token, two of them at a time with all parts' sums in flight,
    // added in the order of K.
    const int c = n0 + 2 * lane;
    const bool stored = c < p.N;  // N is even
    uint32_t from[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) from[s] = mapa_shared(smem_u32(sums) + rank * m_own * 512 + lane * 8, min(s, S - 1));
#pragma unroll 1
    for (int i0 = warp; i0 < mine; i0 += 16) {
      float2 g[2][8], u[2][8];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < S) {
            // (a token past the last is read as the last and not stored)
            const uint32_t at = from[s] + min(i0 + 8 * j, mine - 1) * 512;
            g[j][s] = ld_shared_cluster_v2(at);
            u[j][s] = ld_shared_cluster_v2(at + 256);
          }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int s = 1; s < 8; ++s)
          if (s < S) {
            g[j][0].x += g[j][s].x, g[j][0].y += g[j][s].y;
            u[j][0].x += u[j][s].x, u[j][0].y += u[j][s].y;
          }
        const float2 gs = g[j][0], us = u[j][0];
        if (i0 + 8 * j < mine && stored) {
          const int64_t t = rank * m_own + i0 + 8 * j;
          *reinterpret_cast<uint32_t*>(p.h + t * p.ldh + c) = pack16<HALF>(ffn_act(gs.x, p.act) * us.x, ffn_act(gs.y, p.act) * us.y);
          if (p.gate) {
            *reinterpret_cast<float2*>(p.gate + t * p.N + c) = gs;
            *reinterpret_cast<float2*>(p.up + t * p.N + c) = us;
          }
        }
      }
    }
  }
  if (S > 1) cluster_sync();  // no CTA leaves while another may still read its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NT);
  }
  if (threadIdx.x == 0 && *abort_flag) report_status(p.status, kStatusTimeout);
}

template <int NT, bool HALF>
cudaError_t launch_stream(const FfnStreamMaps& maps, const FfnStreamArgs& p, cudaStream_t st) {
  using C = FfnStreamCfg<NT>;
  auto kernel = k_ffn_stream<NT, HALF>;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + 63) / 64 * p.split));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::STAGES * C::STAGE_BYTES + 1024 + 512;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_ffn_stream(const FfnStreamMaps& maps, const FfnStreamArgs& p, cudaStream_t st) {
  if (p.M <= 32) return p.half ? launch_stream<32, true>(maps, p, st) : launch_stream<32, false>(maps, p, st);
  if (p.M <= 64) return p.half ? launch_stream<64, true>(maps, p, st) : launch_stream<64, false>(maps, p, st);
  return p.half ? launch_stream<128, true>(maps, p, st) : launch_stream<128, false>(maps, p, st);
}

}  // namespace nvfp4

// Forward pass of the 16-bit gated feed-forward block for few tokens: h = act(x Wg^T) * (x Wu^T). The same sums as
// ffn_tile.cu with the operands exchanged: 64 gate and 64 up rows on the MMA's 128-lane side, the tokens
// (padded to 16) on its N side, so that no token is padded to a tile of 256.
//
// Bound by reading the weights, each once, in 64-column blocks by TMA; the tokens come from L2. A CTA
// takes one tile of 64 columns of h (with up to 64 tokens two CTAs share an SM, so that all tiles of a
// layer of 19,456 are in flight at once and the uneven rest of a division by 152 costs nothing: an SM
// with two tiles draws twice the bandwidth). The tensor core sums all of K in TMEM; the four epilogue warps put
// the sums into shared memory, where gate and up of a column, which lie in different lanes, meet.
// Few tiles: S CTAs of a cluster sum a part of K each, and each receives all parts' sums of its share of the
// tokens through distributed shared memory.
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
  static constexpr int MAX_STAGES = 8;
  static constexpr int ROOM = 113 * 1024 - 1024 - 512;
};

template <int NT, bool HALF>
__global__ void __launch_bounds__(FfnStreamCfg<NT>::THREADS, FfnStreamCfg<NT>::CTAS)
    k_ffn_stream(const __grid_constant__ FfnStreamMaps maps, const __grid_constant__ FfnStreamArgs p) {
  using C = FfnStreamCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int STAGES = p.stages;
  // sums leave from the ring, [token][128] (every stage has been consumed by then); with S > 1 they arrive in
  // recv [source rank][own token][128]
  float* part = reinterpret_cast<float*>(smem);
  float* recv = reinterpret_cast<float*>(smem + p.recv_at);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.bars_at);
  uint64_t* empty = full + C::MAX_STAGES;
  uint64_t* done = empty + C::MAX_STAGES;  // all sums are complete
  uint64_t* red_bar = done + 1;            // all S partials of this CTA's tokens have landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(red_bar + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  // items: the token tiles of a weight tile one after the other, which share its bytes in L2; then the parts of K
  const int S = p.split;
  const int item = blockIdx.x / S, rank = static_cast<int>(blockIdx.x) - item * S;
  const int m0 = item % p.mt * NT, n0 = item / p.mt * 64;
  const int M = min(NT, p.M - m0);    // tokens of this tile
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
    mbar_init(red_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (S > 1 && mine > 0) mbar_arrive_expect_tx(red_bar, static_cast<uint32_t>(S * mine * 512));
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
  // every CTA's reduction barrier exists before any CTA of the cluster sends (the sender waits)
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
        if (t < M) part[t * 128 + q * 32 + lane] = __uint_as_float(r[j]);
      }
    }
    const float* src = part;
    bool received = ok;
    if (S > 1) {
      // Every CTA sends owner o the block of o's tokens, the owners add their S slots in rank order. Every CTA
      // sends, also after an abort, and each owner waits for all (bounded), so that no CTA leaves while a copy
      // into its shared memory is in flight.
      fence_proxy_async_shared();
      named_sync(1, 128);
      if (warp == 4) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (lane == 0) {
          for (int o = 0; o < S; ++o) {
            const int n_o = min(m_own, M - o * m_own);
            if (n_o <= 0) continue;
            bulk_copy_to_cluster(mapa_shared(smem_u32(recv + rank * m_own * 128), o), part + o * m_own * 128,
                                 static_cast<uint32_t>(n_o * 512), mapa_shared(smem_u32(red_bar), o));
          }
          bulk_commit_group();
          bulk_wait_group_read0();
        }
        __syncwarp();
      }
      volatile int32_t no_abort = 0;
      received = mine > 0 && mbar_wait_warp(red_bar, 0, &no_abort, 4 * wd);
      if (mine > 0 && !received) *abort_flag = 1;
      src = recv;
    } else {
      named_sync(1, 128);
    }
    if (received && !*abort_flag) {
      // a thread: two columns of h; a warp: every fourth token, four of them at a time
      const int c = n0 + 2 * lane;
      const bool stored = c < p.N;  // N is even
#pragma unroll 1
      for (int i0 = q; i0 < mine; i0 += 16) {
        float2 g[4], u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = u[j] = make_float2(0.0f, 0.0f);
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (a token past the last is read as the last and not stored)
            const float* row = src + (s * m_own + min(i0 + 4 * j, mine - 1)) * 128 + 2 * lane;
            const float2 a = *reinterpret_cast<const float2*>(row), b = *reinterpret_cast<const float2*>(row + 64);
            g[j].x += a.x, g[j].y += a.y, u[j].x += b.x, u[j].y += b.y;
          }
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = pack16<HALF>(ffn_act(g[j].x, p.act) * u[j].x, ffn_act(g[j].y, p.act) * u[j].y);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t t = m0 + rank * m_own + i0 + 4 * j;
          if (i0 + 4 * j < mine && stored) {
            *reinterpret_cast<uint32_t*>(p.h + t * p.ldh + c) = h[j];
            if (p.gate) {
              *reinterpret_cast<uint32_t*>(p.gate + t * p.N + c) = pack16<HALF>(g[j].x, g[j].y);
              *reinterpret_cast<uint32_t*>(p.up + t * p.N + c) = pack16<HALF>(u[j].x, u[j].y);
            }
          }
        }
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
          tma_load_2d(st + C::W_BYTES + j * 4096, &maps.x, &full[s], kb * 64, m0 + j * 32, pol);
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

  // every thread that arrived on the cluster barrier also waits on it (the sending warp already did)
  if (S > 1 && warp != 4) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NT);
  }
  if (threadIdx.x == 0 && *abort_flag) report_status(p.status, kStatusTimeout);
}

template <int NT, bool HALF>
cudaError_t launch_stream(const FfnStreamMaps& maps, FfnStreamArgs p, cudaStream_t st) {
  using C = FfnStreamCfg<NT>;
  auto kernel = k_ffn_stream<NT, HALF>;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  const int most = p.M < NT ? p.M : NT, m_own = (most + p.split - 1) / p.split;
  const int recv_bytes = p.split > 1 ? p.split * m_own * 512 : 0;  // at most (NT + 7) * 512: split <= 8
  int stages = (C::ROOM - recv_bytes) / C::STAGE_BYTES;
  if (stages > C::MAX_STAGES) stages = C::MAX_STAGES;
  static_assert(C::ROOM - NT * 512 - 1024 > 2 * C::STAGE_BYTES && 2 * C::STAGE_BYTES >= NT * 512,
                "room for two stages beside the partial sums, which hold all tokens' sums");
  p.stages = stages;
  p.recv_at = stages * C::STAGE_BYTES;
  p.bars_at = p.recv_at + recv_bytes;
  cudaLaunchConfig_t cfg = {};
  p.mt = (p.M + NT - 1) / NT;
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + 63) / 64 * p.mt * p.split));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = p.bars_at + 1024 + 512;
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
  return p.half ? launch_stream<64, true>(maps, p, st) : launch_stream<64, false>(maps, p, st);
}

}  // namespace nvfp4

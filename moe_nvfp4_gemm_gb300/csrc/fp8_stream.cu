// FP8 block-scaled GEMM for few rows per weight: decode-size dense layers and small grouped (MoE)
// products. Same sums as fp8_gemm.cu, with the operands exchanged: 128 weight rows on the MMA's
// 128-lane side, the tokens (padded to 16) on its N side, so that no token is padded to a tile.
//
// Bound by reading the weights: one 128-row x 128-byte TMA tile per block of K, each read once,
// the tokens from L2. The tensor core sums one block of 128 into one of several TMEM buffers; the
// epilogue warps add it, times the token scales (put into shared memory by a warp of their own, the
// weight block's scale multiplied in), to fp32 sums in registers.
//   dense:   grid = (N / 128) x S CTAs in clusters of S along K; the S partial sums meet through
//            distributed shared memory, each CTA owning some of the tokens.
//   grouped: a persistent grid walks (token tile, weight tile) items of the device-built list; for
//            problems whose items are all resident at once (fp8_narrow.cu has the larger ones).
// Data that the previous kernel may have written is read with plain loads (see fp8_gemm.cu).
#include <stdint.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

enum { kFp8Dense = 0, kFp8DenseRowScale = 1, kFp8Grouped = 2 };

// NT: token columns of the accumulator (and rows of the token tile).
template <int NT>
struct Fp8StreamCfg {
  static constexpr int COLS = 32;  // token columns per epilogue warp
  static constexpr int EPI_WARPS = 4 * (NT / COLS);
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int CTAS = NT == 32 ? 2 : 1;  // per SM (two of NT = 64 would leave 80 registers: spills)
  static constexpr int BUFS = 4;
  static constexpr int TMEM_COLS = BUFS * NT;
  static constexpr int STAGE_BYTES = 16384 + NT * 128;
  // Scales of GROUPS x GROUP blocks of K: per block NT token scales (times the weight block's) and,
  // with a scale per weight row, 128 of those.
  static constexpr int GROUP = 8, GROUPS = 4;
  __host__ __device__ static constexpr int slot_floats(int mode) { return mode == 1 ? NT + 128 : NT; }
  __host__ __device__ static constexpr int scale_bytes(int mode) { return GROUPS * GROUP * slot_floats(mode) * 4; }
};

struct Fp8Item {
  int wt, e, row0, rows, kb0, kb1;
};

template <int NT, int MODE>
DEVI bool fp8_item(const Fp8GemmArgs& p, int i, int n_items, int NTW, int KB, Fp8Item& it) {
  if (i >= n_items) return false;
  if (MODE == kFp8Grouped) {
    const int4 d = p.tiles[i / NTW];
    it.wt = i % NTW;
    it.e = d.x;
    it.row0 = d.y;
    it.rows = d.z;
    it.kb0 = 0;
    it.kb1 = KB;
  } else {
    it.wt = i / p.split;
    it.e = 0;
    it.row0 = 0;
    it.rows = static_cast<int>(p.M);
    const int sp = i % p.split;
    it.kb0 = static_cast<int>(static_cast<int64_t>(KB) * sp / p.split);
    it.kb1 = static_cast<int>(static_cast<int64_t>(KB) * (sp + 1) / p.split);
  }
  return true;
}

template <int NT, int MODE>
__global__ void __launch_bounds__(Fp8StreamCfg<NT>::THREADS, Fp8StreamCfg<NT>::CTAS)
    k_fp8_stream(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const __grid_constant__ Fp8GemmArgs p) {
  using C = Fp8StreamCfg<NT>;
  constexpr bool GROUPED = MODE == kFp8Grouped;
  constexpr int BUFS = C::BUFS;
  constexpr int MAX_STAGES = 12;
  constexpr int SCALE_BYTES = C::scale_bytes(MODE), SLOT = C::slot_floats(MODE);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int STAGES = p.stages;
  float* scale_buf = reinterpret_cast<float*>(smem + STAGES * C::STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES + SCALE_BYTES);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* tfull = empty + MAX_STAGES;  // [BUFS]
  uint64_t* tempty = tfull + BUFS;       // [BUFS]
  uint64_t* drain = tempty + BUFS;
  uint64_t* red_bar = drain + 1;  // all S partials of this CTA's tokens have landed
  uint64_t* sfull = red_bar + 1;         // [GROUPS] a group's scales are in shared memory
  uint64_t* sempty = sfull + C::GROUPS;  // [GROUPS] and have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + C::GROUPS);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  // split-K: partial sums leave from the ring ([token][128] fp32; every stage has been consumed
  // by then) and arrive in recv [source rank][own token][128]
  float* part = reinterpret_cast<float*>(smem);
  float* recv = reinterpret_cast<float*>(smem + STAGES * C::STAGE_BYTES + SCALE_BYTES + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N);
  const int NTW = (N + 127) / 128;
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int S = GROUPED ? 1 : p.split;
  const int m_own = (M + S - 1) / S;  // split-K: tokens per owner
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);  // the weight warp and the token warp
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::EPI_WARPS);
    }
    for (int g = 0; g < C::GROUPS; ++g) {
      mbar_init(&sfull[g], 1);
      mbar_init(&sempty[g], C::EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(red_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (S > 1) {
      const int mine = min(m_own, M - static_cast<int>(cluster_ctarank()) * m_own);
      if (mine > 0) mbar_arrive_expect_tx(red_bar, static_cast<uint32_t>(S * mine * 512));
    }
    if (!GROUPED) {
      // this CTA's first weight blocks into L2 while the previous kernel may still run
      Fp8Item it;
      fp8_item<NT, MODE>(p, blockIdx.x, NTW * S, NTW, KB, it);
      for (int kb = it.kb0; kb < min(it.kb1, it.kb0 + p.l2_prefetch); ++kb) tma_prefetch_2d(&tmW, kb * 128, it.wt * 128);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // every CTA's reduction barrier exists before any CTA of the cluster sends (the sender waits)
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  griddep_wait();
  const int n_items = GROUPED ? p.n_tiles[0] * NTW : NTW * S;
  const int first = blockIdx.x, stride = GROUPED ? gridDim.x : n_items;

  if (warp >= 4) {
    const int q = warp & 3, h = (warp - 4) >> 2;
    constexpr int COLS = C::COLS;
    int buf = 0, grp = 0;
    uint32_t bph = 0, gph = 0;
    bool ok = true;
    uint64_t acc[COLS / 2];
    Fp8Item it;
    for (int i = first; ok && fp8_item<NT, MODE>(p, i, n_items, NTW, KB, it); i += stride) {
      const int wrow = it.wt * 128 + q * 32 + lane;  // weight row of this lane: output column
      const int c0 = h * COLS;                       // first token column of this warp
      const int n = it.rows - c0;                    // its tokens (may be <= 0)
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) acc[j] = 0;
#pragma unroll 1
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        const int in_group = (kb - it.kb0) & (C::GROUP - 1);
        if (in_group == 0 && !mbar_wait_warp(&sfull[grp], gph, abort_flag, wd)) {
          ok = false;
          break;
        }
        const float* sc = scale_buf + (grp * C::GROUP + in_group) * SLOT;
        if (!mbar_wait_warp(&tfull[buf], bph, abort_flag, wd)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT + c0;
        const float ws = MODE == kFp8DenseRowScale ? sc[NT + q * 32 + lane] : 1.0f;
        const uint64_t ws2 = f2(ws, ws);
        // 16 columns, and 16 more where the warp has them (n is the same for all its lanes)
        uint32_t r[2][16];
        const bool wide = n > 16;
        if (n > 0) tmem_ld16(taddr, r[0]);
        if (wide) tmem_ld16(taddr + 16, r[1]);
        tmem_ld_wait16(r[0]);
        tmem_ld_wait16(r[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 0 ? n > 0 : wide) {
            const float4* cv = reinterpret_cast<const float4*>(sc + c0 + 16 * c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 v = cv[j];
              uint64_t s0 = f2(v.x, v.y), s1 = f2(v.z, v.w);
              if (MODE == kFp8DenseRowScale) s0 = f2_mul(s0, ws2), s1 = f2_mul(s1, ws2);
              uint64_t* a = acc + 8 * c + 2 * j;
              a[0] = f2_fma(f2(__uint_as_float(r[c][4 * j]), __uint_as_float(r[c][4 * j + 1])), s0, a[0]);
              a[1] = f2_fma(f2(__uint_as_float(r[c][4 * j + 2]), __uint_as_float(r[c][4 * j + 3])), s1, a[1]);
            }
          }
        }
        if (in_group == C::GROUP - 1 || kb + 1 == it.kb1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[grp]);
          if (++grp == C::GROUPS) {
            grp = 0;
            gph ^= 1;
          }
        }
        if (++buf == BUFS) {
          buf = 0;
          bph ^= 1;
        }
      }
      if (!ok && S == 1) break;
      if (S > 1) {
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (j < n) {
            float lo, hi;
            f2_split(acc[j >> 1], lo, hi);
            part[(c0 + j) * 128 + q * 32 + lane] = (j & 1) ? hi : lo;
          }
      } else if (wrow < N) {
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (j < n) {
            float lo, hi;
            f2_split(acc[j >> 1], lo, hi);
            const float v = (j & 1) ? hi : lo;
            const int64_t at = static_cast<int64_t>(it.row0 + c0 + j) * N + wrow;
            if (!GROUPED && p.f32)
              static_cast<float*>(p.y)[at] = v;
            else
              static_cast<uint16_t*>(p.y)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
          }
      }
    }
    if (S > 1) {
      // One-way split-K reduction, as in the NVFP4 streaming kernel: each CTA sends owner o the
      // block of o's tokens, the owners add their S slots in rank order. Every CTA sends, also
      // after an abort, and each owner waits for all (bounded), so that no CTA leaves while a
      // copy into its shared memory is in flight.
      fence_proxy_async_shared();
      named_sync(1, 32 * C::EPI_WARPS);
      const int rank = static_cast<int>(cluster_ctarank());
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
      const int mine = min(m_own, M - rank * m_own);
      volatile int32_t no_abort = 0;
      const bool received = mine > 0 && mbar_wait_warp(red_bar, 0, &no_abort, 4 * wd);
      if (mine > 0 && !received) *abort_flag = 1;
      if (received && !*abort_flag) {
        const int wrow = (static_cast<int>(blockIdx.x) / S) * 128 + q * 32 + lane;
        for (int idx = h; idx < mine; idx += C::EPI_WARPS / 4) {
          float v = 0.0f;
          for (int c = 0; c < S; ++c) v += recv[(c * m_own + idx) * 128 + q * 32 + lane];
          const int64_t at = static_cast<int64_t>(rank * m_own + idx) * N + wrow;
          if (wrow < N) {
            if (p.f32)
              static_cast<float*>(p.y)[at] = v;
            else
              static_cast<uint16_t*>(p.y)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
          }
        }
      }
    }
  } else {
    if (warp == 0 || warp == 2) {
      // warp 0 requests every stage's weight tile, warp 2 its token rows
      const uint64_t pol = warp == 0 ? policy_evict_first() : policy_evict_last();
      int s = 0, issued = 0;
      uint32_t ph = 0;
      uint32_t used = 0, phases = 0;  // per stage: requested at all, phase of the last request
      Fp8Item it;
      for (int i = first; fp8_item<NT, MODE>(p, i, n_items, NTW, KB, it) && !*abort_flag; i += stride) {
        const int nbox = (it.rows + 31) >> 5;
        const int wrow0 = it.e * N + it.wt * 128;
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!mbar_wait_warp(&empty[s], ph ^ 1, abort_flag, wd)) break;
          uint8_t* st = smem + s * C::STAGE_BYTES;
          if (warp == 0) {
            // test hook: the first CTA withholds a stage's expect-tx arrival and weight load
            const bool withheld = blockIdx.x == 0 && ++issued == p.drop_stage;
            if (!withheld && elect_one()) {
              mbar_arrive_expect_tx(&full[s], 16384);
              tma_load_2d(st, &tmW, &full[s], kb * 128, wrow0, pol);
            }
          } else if (elect_one()) {
            mbar_arrive_expect_tx(&full[s], nbox * 4096);
            for (int j = 0; j < nbox; ++j)
              tma_load_2d(st + 16384 + j * 4096, &tmX, &full[s], kb * 128, it.row0 + j * 32, pol);
          }
          __syncwarp();
          used |= 1u << s;
          phases = (phases & ~(1u << s)) | ph << s;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
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
      int s = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      Fp8Item it;
      for (int i = first; fp8_item<NT, MODE>(p, i, n_items, NTW, KB, it) && !*abort_flag; i += stride) {
        const uint32_t idesc = idesc_e4m3(128, ((it.rows + 15) >> 4) * 16);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!mbar_wait_warp(&tempty[buf], bph ^ 1, abort_flag, wd)) break;
          if (!mbar_wait_warp(&full[s], ph, abort_flag, wd)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t addr = smem_u32(smem + s * C::STAGE_BYTES);
            const uint64_t wdesc = desc_sw128(addr), xdesc = desc_sw128(addr + 16384);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc_mma_f8(tmem + buf * NT, wdesc + 2 * kk, xdesc + 2 * kk, idesc, kk != 0);
            tc_commit(&empty[s]);
            tc_commit(&tfull[buf]);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
          if (++buf == BUFS) {
            buf = 0;
            bph ^= 1;
          }
        }
      }
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      volatile int32_t dummy = 0;
      mbar_wait_warp(drain, 0, &dummy, wd);
    } else {
      // warp 3: the scales, a group of blocks at a time and up to GROUPS groups ahead of the epilogue.
      // A load issued now queues behind the TMA loads that the SM has in flight; in the epilogue
      // warps its latency paced every block (M = 33, 8192 x 8192: 24 us, 20 us in two halves of K).
      constexpr int NX = NT / 32, U = MODE == kFp8DenseRowScale ? 2 : 8;  // blocks per batch of loads
      int grp = 0;
      uint32_t gph = 0;
      bool ok = true;
      Fp8Item it;
      for (int i = first; ok && fp8_item<NT, MODE>(p, i, n_items, NTW, KB, it); i += stride) {
        // tokens past the tile's and rows past N read a scale inside it; their sums are not stored
        int tok[NX], wr[4];
#pragma unroll
        for (int j = 0; j < NX; ++j) tok[j] = it.row0 + min(lane + 32 * j, it.rows - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) wr[j] = min(it.wt * 128 + lane + 32 * j, N - 1);
        const float* sw = p.sb + (static_cast<int64_t>(it.e) * NTW + it.wt) * KB;
        for (int g0 = it.kb0; g0 < it.kb1; g0 += C::GROUP) {
#pragma unroll 1
          for (int b0 = 0; b0 < C::GROUP; b0 += U) {
            float x[U][NX], w[U][MODE == kFp8DenseRowScale ? 4 : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int kb = min(g0 + b0 + u, it.kb1 - 1);
#pragma unroll
              for (int j = 0; j < NX; ++j) x[u][j] = (p.sa + static_cast<int64_t>(kb) * M)[tok[j]];
              if (MODE == kFp8DenseRowScale) {
#pragma unroll
                for (int j = 0; j < (MODE == kFp8DenseRowScale ? 4 : 1); ++j)
                  w[u][j] = (p.sb + static_cast<int64_t>(kb) * N)[wr[j]];
              } else {
                w[u][0] = sw[kb];
              }
            }
            if (b0 == 0 && !mbar_wait_warp(&sempty[grp], gph ^ 1, abort_flag, wd)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
              float* d = scale_buf + (grp * C::GROUP + b0 + u) * SLOT + lane;
#pragma unroll
              for (int j = 0; j < NX; ++j) d[32 * j] = MODE == kFp8DenseRowScale ? x[u][j] : x[u][j] * w[u][0];
              if (MODE == kFp8DenseRowScale) {
#pragma unroll
                for (int j = 0; j < (MODE == kFp8DenseRowScale ? 4 : 1); ++j) d[NT + 32 * j] = w[u][j];
              }
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[grp]);
          if (++grp == C::GROUPS) {
            grp = 0;
            gph ^= 1;
          }
        }
      }
    }
  }

  // every thread that arrived on the cluster barrier also waits on it (the sending warp already did)
  if (S > 1 && warp != 4) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (threadIdx.x == 0 && *abort_flag) report_status(p.status, kStatusTimeout);
}

// ---- host launchers -------------------------------------------------------------------------------

template <int NT, int MODE>
static cudaError_t launch_fp8_stream_t(const CUtensorMap& tmW, const CUtensorMap& tmX, Fp8GemmArgs p, int grid,
                                       int recv_bytes, cudaStream_t st) {
  using C = Fp8StreamCfg<NT>;
  auto kernel = k_fp8_stream<NT, MODE>;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  const int fixed = 1024 + C::scale_bytes(MODE) + 512 + recv_bytes;
  int stages = ((C::CTAS == 2 ? 113 * 1024 : 226 * 1024) - fixed) / C::STAGE_BYTES;
  if (stages > 12) stages = 12;
  // the outgoing partials (a multiple of 512 bytes per token) reuse the ring
  while (recv_bytes > 0 && stages * C::STAGE_BYTES < static_cast<int>(p.M) * 512) ++stages;
  if (stages < 2) stages = 2;
  p.stages = stages;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = fixed + stages * C::STAGE_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = MODE == kFp8Grouped ? 1 : p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Token tiles of `tile_rows` rows (32 or 64; grouped: 32); tmX has 32-row boxes.
cudaError_t launch_fp8_stream(const CUtensorMap& tmW, const CUtensorMap& tmX, const Fp8GemmArgs& p, int tile_rows,
                              int sms, cudaStream_t st) {
  const int NTW = static_cast<int>((p.N + 127) / 128);
  if (p.tiles) {
    const int64_t items = static_cast<int64_t>(p.max_tiles) * NTW, slots = 2 * static_cast<int64_t>(sms);
    const int grid = static_cast<int>(items < slots ? items : slots);
    return launch_fp8_stream_t<32, kFp8Grouped>(tmW, tmX, p, grid, 0, st);
  }
  const int M = static_cast<int>(p.M), m_own = (M + p.split - 1) / p.split;
  const int recv = p.split > 1 ? p.split * m_own * 512 : 0;
  const int grid = NTW * p.split;
  if (p.b_rows == 1) {
    if (tile_rows == 32) return launch_fp8_stream_t<32, kFp8DenseRowScale>(tmW, tmX, p, grid, recv, st);
    return launch_fp8_stream_t<64, kFp8DenseRowScale>(tmW, tmX, p, grid, recv, st);
  }
  if (tile_rows == 32) return launch_fp8_stream_t<32, kFp8Dense>(tmW, tmX, p, grid, recv, st);
  return launch_fp8_stream_t<64, kFp8Dense>(tmW, tmX, p, grid, recv, st);
}

}  // namespace nvfp4

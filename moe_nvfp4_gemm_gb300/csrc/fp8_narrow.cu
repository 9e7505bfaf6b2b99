// FP8 block-scaled GEMM with the tokens on the MMA's narrow side, for experts of up to a few hundred
// rows (rows sorted by expert) and for dense layers: of 33 to 128 rows where the weight is wide, and of
// any number of rows from 9 on whose tiles are all resident at once where K is short (the rule with its
// measurements: capi.cu). With the weight of row m's expert (or the one weight),
// y[m, n] = sum_c sa[c, m] sb(c, n / 128) sum_{k in block c} a[m, k] b[n, k], a, b E4M3.
//
// A CTA pair (cta_group::2) takes 256 rows of a weight as the MMA's M and up to 128 of its
// tokens as N, 64 or 128: with the tokens on M a tile of 256 would be mostly empty. As in the tile
// kernel (fp8_gemm.cu) the tensor core sums one block of 128 of K from zero into a TMEM buffer, and
// the epilogue warps add it, times its scales, to fp32 registers; as in the streaming kernel the
// weights are read once, and the scales differ by column (a warp of their own brings them, the
// weight block's multiplied in). 128 columns leave room for four buffers, so that the MMA runs
// ahead of the hand-offs, and registers for loading a block's next chunk, or the next block's
// first, under the arithmetic of the one before.
//
// What bounds it: up to ~100 rows an expert the weights' bytes (256 experts of 6144 x 2048, 64 rows: 514 us,
// 0.99 of the measured copy rate; 256-row tiles 696, streaming 742; dense 28672 x 8192, 128 rows: 51 us,
// 256-row tiles 68). With more, ~720 cycles for a
// block of 128 tokens, and second tiles (128 rows on average: 714 us; its bytes 544). The loop must be free
// of conditions around the TMEM loads: guarding the last ones by `if` made the compiler keep the
// registers' old values too, and a block took 1,300 cycles instead of 720. Both chunks of a block by one
// load, with registers for two blocks, was slower (128 rows 773 us).
#include <stdint.h>

#include <type_traits>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

struct Fp8NarrowCfg {
  // warps 0-3: producer, MMA issuer, scales, idle; warps 4-11: epilogue. 384 x 168 registers at launch.
  static constexpr int THREADS = 384;
  static constexpr int CONTROL_REGS = 104, EPILOGUE_REGS = 200;
  static_assert(128 * CONTROL_REGS + 256 * EPILOGUE_REGS <= 384 * 168, "register shares");
  static constexpr int W_BYTES = 128 * 128, X_BYTES = 64 * 128;  // a CTA's weight rows, half of the tokens
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int STAGES = 7;
  static constexpr int X_BOX = 32;           // token rows of one TMA load
  static constexpr int BUFS = 4;             // TMEM buffers of 128 columns
  static constexpr int OUT_BYTES = 8 * 4096;  // 64 tokens x 32 weight rows per epilogue warp
  // Scales of GROUPS x GROUP blocks of K: 128 tokens' (times the weight block's), the weight block's.
  static constexpr int GROUP = 8, GROUPS = 4, SLOT = 132;
  static constexpr int SCALE_BYTES = GROUPS * GROUP * SLOT * 4;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + SCALE_BYTES + 1024 + 512;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Walks the tiles t = first, first + step, ...: token tile t / nt of the list, weight tile t % nt. The
// list's next entry is loaded a tile ahead. Plain loads behind griddep_wait: the list and the scales
// may be the previous kernel's, which this one overlaps (programmatic dependent launch).
struct Fp8Walk {
  const int4* list;
  int t, step, tiles, nt, mt;
  int M;
  int expert, m0, rows, n0;
  int4 ahead;
  DEVI void look(int at) {
    if (list) {
      ahead = list[at / nt];
    } else {  // one weight: token tiles of M rows
      const int r = at % mt * 128;
      ahead = make_int4(0, r, min(128, M - r), 0);
    }
  }
  DEVI void start(const Fp8GemmArgs& p, int first, int step_) {
    list = p.tiles;
    M = static_cast<int>(p.M);
    nt = (static_cast<int>(p.N) + 255) / 256;
    mt = (M + 127) / 128;
    t = first - step_;
    step = step_;
    tiles = nt * (list ? p.n_tiles[0] : mt);
    if (first < tiles) look(first);
    next();
  }
  DEVI bool valid() const { return t < tiles; }
  DEVI void next() {
    t += step;
    if (t >= tiles) return;
    expert = ahead.x;
    m0 = ahead.y;
    rows = ahead.z;
    n0 = (list ? t % nt : t / mt) * 256;
    if (t + step < tiles) look(t + step);
  }
  DEVI int columns() const { return (rows + 63) & ~63; }  // the MMA's N
};

__global__ void __launch_bounds__(Fp8NarrowCfg::THREADS, 1)
    k_fp8_narrow(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ Fp8GemmArgs p) {
  using C = Fp8NarrowCfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_buf = smem + STAGES * C::STAGE_BYTES;
  float* scale_buf = reinterpret_cast<float*>(out_buf + C::OUT_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(out_buf + C::OUT_BYTES + C::SCALE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;    // [BUFS]
  uint64_t* tempty = tfull + C::BUFS;  // [BUFS]
  uint64_t* sfull = tempty + C::BUFS;  // [GROUPS]
  uint64_t* sempty = sfull + C::GROUPS;
  uint64_t* drain = sempty + C::GROUPS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  const uint32_t rank = cluster_ctarank();  // the even CTA issues the MMAs
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);  // one elected lane per epilogue warp, both CTAs
    }
    for (int g = 0; g < C::GROUPS; ++g) {
      mbar_init(&sfull[g], 1);
      mbar_init(&sempty[g], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // set-up overlaps the previous kernel; every memory access waits for it

  const int M = static_cast<int>(p.M), N = static_cast<int>(p.N);
  const int nb = (N + 127) / 128;
  const int KB = static_cast<int>((p.K + 127) / 128);
  Fp8Walk w;

  if (warp >= 4) {
    regs_inc<C::EPILOGUE_REGS>();
    w.start(p, blockIdx.x / 2, gridDim.x / 2);
    const int q = warp & 3, h = (warp - 4) >> 2;
    uint8_t* box = out_buf + (warp - 4) * 4096;
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    uint32_t block = 0, group = 0;  // blocks of K and groups of scales so far
    bool ok = true;
    for (; w.valid() && ok; w.next()) {
      const int half = w.columns() >> 1;  // this warp's tokens: 32 or 64
      auto tile = [&](auto chunks_) {
        // The block sums in chunks of 32 tokens, the next chunk's load (of the next block, too) under this
        // one's arithmetic. fp32 pairs of neighbouring tokens: acc[16 c + 8 i + 2 g + j] is weight row
        // 16 i + 8 j + lane / 4 of the warp's 32, tokens 32 c + 8 g + 2 (lane % 4) and the next of its half.
        constexpr int CHUNKS = decltype(chunks_)::value;
        uint64_t acc[16 * CHUNKS];
#pragma unroll
        for (int i = 0; i < 16 * CHUNKS; ++i) acc[i] = 0;
        uint32_t r[2][32];
        const uint32_t row_at = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * (32 * CHUNKS);
        auto load = [&](int u, uint32_t* d) {
          const uint32_t blk = block + u / CHUNKS;
          if (CHUNKS == 1 || u % CHUNKS == 0) {
            ok = mbar_wait_warp(&tfull[blk & (C::BUFS - 1)], blk / C::BUFS & 1, abort_flag, wd) && ok;
            tc_fence_after();
          }
          const uint32_t at = row_at + (blk & (C::BUFS - 1)) * 128 + u % CHUNKS * 32;
          tmem_ld_frag32(at, d);
          tmem_ld_frag32(at + (16u << 16), d + 16);
        };
        // Unit u = CHUNKS kb + c, in r[i]; `more`: unit u + 1 follows. After a time-out (ok false) the
        // remaining waits end at once, and the sums are not used.
        auto unit = [&](int kb, auto i_, auto more_) {
          constexpr int i = decltype(i_)::value, c = CHUNKS == 1 ? 0 : i;
          constexpr bool more = decltype(more_)::value;
          if (c == CHUNKS - 1) {  // the block has landed
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive_cluster(tempty_leader + 8 * ((block + kb) & (C::BUFS - 1)));
          }
          const int in_group = kb & (C::GROUP - 1);
          if (c == 0 && in_group == 0)
            ok = mbar_wait_warp(&sfull[group & (C::GROUPS - 1)], group / C::GROUPS & 1, abort_flag, wd) && ok;
          if (more) load(CHUNKS == 1 ? kb + 1 : 2 * kb + i + 1, r[i ^ 1]);
          const float* sc = scale_buf + ((group & (C::GROUPS - 1)) * C::GROUP + in_group) * C::SLOT + h * (32 * CHUNKS) +
                            c * 32 + 2 * (lane & 3);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint64_t f = *reinterpret_cast<const uint64_t*>(sc + g * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t* x = r[i] + 16 * (j >> 1) + 4 * g + 2 * (j & 1);
              uint64_t& a = acc[16 * c + 8 * (j >> 1) + 2 * g + (j & 1)];
              a = f2_fma(f2(__uint_as_float(x[0]), __uint_as_float(x[1])), f, a);
            }
          }
          if (c == CHUNKS - 1 && (in_group == C::GROUP - 1 || kb + 1 == KB)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sempty[group & (C::GROUPS - 1)]);
            ++group;
          }
          if (more) tmem_ld_wait32(r[i ^ 1]);
        };
        constexpr std::integral_constant<int, 0> even;
        constexpr std::integral_constant<int, 1> odd;
        load(0, r[0]);
        tmem_ld_wait32(r[0]);
        int kb = 0;
        if constexpr (CHUNKS == 2) {
#pragma unroll 1
          for (; kb + 1 < KB; ++kb) {
            unit(kb, even, std::true_type());
            unit(kb, odd, std::true_type());
          }
          unit(kb, even, std::true_type());
          unit(kb, odd, std::false_type());
        } else {
#pragma unroll 1
          for (; kb + 2 < KB; kb += 2) {
            unit(kb, even, std::true_type());
            unit(kb + 1, odd, std::true_type());
          }
          if (kb + 2 == KB) {
            unit(kb, even, std::true_type());
            unit(kb + 1, odd, std::false_type());
          } else {
            unit(kb, even, std::false_type());
          }
        }
        block += KB;
        if (!ok) return;
        const int64_t row0 = w.m0 + h * half;
        const int tokens = min(w.rows - h * half, half), col0 = w.n0 + static_cast<int>(rank) * 128 + q * 32;
        if (tokens <= 0 || col0 >= N) return;
        // [token][32 weight rows] in the warp's box, 16-byte piece j of token t at j ^ (t / 2 % 4)
        const uint32_t at = smem_u32(box) + (lane & 7) * 64 + (((lane >> 3) ^ (lane >> 1 & 3)) << 4);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float lo, hi;
              f2_split(acc[16 * c + 8 * (i >> 1) + 2 * g + (i & 1)], lo, hi);
              m[i] = pack_bf16x2(lo, hi);
            }
            st_matrix_x4_trans(at + (4 * c + g) * 512, m[0], m[1], m[2], m[3]);
          }
        __syncwarp();
        uint16_t* y = static_cast<uint16_t*>(p.y) + row0 * N + col0;
        if (N % 8 == 0) {  // 16 bytes a lane, eight tokens at a time
          if (col0 + 8 * (lane & 3) < N)
            for (int i = lane >> 2; i < tokens; i += 8)
              *reinterpret_cast<uint4*>(y + static_cast<int64_t>(i) * N + 8 * (lane & 3)) =
                  *reinterpret_cast<const uint4*>(box + i * 64 + (((lane & 3) ^ (i >> 1 & 3)) << 4));
        } else if (col0 + lane < N) {
          for (int i = 0; i < tokens; ++i)
            y[static_cast<int64_t>(i) * N + lane] =
                reinterpret_cast<const uint16_t*>(box)[i * 32 + (((lane >> 3) ^ (i >> 1 & 3)) << 3) + (lane & 7)];
        }
        __syncwarp();
      };
      if (half == 32)
        tile(std::integral_constant<int, 1>());
      else
        tile(std::integral_constant<int, 2>());
    }
  } else {
    regs_dec<C::CONTROL_REGS>();
    if (warp < 3) w.start(p, blockIdx.x / 2, gridDim.x / 2);
    if (warp == 0) {
      const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
      int s = 0;
      uint32_t ph = 0;
      uint32_t used = 0, phases = 0;  // per stage: requested at all, phase of the last request
      int issued = 0;
      for (; w.valid() && !*abort_flag; w.next()) {
        const int half = w.columns() >> 1;
        const int x_row = w.m0 + static_cast<int>(rank) * half;
        const int w_row = w.expert * N + w.n0 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_warp(&empty[s], ph ^ 1, abort_flag, wd)) break;
          // test hook: the first CTA withholds its expect-tx arrival and loads
          const bool withheld = blockIdx.x == 0 && ++issued == p.drop_stage;
          if (!withheld && elect_one()) {
            uint8_t* st = smem + s * C::STAGE_BYTES;
            const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
            if (leader) mbar_arrive_expect_tx(&full[s], 2 * (C::W_BYTES + half * 128));
            tma_load_2d_pair(st, &tmW, bar, kb * 128, w_row, pol_w);
            for (int i = 0; i < half; i += C::X_BOX)
              tma_load_2d_pair(st + C::W_BYTES + i * 128, &tmX, bar, kb * 128, x_row + i, pol_x);
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
      griddep_launch_dependents();
      // The even CTA's full barriers count both CTAs' bytes: let them all land.
      if (leader)
        for (int i = 0; i < STAGES; ++i)
          if (used >> i & 1) {
            volatile int32_t dummy = 0;
            mbar_wait_warp(&full[i], phases >> i & 1, &dummy, wd);
          }
    } else if (warp == 1 && leader) {
      int s = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      for (; w.valid() && !*abort_flag; w.next()) {
        const uint32_t idesc = idesc_e4m3(256, w.columns());
        for (int kb = 0; kb < KB; ++kb) {
          // both polled at once: each answer takes ~110 cycles, a block's issue 210 (64 rows of 28672 x 8192
          // 45.7 -> 44.3 us, of 5003 x 2064 9.7 -> 9.0)
          const uint32_t got = mbar_try_wait(smem_u32(&full[s]), ph), free = mbar_try_wait(smem_u32(&tempty[buf]), bph ^ 1);
          if (!__all_sync(0xffffffffu, got & free)) {
            if (!mbar_wait_warp(&full[s], ph, abort_flag, wd)) break;
            if (!mbar_wait_warp(&tempty[buf], bph ^ 1, abort_flag, wd)) break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t w_addr = smem_u32(smem + s * C::STAGE_BYTES);
            const uint64_t wdesc = desc_sw128(w_addr), xdesc = desc_sw128(w_addr + C::W_BYTES);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc_mma_f8_pair(tmem + buf * 128, wdesc + 2 * kk, xdesc + 2 * kk, idesc, kk != 0);
            tc_commit_pair(&empty[s], 3u);
            tc_commit_pair(&tfull[buf], 3u);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
          if (++buf == C::BUFS) {
            buf = 0;
            bph ^= 1;
          }
        }
      }
      if (elect_one()) tc_commit_pair(drain, 1u);
      __syncwarp();
      volatile int32_t dummy = 0;
      mbar_wait_warp(drain, 0, &dummy, wd);
    } else if (warp == 2) {
      // The scales, a group of blocks at a time, requested two to three groups ahead (a load queues behind
      // the TMA loads that the SM has in flight). Tokens past the tile's read a scale inside it; their
      // sums are not stored.
      uint32_t requested = 0;
      int g0 = 0;
      bool ok = true;
      auto request = [&]() {
        if (w.valid() && ok) {
          const uint32_t g = requested & (C::GROUPS - 1);
          ok = mbar_wait_warp(&sempty[g], (requested / C::GROUPS & 1) ^ 1, abort_flag, wd);
          if (ok) {
            int tok[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) tok[j] = w.m0 + min(lane + 32 * j, w.rows - 1);
            const float* sw =
                p.sb + (static_cast<int64_t>(w.expert) * nb + min((w.n0 >> 7) + static_cast<int>(rank), nb - 1)) * KB;
            const int n = min(C::GROUP, KB - g0);
            float* d = scale_buf + g * (C::GROUP * C::SLOT);
            for (int u = 0; u < n; ++u, d += C::SLOT) {
              const float* sa = p.sa + static_cast<int64_t>(g0 + u) * M;
#pragma unroll
              for (int j = 0; j < 4; ++j) cp_async4(d + 32 * j + lane, sa + tok[j]);
              if (lane == 0) cp_async4(d + 128, sw + g0 + u);
            }
            ++requested;
            g0 += C::GROUP;
            if (g0 >= KB) {
              g0 = 0;
              w.next();
            }
          }
        }
        cp_async_commit();
      };
#pragma unroll 1
      for (int i = 0; i < C::GROUPS - 1; ++i) request();
#pragma unroll 1
      for (uint32_t done = 0; ok && done < requested; ++done) {
        cp_async_wait<C::GROUPS - 2>();
        __syncwarp();
        const uint32_t g = done & (C::GROUPS - 1);
        float* d = scale_buf + g * (C::GROUP * C::SLOT);
#pragma unroll
        for (int u = 0; u < C::GROUP; ++u) {
          const float s = d[u * C::SLOT + 128];
          float4* x = reinterpret_cast<float4*>(d + u * C::SLOT) + lane;
          float4 v = *x;
          v.x *= s, v.y *= s, v.z *= s, v.w *= s;
          *x = v;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[g]);
        request();
      }
      cp_async_wait<0>();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) report_status(p.status, kStatusTimeout);
}

cudaError_t launch_fp8_narrow(const CUtensorMap& tmW, const CUtensorMap& tmX, const Fp8GemmArgs& p, int grid,
                                    cudaStream_t st) {
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(k_fp8_narrow));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Fp8NarrowCfg::THREADS);
  cfg.dynamicSmemBytes = Fp8NarrowCfg::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k_fp8_narrow, tmW, tmX, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace nvfp4

// Tile products of the 16-bit gated feed-forward block, bf16 or fp16 operands, fp32 sums:
//   forward   g = x Wg^T, u = x Wu^T, h = act(g) u         x [M, K], Wg, Wu [I, K], h [M, I]
//   input     dx = dg Wg + du Wu                           dg, du [M, I], dx [M, K]
//   weight    dWg = dg^T x, dWu = du^T x                   dWg, dWu [I, K]
// with act(g) = g s, s = sigma(p(g)); silu: p = g, gelu (tanh form): p = 2 sqrt(2/pi) (g + 0.044715 g^3).
//
// One persistent kernel body: a CTA pair (cta_group::2) computes 256 x 256 sums per tile, K in stages of
// 64, two TMEM buffers (all 512 columns), so that the MMAs of a tile run while the one before is stored.
// The forward tile has 128 gate and 128 up columns: the pair's even CTA loads rows of Wg, the odd one
// rows of Wu, and both halves of the sums of a row meet in one thread, which applies the activation
// to the fp32 sums. The gradients need no transposed copies: the products read W along its rows
// (input) and all operands along theirs (weight) as MN-major tiles, two 64 x 64 boxes for 128 rows. Both
// gradients' tiles are one launch, so that the few tiles of the one fill the pairs that the other leaves.
//
// Products of few tiles are cut along their contraction into parts; the parts' fp32 sums go to
// the workspace and are added, in the order of the contraction, by k_ffn_join.
//
// Bound by the tensor cores: 4096 x 14336 x 8192 forward 0.94-1.14 ms (up to 2.04 PFLOP/s in a burst, less under the power
// cap), 4096 x 8192 x 4096 forward 272 us, both gradients 594-616 us (1.78-1.85 PFLOP/s).
#include <stdint.h>

#include "ffn.cuh"
#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

struct FfnCfg {
  // warps 0-3: producer, MMA issuer, two idle; warps 4-11: epilogue
  static constexpr int THREADS = 384;
  static constexpr int TILE_BYTES = 128 * 128;  // 128 rows x 64 of the contraction
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int OUT_BYTES = 8 * 4096;  // one 32-row x 128-byte store box per epilogue warp
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + 1024 + 256;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// One item of the persistent walk: a tile of a product and a part of its contraction.
struct FfnItem {
  int product, which;  // of p.in; its result, 0 or 1
  int m0, n0;          // first row and column of the tile
  int kb0, kb1;        // its blocks of 64
  int part;
};

DEVI FfnItem ffn_item(const FfnTileArgs& p, int i) {
  FfnItem it;
  it.product = i >= p.in[0].items;
  if (it.product) i -= p.in[0].items;
  const FfnProduct& q = p.in[it.product];
  const int tiles = q.mt * q.nt, per_result = tiles * q.split;
  it.which = i / per_result;
  i -= it.which * per_result;
  it.part = i / tiles;
  int mb, nb;
  tile_coords(i - it.part * tiles, q.mt, q.nt, q.raster, mb, nb);
  it.m0 = mb * 256;
  it.n0 = nb * 256;
  it.kb0 = static_cast<int>(static_cast<int64_t>(q.kblocks) * it.part / q.split);
  it.kb1 = static_cast<int>(static_cast<int64_t>(q.kblocks) * (it.part + 1) / q.split);
  return it;
}

// A warp's 32 rows x 128 bytes of packed results, w[4 c .. 4 c + 3] in 16-byte piece c, through its
// box (piece c of row r at c ^ (r % 8)) to the tensor.
DEVI void ffn_store_box(uint8_t* box, const CUtensorMap* tm, int col, int row, const uint32_t (&w)[32]) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) bulk_wait_group_read0();  // the previous box has left the buffer
  __syncwarp();
  const uint32_t at = smem_u32(box) + lane * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + ((c ^ (lane & 7)) << 4)), "r"(w[4 * c]),
                 "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                 : "memory");
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tm, box, col, row);
    bulk_commit_group();
  }
}

template <bool FORWARD, bool HALF>
__global__ void __launch_bounds__(FfnCfg::THREADS, 1)
    k_ffn_tile(const __grid_constant__ FfnTileMaps maps, const __grid_constant__ FfnTileArgs p) {
  using C = FfnCfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_buf = smem + STAGES * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_buf + C::OUT_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;  // [2]
  uint64_t* tempty = tfull + 2;      // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;  // issues the pair's MMAs
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);  // one elected lane per epilogue warp, both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
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

  const int items = p.in[0].items + p.in[1].items;
  const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;

  if (warp >= 4) {
    const int q = warp & 3, h = (warp - 4) >> 2;
    uint8_t* box = out_buf + (warp - 4) * 4096;
    const uint32_t tempty_leader[2] = {mapa_shared(smem_u32(&tempty[0]), 0), mapa_shared(smem_u32(&tempty[1]), 0)};
    int buf = 0;
    uint32_t bph = 0;
    for (int i = pair; i < items; i += npairs) {
      const FfnItem it = ffn_item(p, i);
      if (!mbar_wait_warp(&tfull[buf], bph, abort_flag, wd)) break;
      tc_fence_after();
      const int row0 = it.m0 + rank * 128 + q * 32;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive_cluster(tempty_leader[buf]);
      };
      const FfnProduct& pr = p.in[it.product];
      if (pr.split > 1) {
        // fp32 sums to [part][tile rows][tile columns] of the workspace
        const int wrow = (it.which * pr.split + it.part) * pr.mt * 256 + row0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(lanes + h * 128 + c * 32, r);
          tmem_ld_wait32(r);
          if (c == 3) release();
          if (row0 < pr.M) ffn_store_box(box, &maps.part[it.product], it.n0 + h * 128 + c * 32, wrow, r);
        }
      } else if constexpr (FORWARD) {
        // 64 columns of h: their gate sums, and the up sums 128 columns further on
        const int col = it.n0 / 2 + h * 64;
        const bool stored = row0 < pr.M && col < pr.N;
        uint32_t hw[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t g[32], u[32];
          tmem_ld32(lanes + h * 64 + c * 32, g);
          tmem_ld32(lanes + 128 + h * 64 + c * 32, u);
          tmem_ld_wait32(g);
          tmem_ld_wait32(u);
          if (c == 1) release();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            hw[16 * c + j] = pack16<HALF>(ffn_act(__uint_as_float(g[2 * j]), p.act) * __uint_as_float(u[2 * j]),
                                          ffn_act(__uint_as_float(g[2 * j + 1]), p.act) * __uint_as_float(u[2 * j + 1]));
          if (p.save && row0 + lane < pr.M) {
            // whole 32-byte sectors from the registers: through the box the five stores of a tile wait for each other
            // (333 x 2816 x 1024 with its gradients: 44 us instead of 33)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float* to = static_cast<float*>(p.y[1 + k]) + static_cast<int64_t>(row0 + lane) * pr.N + col + c * 32;
              const uint32_t(&w)[32] = k ? u : g;
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                if (col + c * 32 + j < pr.N) {
                  const uint32_t w8[8] = {w[j], w[j + 1], w[j + 2], w[j + 3], w[j + 4], w[j + 5], w[j + 6], w[j + 7]};
                  st_global_v8(to + j, w8);
                }
            }
          }
        }
        if (stored) ffn_store_box(box, &maps.y[0], col, row0, hw);
      } else {
        const CUtensorMap* y = &maps.y[it.product + it.which];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int col = it.n0 + h * 128 + b * 64;
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
            tmem_ld32(lanes + h * 128 + b * 64 + c * 32, r);
            tmem_ld_wait32(r);
            if (b == 1 && c == 1) release();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[16 * c + j] = pack16<HALF>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
          }
          if (row0 < pr.M && col < pr.N) ffn_store_box(box, y, col, row0, w);
        }
      }
      buf ^= 1;
      bph ^= buf == 0;
    }
    if (lane == 0) bulk_wait_group0();  // this warp's stores are complete before the CTA exits
    __syncwarp();
  } else if (warp == 0) {
    const uint64_t pol = policy_evict_last();
    // weights that one row of tiles reads once are not kept
    const uint64_t pol_w = FORWARD && p.in[0].mt == 1 ? policy_evict_first() : pol;
    int s = 0, issued = 0;
    uint32_t ph = 0;
    uint32_t used = 0, phases = 0;  // per stage: requested at all, phase of the last request
    for (int i = pair; i < items && !*abort_flag; i += npairs) {
      const FfnItem it = ffn_item(p, i);
      const int am = it.m0 + static_cast<int>(rank) * 128;
      const int bn = FORWARD ? it.n0 / 2 : it.n0 + static_cast<int>(rank) * 128;
      const int half = p.in[0].kblocks / 2;
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        if (!mbar_wait_warp(&empty[s], ph ^ 1, abort_flag, wd)) break;
        // test hook: the first CTA withholds its expect-tx arrival and loads
        const bool withheld = blockIdx.x == 0 && ++issued == p.drop_stage;
        if (!withheld && elect_one()) {
          uint8_t* st = smem + s * C::STAGE_BYTES;
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
          if constexpr (FORWARD) {
            tma_load_2d_pair(st, &maps.a[0], bar, kb * 64, am, pol);
            tma_load_2d_pair(st + C::TILE_BYTES, &maps.b[rank], bar, kb * 64, bn, pol_w);
          } else {
            // boxes of 64 x 64. Input: the contraction is the gate's columns, then the up's; dg and du lie along it.
            // Weight: all operands lie along their rows.
            const int second = it.product ? it.which : kb >= half;
            const int k0 = (it.product || !second ? kb : kb - half) * 64;
            const CUtensorMap* ta = &maps.a[it.product ? p.up_first ^ second : second];
            const CUtensorMap* tb = &maps.b[it.product ? 2 : second];
            tma_load_2d_pair(st, ta, bar, it.product ? am : k0, it.product ? k0 : am, pol);
            tma_load_2d_pair(st + C::TILE_BYTES / 2, ta, bar, it.product ? am + 64 : k0, it.product ? k0 : am + 64, pol);
            tma_load_2d_pair(st + C::TILE_BYTES, tb, bar, bn, k0, pol);
            tma_load_2d_pair(st + C::TILE_BYTES * 3 / 2, tb, bar, bn + 64, k0, pol);
          }
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
      for (int j = 0; j < STAGES; ++j)
        if (used >> j & 1) {
          volatile int32_t dummy = 0;
          mbar_wait_warp(&full[j], phases >> j & 1, &dummy, wd);
        }
  } else if (warp == 1 && leader) {
    int s = 0, buf = 0;
    uint32_t ph = 0, bph = 0;
    for (int i = pair; i < items && !*abort_flag; i += npairs) {
      const FfnItem it = ffn_item(p, i);
      const bool a_mn = !FORWARD && it.product == 1;
      constexpr bool B_MN = !FORWARD;
      const uint32_t idesc = a_mn ? idesc_f16(256, 256, !HALF, true, B_MN) : idesc_f16(256, 256, !HALF, false, B_MN);
      const uint32_t a_step = a_mn ? 128 : 2;
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        if (!mbar_wait_warp(&full[s], ph, abort_flag, wd)) break;
        if (kb == it.kb0 && !mbar_wait_warp(&tempty[buf], bph ^ 1, abort_flag, wd)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t addr = smem_u32(smem + s * C::STAGE_BYTES);
          // a step of 16: 32 bytes of a K-major row, two 8-row groups (2,048 bytes) of an MN-major tile
          const uint64_t ad = a_mn ? desc_sw128_mn(addr, C::TILE_BYTES / 2) : desc_sw128(addr);
          const uint64_t bd = B_MN ? desc_sw128_mn(addr + C::TILE_BYTES, C::TILE_BYTES / 2) : desc_sw128(addr + C::TILE_BYTES);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_pair(tmem + buf * 256, ad + a_step * kk, bd + (B_MN ? 128 : 2) * kk, idesc,
                            kb != it.kb0 || kk != 0);
          tc_commit_pair(&empty[s], 3);
          if (kb + 1 == it.kb1) tc_commit_pair(&tfull[buf], 3);
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
      buf ^= 1;
      bph ^= buf == 0;
    }
    if (elect_one()) tc_commit_pair(drain, 1);
    __syncwarp();
    volatile int32_t dummy = 0;
    mbar_wait_warp(drain, 0, &dummy, wd);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still read its shared memory or signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) report_status(p.status, kStatusTimeout);
}

// ---- joining the parts ----------------------------------------------------------------------------

// y[r, c] = the parts' sums in the order of the contraction, eight columns a thread. Forward: columns
// 256 b + j and 256 b + 128 + j of the workspace are gate and up of column 128 b + j of h.
template <bool FORWARD, bool HALF>
__global__ void __launch_bounds__(256) k_ffn_join(const __grid_constant__ FfnTileArgs p) {
  griddep_wait();
  griddep_launch_dependents();
#pragma unroll 1
  for (int product = 0; product < (FORWARD ? 1 : 2); ++product) {
    const FfnProduct& q = p.in[product];
    if (q.items == 0 || q.split == 1) continue;
    const int groups = q.N / 8, results = q.items / (q.mt * q.nt * q.split);
    const int64_t total = static_cast<int64_t>(q.M) * groups * results;
    const int64_t cols = static_cast<int64_t>(q.nt) * 256, part = static_cast<int64_t>(q.mt) * 256 * cols;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
      const int c = static_cast<int>(i % groups) * 8;
      const int64_t row = i / groups;
      const int which = static_cast<int>(row / q.M);
      const int64_t r = row - static_cast<int64_t>(which) * q.M;
      auto sum = [&](int64_t at, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        const float* src = q.ws + which * q.split * part + r * cols + at;
#pragma unroll 4
        for (int s = 0; s < q.split; ++s, src += part) {
          const float4 lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + 4);
          v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
          v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
        }
      };
      auto store = [&](void* y, int64_t ld, const float (&v)[8]) {
        uint16_t* to = static_cast<uint16_t*>(y) + r * ld + c;
        st_global_v4(to, pack16<HALF>(v[0], v[1]), pack16<HALF>(v[2], v[3]), pack16<HALF>(v[4], v[5]), pack16<HALF>(v[6], v[7]));
      };
      float v[8];
      if (FORWARD) {
        const int64_t at = static_cast<int64_t>(c / 128) * 256 + c % 128;
        float u[8];
        sum(at, v);
        sum(at + 128, u);
        if (p.save)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float(&w)[8] = k ? u : v;
            float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.y[1 + k]) + r * q.N + c);
            to[0] = make_float4(w[0], w[1], w[2], w[3]);
            to[1] = make_float4(w[4], w[5], w[6], w[7]);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ffn_act(v[j], p.act) * u[j];
      } else {
        sum(c, v);
      }
      store(p.y[product + which], FORWARD ? p.ldy : q.N, v);
    }
  }
}

// ---- gradients of the sums ------------------------------------------------------------------------

// dg = dh u act'(g), du = dh act(g) for eight neighbouring values a thread, from the forward call's fp32 sums: bound by
// its 14 bytes an element. dg and du are rounded to 16 bits, as the tensor cores read them: half a step of the type,
// like the rounding of the results, and with it all that the gradients lose (kept as 16-bit values, g and u
// would bring the gradients' error from 1.4 to 1.8 times that of the one rounding of a result). In fp16 one beyond 65,504
// becomes infinite and one below 2^-25 zero, as in any fp16 backward pass; bf16 has fp32's range.
template <bool HALF>
__global__ void __launch_bounds__(256) k_ffn_grad(const __grid_constant__ FfnGradArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int groups = p.I / 8;
  const int64_t total = static_cast<int64_t>(p.M) * groups;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / groups;
    const int c = static_cast<int>(i - r * groups) * 8;
    const float4* gs = reinterpret_cast<const float4*>(p.gate) + 2 * i;
    const float4* us = reinterpret_cast<const float4*>(p.up) + 2 * i;
    const float4 g0 = gs[0], g1 = gs[1], u0 = us[0], u1 = us[1];
    const uint4 dv = *reinterpret_cast<const uint4*>(p.dh + r * p.lddh + c);
    const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w}, u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    const uint32_t d[4] = {dv.x, dv.y, dv.z, dv.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a0, a1, s0, s1;
      ffn_act_grad(g[2 * j], p.act, a0, s0);
      ffn_act_grad(g[2 * j + 1], p.act, a1, s1);
      const float d0 = unpack16<HALF>(d[j], 0), d1 = unpack16<HALF>(d[j], 1);
      og[j] = pack16<HALF>(d0 * u[2 * j] * s0, d1 * u[2 * j + 1] * s1);
      ou[j] = pack16<HALF>(d0 * a0, d1 * a1);
    }
    reinterpret_cast<uint4*>(p.dg)[i] = make_uint4(og[0], og[1], og[2], og[3]);
    reinterpret_cast<uint4*>(p.du)[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// ---- host launchers -------------------------------------------------------------------------------

template <typename Kernel, typename... Args>
static cudaError_t launch_dependent(Kernel kernel, int grid, int block, int smem, int cluster, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool FORWARD, bool HALF>
static cudaError_t launch_tile(const FfnTileMaps& maps, const FfnTileArgs& p, int sms, cudaStream_t st) {
  auto kernel = k_ffn_tile<FORWARD, HALF>;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  const int items = p.in[0].items + p.in[1].items, pairs = items < sms / 2 ? items : sms / 2;
  e = launch_dependent(kernel, 2 * pairs, FfnCfg::THREADS, FfnCfg::SMEM_BYTES, 2, st, maps, p);
  if (e != cudaSuccess) return e;
  int64_t threads = 0;
  for (const FfnProduct& q : p.in)
    if (q.items > 0 && q.split > 1) threads += static_cast<int64_t>(q.M) * (q.N / 8) * (q.items / (q.mt * q.nt * q.split));
  if (threads == 0) return cudaSuccess;
  const int64_t blocks = (threads + 255) / 256, most = 8 * static_cast<int64_t>(sms);
  return launch_dependent(k_ffn_join<FORWARD, HALF>, static_cast<int>(blocks < most ? blocks : most), 256, 0, 1, st, p);
}

cudaError_t launch_ffn_tile(const FfnTileMaps& maps, const FfnTileArgs& p, bool forward, int sms, cudaStream_t st) {
  if (forward) return p.half ? launch_tile<true, true>(maps, p, sms, st) : launch_tile<true, false>(maps, p, sms, st);
  return p.half ? launch_tile<false, true>(maps, p, sms, st) : launch_tile<false, false>(maps, p, sms, st);
}

cudaError_t launch_ffn_grad(const FfnGradArgs& p, int sms, cudaStream_t st) {
  const int64_t blocks = (p.M * (p.I / 8) + 255) / 256, most = 8 * static_cast<int64_t>(sms);
  const int grid = static_cast<int>(blocks < most ? blocks : most);
  return p.half ? launch_dependent(k_ffn_grad<true>, grid, 256, 0, 1, st, p)
                : launch_dependent(k_ffn_grad<false>, grid, 256, 0, 1, st, p);
}

}  // namespace nvfp4

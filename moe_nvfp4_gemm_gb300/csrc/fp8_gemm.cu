// FP8 block-scaled tile GEMM: y[m, n] = sum_c sa[c, m] sb(c, n) sum_{k in block c} a[m, k] b[n, k],
// a, b E4M3, c running over blocks of 128 of K, sb one scale per 128 rows of b or one per row.
//
// The tensor core sums one block of 128 (four K = 32 MMAs) from zero into a TMEM buffer; the
// epilogue warps read the 256 x 256 block sums back and add them, times their scales, to the
// result, which stays in their registers (fp32) for the whole of K. So each block sum meets
// its two fp32 scales exactly once, and two TMEM buffers (all 512 columns) let the MMA of block
// c + 1 run while block c is read.
//
// One CTA pair (cta_group::2) per 256 x 256 tile of y: per block of K each CTA loads 128 rows of a
// and of b (32 KB by TMA, 128-byte swizzle) and the pair's MMAs take 512 cycles at the full rate.
// What bounds it: a block takes ~860 cycles (4096 x 28672 x 8192: 712 us, 2.70 PFLOP/s; under the power
// cap 800 us), half of the chain MMA - commit - TMEM loads and arithmetic - release, as there are two
// buffers. The eight epilogue warps of a CTA need ~530 of it to read (4 x tcgen05.ld of 32 columns)
// and add (64 packed fma) their 128 columns of a row; a ready barrier costs ~110; without the arithmetic
// the same loop takes ~580. Tried without gain: 16 epilogue warps of 64 columns, four half-width
// buffers, 64-column loads, plain instead of packed fma, the row scales through a warp of their own,
// plain stores instead of TMA (765 us). What does cost is any register that spills in the loop: it
// comes back through the memory system, behind the TMA loads in flight (1.7 times the time).
#include <stdint.h>

#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

struct Fp8PairCfg {
  // warps 0-3: producer, MMA issuer, two idle; warps 4-11: epilogue. 384 x 168 registers at
  // launch; the epilogue takes what the first warpgroup gives up: 128 x 72 + 256 x 216 = 384 x 168.
  static constexpr int THREADS = 384;
  static constexpr int CONTROL_REGS = 72, EPILOGUE_REGS = 216;
  static_assert(128 * CONTROL_REGS + 256 * EPILOGUE_REGS <= 384 * 168, "register shares");
  static constexpr int TILE_BYTES = 128 * 128;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int OUT_BYTES = 8 * 4096;  // one 32-row x 128-byte store box per epilogue warp
  // COLSCALE: slots of 256 column and 128 row scales. When block c is written the MMA of block c - 3 is
  // known to be done, so the buffer of block c - 5 was released and all warps are past block c - 6.
  static constexpr int SLOTS = 8, SCALES = 384;
  static constexpr int SCALE_BYTES = SLOTS * SCALES * 4;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + SCALE_BYTES + 1024 + 256;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Loads that stay at their place: hoisted, a block's scales would not fit the registers.
DEVI uint64_t ld_shared_b64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
DEVI float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

struct Fp8Tile {
  int m0, m_end;  // rows of a and y: [m0, m_end)
  int b_row;      // first row of b
  int n0;         // first column of y
  const float* sb;
};

// Everything that the previous kernel in the stream may have written (tile list, scales) is read
// with plain loads: this kernel starts while that one may still run (programmatic dependent
// launch), so the data is not read-only for the kernel's life, as the non-coherent path (__ldg)
// requires; a plain load stays behind griddep_wait.
template <bool GROUPED>
DEVI Fp8Tile fp8_tile(const Fp8GemmArgs& p, int t, int mt, int nt, int kbs) {
  Fp8Tile r;
  const int N = static_cast<int>(p.N);
  if (GROUPED) {
    const int4 d = p.tiles[t / nt];
    r.n0 = (t % nt) * 256;
    r.m0 = d.y;
    r.m_end = d.y + d.z;
    r.b_row = d.x * N + r.n0;
    r.sb = p.sb + static_cast<int64_t>(d.x) * ((N + 127) / 128) * kbs;
  } else {
    r.m0 = (t % mt) * 256;
    r.n0 = (t / mt) * 256;
    r.m_end = static_cast<int>(p.M);
    r.b_row = r.n0;
    r.sb = p.sb;
  }
  return r;
}

// A warp's 32 rows x 128 bytes of results to y, through its 4 KB box (16-byte chunk c of row r at
// chunk c ^ (r % 8)): by a TMA store (whole boxes), or with plain stores where y's rows are
// not 16-byte aligned (a row at a time) or a grouped tile ends inside the box (four rows at a time).
template <bool F32, typename Fill>
DEVI void fp8_store_box(const Fp8GemmArgs& p, uint8_t* buf, Fill&& fill, const CUtensorMap* tmY, bool by_tma, int row0,
                        int m_end, int col0, int N) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) bulk_wait_group_read0();  // the previous box has left the buffer
  __syncwarp();
  fill(smem_u32(buf));
  if (by_tma) {
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tmY, buf, col0, row0);
      bulk_commit_group();
    }
  } else {
    __syncwarp();
    const int rows = min(32, m_end - row0);
    constexpr int PER16 = F32 ? 4 : 8;  // values per 16 bytes
    if (N % PER16 == 0) {  // four rows at a time, 16 bytes a lane
      const int c = lane & 7;
      if (col0 + c * PER16 < N)
        for (int r = lane >> 3; r < rows; r += 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
          uint8_t* y = static_cast<uint8_t*>(p.y) + (static_cast<int64_t>(row0 + r) * N + col0 + c * PER16) * (16 / PER16);
          *reinterpret_cast<uint4*>(y) = v;
        }
      __syncwarp();
      return;
    }
    for (int r = 0; r < rows; ++r) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
      const int64_t at = static_cast<int64_t>(row0 + r) * N + col0;
      if (F32) {
        if (col0 + lane < N) static_cast<float*>(p.y)[at + lane] = __uint_as_float(v);
      } else {
        uint16_t* y = static_cast<uint16_t*>(p.y) + at + 2 * lane;
        if (col0 + 2 * lane < N) y[0] = static_cast<uint16_t>(v & 0xFFFFu);
        if (col0 + 2 * lane + 1 < N) y[1] = static_cast<uint16_t>(v >> 16);
      }
    }
    __syncwarp();
  }
}

// COLSCALE: one scale per row of b (a column of y), applied before the row scale; otherwise one per 128
// rows of b, which a warp's 128 columns share. A broadcast read of shared memory returns 16 bytes a lane
// all the same, so with a lane to a row the columns' scales cost 1,024 cycles a block and CTA; with the
// 16 x 256-bit TMEM loads a lane has four rows of a column pair, and a quarter of that is left. A warp of
// its own brings the scales (through cp.async of each epilogue warp 187 us for 4096 x 6144 x 4112 with
// fp32 results, now 136: a block takes ~1,320 cycles, half of them the 128 packed operations).
//
// SPLIT > 1: K in SPLIT parts, for products of few tiles. The SPLIT pairs of a cluster sum one tile's
// parts, then each CTA gets a SPLIT-th of its rows' columns from all of them through distributed
// shared memory, adds them in the order of K and stores them (one tile per cluster).
template <bool COLSCALE, bool GROUPED, bool F32, int SPLIT>
__global__ void __launch_bounds__(Fp8PairCfg::THREADS, 1)
    k_fp8_gemm_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmY, const __grid_constant__ Fp8GemmArgs p) {
  using C = Fp8PairCfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_buf = smem + STAGES * C::STAGE_BYTES;
  float* scale_buf = reinterpret_cast<float*>(out_buf + C::OUT_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(out_buf + C::OUT_BYTES + C::SCALE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;  // [2]
  uint64_t* tempty = tfull + 2;      // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  // pair `part` of the cluster: its even CTA, which issues the MMAs, has cluster rank `lead`
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
  const int part = static_cast<int>(crank >> 1);
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], COLSCALE ? 2 : 1);  // the MMA's commit; the warp of the scales
      mbar_init(&tempty[b], 16);  // one elected lane per epilogue warp, both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmY);
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
  const int nt = (N + 255) / 256;
  const int mt = (M + 255) / 256;
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int tiles = GROUPED ? p.n_tiles[0] * nt : mt * nt;
  const int pair = blockIdx.x / (2 * SPLIT), npairs = gridDim.x / (2 * SPLIT);
  // this pair's blocks of K
  const int kb_begin = SPLIT > 1 ? KB * part / SPLIT : 0, kb_end = SPLIT > 1 ? KB * (part + 1) / SPLIT : KB;

  if (warp >= 4) {
    regs_inc<C::EPILOGUE_REGS>();
    const int q = warp & 3, h = (warp - 4) >> 2;
    uint8_t* box = out_buf + (warp - 4) * 4096;
    const uint32_t tempty_leader[2] = {mapa_shared(smem_u32(&tempty[0]), lead), mapa_shared(smem_u32(&tempty[1]), lead)};
    const bool aligned_rows = N % (F32 ? 4 : 8) == 0;
    int buf = 0;
    uint32_t bph = 0, block = 0;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += npairs) {
      // (with COLSCALE the tile is not needed before its results are stored)
      Fp8Tile tl = {};
      if (!COLSCALE) tl = fp8_tile<GROUPED>(p, t, mt, nt, KB);
      // One block's 128 columns of the warp's rows from TMEM, 32 columns at a time (`load`) with the next
      // chunk's load under this one's arithmetic `add(chunk, values)`; the buffer is released once its
      // last chunk has landed.
      auto read_block = [&](auto&& load, auto&& add) {
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + h * 128;
        uint32_t r[2][32];
        load(taddr, r[0]);
        tmem_ld_wait32(r[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c + 1 < 4) {
            load(taddr + (c + 1) * 32, r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            // one address or two: whichever leaves all registers of that form unspilled
            if (elect_one()) mbar_arrive_cluster(COLSCALE ? tempty_leader[0] + 8 * buf : tempty_leader[buf]);
          }
          add(c, r[c & 1]);
          if (c + 1 < 4) tmem_ld_wait32(r[(c + 1) & 1]);
        }
        buf ^= 1;
        bph ^= buf == 0;
      };
      // The fp32 sums, as pairs of neighbouring columns for packed arithmetic: a lane has one row's 128
      // columns, or with COLSCALE (16 c + 8 i + 2 g + j) rows 16 i + 8 j + lane / 4, columns
      // 32 c + 8 g + 2 (lane % 4) and the next: a column's scale then comes from shared memory for four rows
      // at once.
      uint64_t acc2[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc2[i] = 0;
      if constexpr (COLSCALE) {
#pragma unroll 1
        for (int kb = kb_begin; kb < kb_end; ++kb, ++block) {
          ok = mbar_wait_warp(&tfull[buf], bph, abort_flag, wd);
          if (!ok) break;
          tc_fence_after();
          uint32_t sc = smem_u32(scale_buf) + (block & (C::SLOTS - 1)) * (C::SCALES * 4);
          float rs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) rs[i] = ld_shared_f32(sc + (256 + q * 32 + 8 * i + (lane >> 2)) * 4);
          sc += (h * 128 + 2 * (lane & 3)) * 4;
          read_block(
              [&](uint32_t at, uint32_t* d) {
                tmem_ld_frag32(at, d);
                tmem_ld_frag32(at + (16u << 16), d + 16);
              },
              [&](int c, const uint32_t* v) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  const uint64_t cs = ld_shared_b64(sc + (c * 32 + g * 8) * 4);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint32_t* x = v + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
                    uint64_t& a = acc2[16 * c + 8 * (i >> 1) + 2 * g + (i & 1)];
                    a = f2_fma(f2_mul(f2(__uint_as_float(x[0]), __uint_as_float(x[1])), cs), f2(rs[i], rs[i]), a);
                  }
                }
              });
        }
      } else {
        // this row's and the warp's column block's scale, loaded two blocks ahead of their use
        const int row = tl.m0 + rank * 128 + q * 32 + lane, col0 = tl.n0 + h * 128;
        const bool row_ok = row < tl.m_end;
        const float* sa = p.sa + row;
        const float* sb = tl.sb + static_cast<int64_t>(col0 >> 7) * KB;
        auto row_scale = [&](int kb) { return row_ok && kb < KB ? sa[static_cast<int64_t>(kb) * M] : 0.0f; };
        auto block_scale = [&](int kb) { return kb < KB && col0 < N ? sb[kb] : 0.0f; };
        float ra = row_scale(kb_begin), rb = row_scale(kb_begin + 1), ca = block_scale(kb_begin), cb = block_scale(kb_begin + 1);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          const float rs = ra * ca;
          ra = rb;
          rb = row_scale(kb + 2);
          ca = cb;
          cb = block_scale(kb + 2);
          ok = mbar_wait_warp(&tfull[buf], bph, abort_flag, wd);
          if (!ok) break;
          tc_fence_after();
          const uint64_t rs2 = f2(rs, rs);
          read_block([&](uint32_t at, uint32_t* d) { tmem_ld32(at, d); },
                     [&](int c, const uint32_t* v) {
#pragma unroll
                       for (int j = 0; j < 16; ++j) {
                         uint64_t& a = acc2[16 * c + j];
                         a = f2_fma(f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), rs2, a);
                       }
                     });
        }
      }
      if (COLSCALE) tl = fp8_tile<GROUPED>(p, t, mt, nt, KB);
      const int row0 = tl.m0 + rank * 128 + q * 32, col0 = tl.n0 + h * 128;
      if constexpr (SPLIT > 1) {
        // Every CTA's ring is free once all its roles are here: it takes the parts of the columns that
        // this CTA stores, [part][warp][4 columns][row, 16 bytes; padded so that a row's columns lie in
        // different banks]. Also after an abort (then garbage, not stored), so that the cluster's
        // barriers pair.
        constexpr int OWN = 128 / SPLIT;  // columns of each warp's 128 that a CTA stores
        constexpr int GROUP = 32 * 4 + 4, WARP_FLOATS = OWN / 4 * GROUP;
        static_assert(SPLIT * 8 * WARP_FLOATS * 4 <= STAGES * C::STAGE_BYTES, "exchange area");
        float* recv = reinterpret_cast<float*>(smem);
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int o = 0; o < SPLIT; ++o) {
          const uint32_t dst = mapa_shared(smem_u32(recv + (part * 8 + warp - 4) * WARP_FLOATS), 2 * o + rank);
#pragma unroll
          for (int c = 0; c < OWN; c += COLSCALE ? 8 : 4) {
            float v[4];
            if constexpr (COLSCALE) {
              const int column = o * OWN + c;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f2_split(acc2[16 * (column / 32) + 8 * (i >> 1) + 2 * (column % 32 / 8) + (i & 1)], v[0], v[1]);
                const int at = (c / 4 + (lane >> 1 & 1)) * GROUP + (8 * i + (lane >> 2)) * 4 + 2 * (lane & 1);
                st_shared_cluster_v2(dst + at * 4, v[0], v[1]);
              }
            } else {
              f2_split(acc2[(o * OWN + c) / 2], v[0], v[1]);
              f2_split(acc2[(o * OWN + c) / 2 + 1], v[2], v[3]);
              st_shared_cluster_v4(dst + (c / 4 * GROUP + lane * 4) * 4, v[0], v[1], v[2], v[3]);
            }
          }
        }
        __syncwarp();
        cluster_sync();
        if (ok && !*abort_flag) {
          // a row at a time (two of 32 columns), lanes along the columns, the parts added in the order of K
          constexpr int PER = F32 ? 1 : 2, LANES = OWN / PER < 32 ? OWN / PER : 32;  // columns a lane, lanes a row
          const int c_first = col0 + part * OWN;
          const bool paired = N % 2 == 0;
#pragma unroll 4
          for (int r = lane / LANES; r < 32; r += 32 / LANES) {
            if (row0 + r >= tl.m_end) continue;
            const int64_t at = static_cast<int64_t>(row0 + r) * N + c_first;
#pragma unroll
            for (int c0 = 0; c0 < OWN; c0 += LANES * PER) {
              const int c = c0 + (lane % LANES) * PER;
              const float* src = recv + (warp - 4) * WARP_FLOATS + (c >> 2) * GROUP + r * 4 + (c & 3);
              float v[PER];
#pragma unroll
              for (int j = 0; j < PER; ++j) v[j] = 0.0f;
#pragma unroll
              for (int s = 0; s < SPLIT; ++s)
#pragma unroll
                for (int j = 0; j < PER; ++j) v[j] += src[s * 8 * WARP_FLOATS + j];
              if constexpr (F32) {
                if (c_first + c < N) static_cast<float*>(p.y)[at + c] = v[0];
              } else {
                const uint32_t w = pack_bf16x2(v[0], v[1]);
                uint16_t* y = static_cast<uint16_t*>(p.y) + at + c;
                if (paired) {
                  if (c_first + c < N) *reinterpret_cast<uint32_t*>(y) = w;
                } else {
                  if (c_first + c < N) y[0] = static_cast<uint16_t>(w & 0xFFFFu);
                  if (c_first + c + 1 < N) y[1] = static_cast<uint16_t>(w >> 16);
                }
              }
            }
          }
        }
        break;
      }
      if (!ok) break;
      // results to y; a grouped tile that ends inside the box's rows must not touch the next expert's
      const bool by_tma = aligned_rows && (!GROUPED || row0 + 32 <= tl.m_end);
      if (row0 < tl.m_end) {
#pragma unroll
        for (int b = 0; b < (F32 ? 4 : 2); ++b) {
          const int c0 = col0 + b * (F32 ? 32 : 64);
          if (c0 < N) {
            // 16-byte piece c of row r at c ^ (r % 8)
            auto fill = [&](uint32_t to) {
              if constexpr (COLSCALE) {
#pragma unroll
                for (int g = 0; g < (F32 ? 4 : 8); ++g)  // eight columns
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int column = b * (F32 ? 32 : 64) + 8 * g, r = 8 * i + (lane >> 2);
                    float lo, hi;
                    f2_split(acc2[16 * (column / 32) + 8 * (i >> 1) + 2 * (column % 32 / 8) + (i & 1)], lo, hi);
                    if (F32)
                      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(
                                       to + r * 128 + (((2 * g + (lane >> 1 & 1)) ^ (r & 7)) << 4) + (lane & 1) * 8),
                                   "f"(lo), "f"(hi)
                                   : "memory");
                    else
                      asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + r * 128 + ((g ^ (r & 7)) << 4) + (lane & 3) * 4),
                                   "r"(pack_bf16x2(lo, hi))
                                   : "memory");
                  }
              } else {
                uint32_t w[32];  // fp32: column 32 b + j; bf16: columns 64 b + 2 j and the next
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  float lo, hi;
                  f2_split(acc2[F32 ? 16 * b + j / 2 : 32 * b + j], lo, hi);
                  w[j] = F32 ? __float_as_uint((j & 1) ? hi : lo) : pack_bf16x2(lo, hi);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + lane * 128 + ((c ^ (lane & 7)) << 4)),
                               "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                               : "memory");
              }
            };
            fp8_store_box<F32>(p, box, fill, &tmY, by_tma, row0, tl.m_end, c0, N);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group0();  // this warp's stores are complete before the CTA exits
    __syncwarp();
  } else {
    regs_dec<C::CONTROL_REGS>();
    if (warp == 0) {
      const uint64_t pol = policy_evict_last();
      int s = 0;
      uint32_t ph = 0;
      uint32_t used = 0, phases = 0;  // per stage: requested at all, phase of the last request
      int issued = 0;
      for (int t = pair; t < tiles && !*abort_flag; t += npairs) {
        const Fp8Tile tl = fp8_tile<GROUPED>(p, t, mt, nt, KB);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_warp(&empty[s], ph ^ 1, abort_flag, wd)) break;
          // test hook: the first CTA withholds its expect-tx arrival and loads
          const bool withheld = blockIdx.x == 0 && ++issued == p.drop_stage;
          if (!withheld && elect_one()) {
            uint8_t* st = smem + s * C::STAGE_BYTES;
            const uint32_t bar = mapa_shared(smem_u32(&full[s]), lead);
            if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
            tma_load_2d_pair(st, &tmA, bar, kb * 128, tl.m0 + rank * 128, pol);
            tma_load_2d_pair(st + C::TILE_BYTES, &tmB, bar, kb * 128, tl.b_row + rank * 128, pol);
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
    } else if (warp == 1) {
      if (leader) {
        const uint32_t idesc = idesc_e4m3(256, 256);
        int s = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        for (int t = pair; t < tiles && !*abort_flag; t += npairs) {
          for (int kb = kb_begin; kb < kb_end; ++kb) {
            // the operands first: they normally wait, so that the issue follows the buffer's release
            if (!mbar_wait_warp(&full[s], ph, abort_flag, wd)) break;
            if (!mbar_wait_warp(&tempty[buf], bph ^ 1, abort_flag, wd)) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t a_addr = smem_u32(smem + s * C::STAGE_BYTES);
              const uint64_t adesc = desc_sw128(a_addr), bdesc = desc_sw128(a_addr + C::TILE_BYTES);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_f8_pair(tmem + buf * 256, adesc + 2 * kk, bdesc + 2 * kk, idesc, kk != 0);
              tc_commit_pair(&empty[s], 3u << lead);
              tc_commit_pair(&tfull[buf], 3u << lead);
            }
            __syncwarp();
            if (++s == STAGES) {
              s = 0;
              ph ^= 1;
            }
            buf ^= 1;
            bph ^= buf == 0;
          }
        }
        if (elect_one()) tc_commit_pair(drain, 1u << lead);
        __syncwarp();
        volatile int32_t dummy = 0;
        mbar_wait_warp(drain, 0, &dummy, wd);
      }
    } else if (COLSCALE && warp == 2) {
      // The scales: loaded AHEAD blocks before they are written to shared memory, written one block
      // before they are announced, on the barrier that the block's MMA completes.
      constexpr int AHEAD = 3;
      int t = pair, kb = kb_begin;
      float v[AHEAD][12];
      bool have[AHEAD];
      Fp8Tile tl = {};
      auto request = [&](int i) {
        have[i] = t < tiles;
        if (!have[i]) return;
        if (kb == kb_begin) tl = fp8_tile<GROUPED>(p, t, mt, nt, KB);
        const int col = tl.n0 + lane, row = tl.m0 + rank * 128 + lane;
        const float* sb = tl.sb + static_cast<int64_t>(kb) * N + col;
        const float* sa = p.sa + static_cast<int64_t>(kb) * M + row;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = col + 32 * j < N ? sb[32 * j] : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][8 + j] = row + 32 * j < tl.m_end ? sa[32 * j] : 0.0f;
        if (++kb == kb_end) {
          kb = kb_begin;
          t += npairs;
        }
      };
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) request(i);
      uint32_t block = 0;
      bool go = true, written = false;
      while (go) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (!go) break;
          if (written) {  // announce block - 1, after the block two before it is complete
            const uint32_t b = block - 1;
            if (b >= 2) go = mbar_wait_warp(&tfull[b & 1], (b >> 1 & 1) ^ 1, abort_flag, wd);
            __syncwarp();
            if (go && lane == 0) mbar_arrive(&tfull[b & 1]);
          }
          written = have[i];
          go = go && written;
          if (written) {
            float* d = scale_buf + (block & (C::SLOTS - 1)) * C::SCALES + lane;
#pragma unroll
            for (int j = 0; j < 12; ++j) d[32 * j] = v[i][j];
          }
          ++block;
          request(i);
        }
      }
    }
    if constexpr (SPLIT > 1) {  // the epilogue warps' two barriers around the exchange of the parts
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
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

// ---- grouped preparation ------------------------------------------------------------------------

// One CTA: checks 0 = offsets[0] <= ... <= offsets[E] <= M and lists the token tiles, (expert, first
// row, rows) with at most tile_rows rows of one expert each; experts without rows get none.
// Malformed offsets are reported and leave an empty list.
__global__ void __launch_bounds__(1024) k_fp8_tiles(const int32_t* offsets, int E, int M, int tile_rows, int4* tiles,
                                                    int32_t* n_tiles, int32_t* status) {
  __shared__ int32_t wsum[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // thread i owns a contiguous run of experts
  const int per = (E + 1023) / 1024;
  const int e0 = min(E, static_cast<int>(threadIdx.x) * per), e1 = min(E, e0 + per);
  bool good = true;
  int mine = 0;
  if (threadIdx.x == 0) good = offsets[0] == 0 && offsets[E] <= M;
  for (int e = e0; e < e1; ++e) {
    const int a = offsets[e], b = offsets[e + 1];
    good = good && a >= 0 && a <= b && b <= M;
    if (good) mine += (b - a + tile_rows - 1) / tile_rows;
  }
  good = __syncthreads_and(good) != 0;
  if (!good) {
    if (threadIdx.x == 0) {
      *n_tiles = 0;
      report_status(status, kStatusBadOffsets);
    }
    return;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  int at = before + incl - mine;
  for (int e = e0; e < e1; ++e) {
    const int a = offsets[e], b = offsets[e + 1];
    for (int r = a; r < b; r += tile_rows) tiles[at++] = make_int4(e, r, min(tile_rows, b - r), 0);
  }
  if (threadIdx.x == 0) *n_tiles = total;
}

// ---- host launchers -------------------------------------------------------------------------------

cudaError_t launch_fp8_tiles(const int32_t* offsets, int E, int M, int tile_rows, int4* tiles, int32_t* n_tiles,
                             int32_t* status, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_fp8_tiles, offsets, E, M, tile_rows, tiles, n_tiles, status);
}

template <bool COLSCALE, bool F32>
static auto pick_fp8_pair(int split) -> void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Fp8GemmArgs) {
  return split == 4 ? k_fp8_gemm_pair<COLSCALE, false, F32, 4>
                    : (split == 2 ? k_fp8_gemm_pair<COLSCALE, false, F32, 2> : k_fp8_gemm_pair<COLSCALE, false, F32, 1>);
}

cudaError_t launch_fp8_gemm_pair(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmY,
                                 const Fp8GemmArgs& p, int grid, cudaStream_t st) {
  void (*kernel)(CUtensorMap, CUtensorMap, CUtensorMap, Fp8GemmArgs);
  if (p.tiles)
    kernel = k_fp8_gemm_pair<false, true, false, 1>;
  else if (p.b_rows == 1)
    kernel = p.f32 ? pick_fp8_pair<true, true>(p.split) : pick_fp8_pair<true, false>(p.split);
  else
    kernel = p.f32 ? pick_fp8_pair<false, true>(p.split) : pick_fp8_pair<false, false>(p.split);
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Fp8PairCfg::THREADS);
  cfg.dynamicSmemBytes = Fp8PairCfg::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.tiles ? 2 : 2 * p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, tmY, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace nvfp4

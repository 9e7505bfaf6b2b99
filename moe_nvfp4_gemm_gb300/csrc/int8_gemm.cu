// Product of 8-bit integers with a scale for each token and each channel:
//   y[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k],  the sum exact.
//
// sm_103a has no integer kind of tcgen05.mma, and mma.sync multiplies integers at 158 TOP/s (fp16 at 603): 16 tokens on
// 8,192 x 8,192 would take 13.6 us, the weights' bytes 9.9. So the sums run through kind::f16: an 8-bit integer is exact in
// fp16, a product of two in fp32, and a sum of 1,024 products, at most 1,024 * 128^2 = 2^24, too. After every
// 1,024 of K (a chunk) the epilogue warps read the sums back, convert them and add them as 32-bit integers.
//
// A CTA pair (cta_group::2) takes 256 channels as the MMA's M and NT tokens as N. The weights stay 8-bit integers up
// to the SM: a TMA ring brings blocks of 128 of K, and a warpgroup turns each channel's 128 bytes into
// fp16 in registers (byte order 0x64uu is 1024 + u; u = b + 128; minus 1152) and stores them to TMEM, from
// where the MMA takes its A operand: the fp16 weights never pass through shared memory, whose bandwidth
// they would fill. Tokens: up to 128 are converted by the same warps into the swizzled shared-memory tile that the
// MMA reads; tiles of 256 come as fp16 from the workspace, converted once by k_int8_widen.
//
// Up to 8 tokens have a kernel without tensor cores (int8_few.cu). Few tiles: the pairs of a cluster (p.split of them)
// sum a tile's parts of K, exchange the integer sums through distributed shared memory and store a share of the tokens each.
//
// Bound by the tensor cores with many tokens (4,096 x 28,672 x 8,192: 0.99 ms, 1.94 PFLOP/s, the fp16 rate; under the power
// cap 1.06), by the loop around a block with few (9 tokens, 8,192 x 8,192: 17.4 us, 3.9 TB/s of weights).
#include <stdint.h>

#include <cuda_fp16.h>

#include <type_traits>

#include "ffn.cuh"
#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

template <int NT>
struct Int8Cfg {
  // warps 0-3: producer of the 8-bit operands, MMA issuer, WIDE: the tokens' producer, idle; then one or two
  // warpgroups that convert, two or one of epilogue warps. 512 x 128 registers at launch.
  static constexpr int THREADS = 512;
  static constexpr bool WIDE = NT == 256;  // tokens come as fp16
  // Converting groups take blocks in turn. Few tokens: bound by the weights' bytes, a block of 16 KB in about 700
  // cycles; a group needs about 600 for the weights and up to 300 for the tokens. With 256 tokens a block's MMAs
  // take 1,024 cycles and one group is enough.
  static constexpr int CONV_GROUPS = WIDE ? 1 : 2;
  static constexpr int EPI_WARP = 4 + 4 * CONV_GROUPS;  // first epilogue warp
  static constexpr int EPI_WARPS = 16 - EPI_WARP;
  static constexpr int CONTROL_REGS = WIDE ? 80 : 96, EPILOGUE_REGS = WIDE ? 176 : 200;
  static_assert(32 * EPI_WARP * CONTROL_REGS + 32 * EPI_WARPS * EPILOGUE_REGS <= 512 * 128, "register shares");
  static constexpr int XROWS = NT / 2;                  // token rows of a CTA
  static constexpr int W_BYTES = 128 * 128;             // 128 channels x 128 of K
  static constexpr int RAW_BYTES = W_BYTES + (WIDE ? 0 : XROWS * 128);
  static constexpr int RAW = WIDE ? 4 : (NT == 128 ? 5 : 7);  // stages of 8-bit operands
  // TMEM: the sums, then A in OPS operand blocks of 128 of K (64 columns). Up to 128 tokens: two buffers of NT columns, a
  // chunk each. 256: three slots of 128 columns; chunks take slots 0, 1 and 1, 2 in turn, the first half of the tokens in the
  // lower one, so that a chunk's first blocks can be summed into the free slot while slot 1 is still read.
  static constexpr int HALVES = WIDE ? 2 : 1, HALF = NT / HALVES, BUFS = WIDE ? 3 : 2;
  // (Operand blocks of 64 of K in WIDE, four of them, made prefill 1,550 us instead of 1,000: a block's hand-overs
  // between converter and MMA cost as much as those of a block of 128.)
  static constexpr int OPS = WIDE ? 2 : 4;
  static constexpr int APART = WIDE ? 2 : 0;  // a chunk's first blocks, summed half by half
  static constexpr int A_COL = BUFS * HALF;
  static_assert(A_COL + 64 * OPS <= 512 && APART <= OPS, "TMEM columns");
  static constexpr int XS = 4;                          // tokens' fp16 tiles of 128 of K
  static constexpr int X_BYTES = XROWS * 256;           // two boxes of XROWS x 64 of K, fp16
  static constexpr int CHUNK = 8;                       // blocks of 128 between two readings of the sums
  static constexpr int COLS = NT * 4 / EPI_WARPS;       // tokens of an epilogue warp
  static constexpr int OUT_BYTES = EPI_WARPS * 4096;    // a box for each epilogue warp
  static constexpr int SMEM_BYTES = RAW * RAW_BYTES + XS * X_BYTES + OUT_BYTES + 1024 + 512;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  // Split sums: tokens that a CTA stores, in groups of eight; the area of a CTA's sums.
  __host__ __device__ static constexpr int own(int split) { return (NT / 8 + split - 1) / split * 8; }
  static_assert(NT * 132 * 4 <= RAW * RAW_BYTES + XS * X_BYTES, "exchange area");
};

struct Int8Tile {
  int m0, n0;
};

DEVI Int8Tile int8_tile(const Int8GemmArgs& p, int t, int nt_tokens) {
  int mb, nb;
  tile_coords(t, p.mt, p.nt, p.raster, mb, nb);
  return {mb * nt_tokens, nb * 256};
}

// Four bytes, signed, as two pairs of fp16.
DEVI void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;  // b + 128
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<uint32_t*>(&x);
  hi = *reinterpret_cast<uint32_t*>(&y);
}

DEVI uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

template <int NT, int OUT>
__global__ void __launch_bounds__(Int8Cfg<NT>::THREADS, 1)
    k_int8_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ Int8GemmArgs p) {
  using C = Int8Cfg<NT>;
  constexpr bool WIDE = C::WIDE;
  constexpr int RAW = C::RAW, OPS = C::OPS, BUFS = C::BUFS, XS = C::XS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* x_buf = smem + RAW * C::RAW_BYTES;
  uint8_t* out_buf = x_buf + XS * C::X_BYTES;
  uint64_t* rfull = reinterpret_cast<uint64_t*>(out_buf + C::OUT_BYTES);  // [RAW] 8-bit operands have landed
  uint64_t* rempty = rfull + RAW;                                         // [RAW] and have been read
  uint64_t* ofull = rempty + RAW;   // [OPS] converted operands are in place (leader)
  uint64_t* oempty = ofull + OPS;   // [OPS] and have been used
  uint64_t* xfull = oempty + OPS;   // [XS] WIDE: the tokens' tile has landed (leader)
  uint64_t* xempty = xfull + XS;    // [XS] and has been used
  uint64_t* tfull = xempty + XS;    // [BUFS] a chunk's sums are complete
  uint64_t* tempty = tfull + BUFS;  // [BUFS] and have been read (leader)
  uint64_t* drain = tempty + BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wd = p.watchdog_ns;
  const int split = p.split;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
  const int part = static_cast<int>(crank >> 1);
  const bool leader = rank == 0;  // issues the pair's MMAs
  if (threadIdx.x == 0) {
    for (int s = 0; s < RAW; ++s) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], 4);  // the converting group's warps
    }
    for (int s = 0; s < OPS; ++s) {
      mbar_init(&ofull[s], 8);  // the converting groups' warps of both CTAs
      mbar_init(&oempty[s], 1);
    }
    for (int s = 0; s < XS; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int b = 0; b < BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * C::EPI_WARPS);  // one elected lane per epilogue warp, both CTAs
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
  const int KB = static_cast<int>((p.K + 127) / 128);
  const int kb_begin = static_cast<int>(static_cast<int64_t>(KB) * part / split);
  const int kb_end = static_cast<int>(static_cast<int64_t>(KB) * (part + 1) / split);
  const int tiles = p.mt * p.nt;
  const int first = blockIdx.x / (2 * split), step = gridDim.x / (2 * split);

  if (warp >= C::EPI_WARP) {
    regs_inc<C::EPILOGUE_REGS>();
    const int q = warp & 3, h = (warp - C::EPI_WARP) >> 2;
    uint8_t* box = out_buf + (warp - C::EPI_WARP) * 4096;
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), lead);
    uint32_t chunk = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const Int8Tile tl = int8_tile(p, t, NT);
      const int own = C::own(split);  // split: tokens that this CTA stores
      // first token: of the CTA's own after the exchange; of 32 tokens c of this warp
      const int own0 = tl.m0 + part * own;
      auto row_of = [&](int c) {
        return tl.m0 + (WIDE ? (c >> 1) * 128 + h * 64 + (c & 1) * 32 : c * 32);
      };
      const int col0 = tl.n0 + static_cast<int>(rank) * 128 + q * 32;
      // A lane holds the scales of tokens 32 c + lane of those that its warp stores, and of channel `lane` of the
      // warp's 32: requested here, so that no load waits behind the sums.
      constexpr int SA = NT / 32 < 4 ? NT / 32 : 4;
      float sa[SA];
#pragma unroll
      for (int c = 0; c < SA; ++c) {
        const int m = (split > 1 ? own0 + 32 * c : row_of(c)) + lane;
        sa[c] = m < M ? p.sa[m] : 0.0f;
      }
      const float sb_lane = col0 + lane < N ? p.sb[col0 + lane] : 0.0f;
      float sb4[4] = {};  // split: of four of the CTA's 128
      if (split > 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = tl.n0 + static_cast<int>(rank) * 128 + 4 * lane + k;
          if (n < N) sb4[k] = p.sb[n];
        }
      }
      // acc[32 c + 16 i + 4 g + 2 j + u]: channel 16 i + 8 j + lane / 4 of the warp's 32, token
      // row_of(c) + 8 g + 2 (lane % 4) + u
      int acc[C::COLS];
#pragma unroll
      for (int i = 0; i < C::COLS; ++i) acc[i] = 0;
      constexpr int PARTS = C::COLS / 32 / C::HALVES;  // of 32 tokens in a buffer
#pragma unroll 1
      for (int kb = kb_begin; kb < kb_end && ok; kb += C::CHUNK, ++chunk) {
        // WIDE: slot 1 first, which the next chunk waits for: this one's second half, then (odd chunks) its first
        auto read = [&](auto half_, int slot, uint32_t phase) {
          constexpr int half = decltype(half_)::value;
          if (!ok) return;
          ok = mbar_wait_warp(&tfull[slot], phase, abort_flag, wd);
          if (!ok) return;
          tc_fence_after();
          const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + slot * C::HALF + h * (32 * PARTS);
#pragma unroll
          for (int c = 0; c < PARTS; ++c) {
            uint32_t r[32];
            tmem_ld_frag32(at + c * 32, r);
            tmem_ld_frag32(at + c * 32 + (16u << 16), r + 16);
            tmem_ld_wait32(r);
            if (c + 1 == PARTS) {
              tc_fence_before();
              __syncwarp();
              if (elect_one()) mbar_arrive_cluster(tempty_leader + 8 * slot);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[32 * (half * PARTS + c) + j] += __float2int_rn(__uint_as_float(r[j]));
          }
        };
        constexpr std::integral_constant<int, 0> lower;
        if constexpr (WIDE) {
          constexpr std::integral_constant<int, 1> upper;
          if ((chunk & 1) == 0) {
            read(upper, 1, chunk & 1);
            read(lower, 0, chunk >> 1 & 1);
          } else {
            read(lower, 1, chunk & 1);
            read(upper, 2, chunk >> 1 & 1);
          }
        } else {
          read(lower, chunk & 1, chunk >> 1 & 1);
        }
      }
      if (split > 1) {
        // Every CTA's sums go to its own shared memory, [token][132] in the place of the operand rings (its roles are
        // done with them: the last tfull followed all MMAs, and those all loads), and each CTA then reads the parts of
        // the tokens that it stores, [part, part + 1) own, from the others, a row of 128 channels at once. Also after an
        // abort (then garbage, not stored), so that the cluster's barriers pair.
        const uint32_t sums = smem_u32(smem);
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int c = 0; c < C::COLS / 32; ++c)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int tok8 = row_of(c) - tl.m0 + 8 * g;
            if (tl.m0 + tok8 >= M) continue;
            const uint32_t at = sums + ((tok8 + 2 * (lane & 3)) * 132 + q * 32 + (lane >> 2)) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (u * 132 + 8 * i) * 4),
                             "r"(acc[32 * c + 16 * (i >> 1) + 4 * g + 2 * (i & 1) + u])
                             : "memory");
          }
        __syncwarp();
        cluster_sync();
        if (ok && !*abort_flag) {
          // a lane: four channels; a warp: every EPI_WARPS-th token, four at a time with all their parts in flight
          const int n = tl.n0 + static_cast<int>(rank) * 128 + 4 * lane;
          const int rows = min(min(own, NT - part * own), M - own0);
          uint32_t from[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) from[s] = mapa_shared(sums + (part * own * 132 + 4 * lane) * 4, 2 * min(s, split - 1) + rank);
          const bool whole = N % 4 == 0 && n < N;  // 16 or 8 bytes at once
#pragma unroll
          for (int c = 0; c < SA; ++c)
#pragma unroll 1
            for (int j0 = warp - C::EPI_WARP; j0 < 32; j0 += 4 * C::EPI_WARPS) {
              if (32 * c + j0 >= rows) break;
              int4 v[4][4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                  // (a row past the last is read inside the tile and not stored)
                  v[j][s] = make_int4(0, 0, 0, 0);
                  if (s < split) v[j][s] = ld_shared_cluster_v4(from[s] + min(32 * c + j0 + j * C::EPI_WARPS, rows - 1) * (132 * 4));
                }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float sa_j = __shfl_sync(0xffffffffu, sa[c], j0 + j * C::EPI_WARPS);
                const int i = 32 * c + j0 + j * C::EPI_WARPS;
                const float f[4] = {static_cast<float>(v[j][0].x + v[j][1].x + v[j][2].x + v[j][3].x) * sa_j * sb4[0],
                                    static_cast<float>(v[j][0].y + v[j][1].y + v[j][2].y + v[j][3].y) * sa_j * sb4[1],
                                    static_cast<float>(v[j][0].z + v[j][1].z + v[j][2].z + v[j][3].z) * sa_j * sb4[2],
                                    static_cast<float>(v[j][0].w + v[j][1].w + v[j][2].w + v[j][3].w) * sa_j * sb4[3]};
                if (i >= rows) continue;
                const int64_t to = static_cast<int64_t>(own0 + i) * N + n;
                if (OUT == kInt8OutF32) {
                  float* y = static_cast<float*>(p.y) + to;
                  if (whole)
                    *reinterpret_cast<float4*>(y) = make_float4(f[0], f[1], f[2], f[3]);
                  else
                    for (int k = 0; k < 4; ++k)
                      if (n + k < N) y[k] = f[k];
                } else {
                  constexpr bool H = OUT == kInt8OutF16;
                  uint16_t* y = static_cast<uint16_t*>(p.y) + to;
                  const uint2 w = make_uint2(pack16<H>(f[0], f[1]), pack16<H>(f[2], f[3]));
                  if (whole) {
                    *reinterpret_cast<uint2*>(y) = w;
                  } else {
                    for (int k = 0; k < 4; ++k)
                      if (n + k < N) y[k] = static_cast<uint16_t>((k < 2 ? w.x : w.y) >> (k & 1 ? 16 : 0));
                  }
                }
              }
            }
        }
        break;
      }
      if (!ok) break;
      if (col0 < N) {
        float sb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sb[i] = __shfl_sync(0xffffffffu, sb_lane, 8 * i + (lane >> 2));
        // 32 tokens x 32 channels at a time through the warp's box (rows of odd lengths are stored value by value, eight
        // tokens under way: 4,925 x 14,555 x 512 122 -> 115 us)
#pragma unroll
        for (int c = 0; c < C::COLS / 32; ++c) {
          const int row0 = row_of(c), rows = min(32, M - row0);
          if (rows <= 0) continue;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float sa0 = __shfl_sync(0xffffffffu, sa[c], 8 * g + 2 * (lane & 3));
            const float sa1 = __shfl_sync(0xffffffffu, sa[c], 8 * g + 2 * (lane & 3) + 1);
            float v[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int* s = acc + 32 * c + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
              v[i][0] = static_cast<float>(s[0]) * sa0 * sb[i];
              v[i][1] = static_cast<float>(s[1]) * sa1 * sb[i];
            }
            if (OUT == kInt8OutF32) {
              // [token][32 channels]: 16-byte piece j of token t at j ^ (t % 8)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const int tok = 8 * g + 2 * (lane & 3) + u, ch = 8 * i + (lane >> 2);
                  reinterpret_cast<float*>(box)[tok * 32 + (((ch >> 2) ^ (tok & 7)) << 2) + (ch & 3)] = v[i][u];
                }
            } else {
              // [token][32 channels], 16-byte piece j of token t at j ^ (t / 2 % 4)
              const uint32_t to = smem_u32(box) + (lane & 7) * 64 + (((lane >> 3) ^ (lane >> 1 & 3)) << 4);
              constexpr bool H = OUT == kInt8OutF16;
              st_matrix_x4_trans(to + g * 512, pack16<H>(v[0][0], v[0][1]), pack16<H>(v[1][0], v[1][1]),
                                 pack16<H>(v[2][0], v[2][1]), pack16<H>(v[3][0], v[3][1]));
            }
          }
          __syncwarp();
          const int64_t at = static_cast<int64_t>(row0) * N + col0;
          if (OUT == kInt8OutF32) {
            float* y = static_cast<float*>(p.y) + at;
            if (N % 4 == 0) {  // 16 bytes a lane, four tokens at a time
              if (col0 + 4 * (lane & 7) < N)
                for (int i = lane >> 3; i < rows; i += 4)
                  *reinterpret_cast<uint4*>(y + static_cast<int64_t>(i) * N + 4 * (lane & 7)) =
                      *reinterpret_cast<const uint4*>(box + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
            } else if (col0 + lane < N) {
#pragma unroll 8
              for (int i = 0; i < rows; ++i)
                y[static_cast<int64_t>(i) * N + lane] =
                    reinterpret_cast<const float*>(box)[i * 32 + (((lane >> 2) ^ (i & 7)) << 2) + (lane & 3)];
            }
          } else {
            uint16_t* y = static_cast<uint16_t*>(p.y) + at;
            if (N % 8 == 0) {  // 16 bytes a lane, eight tokens at a time
              if (col0 + 8 * (lane & 3) < N)
                for (int i = lane >> 2; i < rows; i += 8)
                  *reinterpret_cast<uint4*>(y + static_cast<int64_t>(i) * N + 8 * (lane & 3)) =
                      *reinterpret_cast<const uint4*>(box + i * 64 + (((lane & 3) ^ (i >> 1 & 3)) << 4));
            } else if (col0 + lane < N) {
#pragma unroll 8
              for (int i = 0; i < rows; ++i)
                y[static_cast<int64_t>(i) * N + lane] =
                    reinterpret_cast<const uint16_t*>(box)[i * 32 + (((lane >> 3) ^ (i >> 1 & 3)) << 3) + (lane & 7)];
            }
          }
          __syncwarp();
        }
      }
    }
  } else {
    regs_dec<C::CONTROL_REGS>();
    if (warp == 0) {
      const uint64_t pol_w = p.mt == 1 ? policy_evict_first() : policy_evict_last(), pol_x = policy_evict_last();
      int s = 0, issued = 0;
      uint32_t ph = 0;
      uint32_t used = 0, phases = 0;  // per stage: requested at all, phase of the last request
      for (int t = first; t < tiles && !*abort_flag; t += step) {
        const Int8Tile tl = int8_tile(p, t, NT);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_warp(&rempty[s], ph ^ 1, abort_flag, wd)) break;
          // test hook: the first CTA withholds its expect-tx arrival and loads
          const bool withheld = blockIdx.x == 0 && ++issued == p.drop_stage;
          if (!withheld && elect_one()) {
            uint8_t* st = smem + s * C::RAW_BYTES;
            mbar_arrive_expect_tx(&rfull[s], C::RAW_BYTES);
            tma_load_2d(st, &tmW, &rfull[s], kb * 128, tl.n0 + rank * 128, pol_w);
            if (!WIDE) tma_load_2d(st + C::W_BYTES, &tmX, &rfull[s], kb * 128, tl.m0 + rank * C::XROWS, pol_x);
          }
          __syncwarp();
          used |= 1u << s;
          phases = (phases & ~(1u << s)) | ph << s;
          if (++s == RAW) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      griddep_launch_dependents();
      for (int i = 0; i < RAW; ++i)  // this warp's copies in flight land before the CTA leaves
        if (used >> i & 1) {
          volatile int32_t dummy = 0;
          mbar_wait_warp(&rfull[i], phases >> i & 1, &dummy, wd);
        }
    } else if (warp == 1) {
      if (leader) {
        int s = 0, x = 0;
        uint32_t ph = 0, xph = 0, chunk = 0;
        if constexpr (!WIDE) {
          // A block's MMAs take 256 to 512 cycles: the loop around them is kept short.
          constexpr uint32_t idesc = idesc_f16(256, NT, false);
          const uint64_t xdesc = desc_sw128(smem_u32(x_buf));
          const uint32_t a_tmem = tmem + C::A_COL;
          for (int t = first; t < tiles && !*abort_flag; t += step) {
            int left = C::CHUNK;  // blocks of this chunk
            for (int kb = kb_begin; kb < kb_end; ++kb) {
              const uint32_t slot = chunk & 1;
              if (!mbar_wait_warp(&ofull[s], ph, abort_flag, wd)) break;
              if (left == C::CHUNK && !mbar_wait_warp(&tempty[slot], (chunk >> 1 & 1) ^ 1, abort_flag, wd)) break;
              tc_fence_after();
              const bool last = left == 1 || kb + 1 == kb_end;
              if (elect_one()) {
                const uint64_t xd = xdesc + static_cast<uint32_t>(s * (C::X_BYTES >> 4));
                const uint32_t at = a_tmem + s * 64, dt = tmem + slot * NT;
                const uint32_t more = left != C::CHUNK;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  tc_mma_f16_pair_ts(dt, at + kk * 8, xd + ((kk >> 2) * (C::X_BYTES >> 5) + 2 * (kk & 3)), idesc, kk == 0 ? more : 1);
                tc_commit_pair(&oempty[s], 3u << lead);
                if (last) tc_commit_pair(&tfull[slot], 3u << lead);
              }
              __syncwarp();
              s = (s + 1) & (OPS - 1);
              ph ^= s == 0;
              --left;
              if (last) {
                left = C::CHUNK;
                ++chunk;
              }
            }
          }
        } else {
          for (int t = first; t < tiles && !*abort_flag; t += step) {
            for (int kb = kb_begin; kb < kb_end;) {
              const int in_chunk = (kb - kb_begin) % C::CHUNK;
              // a chunk's first operand blocks are summed half by half, the one in the free slot first, so that
              // slot 1, which may still be read, is needed 1,024 cycles later; the others both halves at once.
              const bool apart = in_chunk == 0;
              const int n = apart ? min(C::APART, kb_end - kb) : 1;
              const int low = static_cast<int>(chunk & 1);  // slot of the first column
              const uint32_t idesc = idesc_f16(256, apart ? C::HALF : NT, false);
              bool go = true;
              int bs = s, bx = x;
              uint32_t bsph = ph, bxph = xph;
              for (int pass = 0; pass < (apart ? 2 : 1) && go; ++pass) {
                // apart: the half in slot 0 or 2, then the other in slot 1
                const int half = apart ? (pass == 0 ? low : low ^ 1) : 0;
                if (in_chunk == 0) {
                  const int slot = low + half;
                  const uint32_t use = slot == 1 ? chunk : chunk >> 1;  // uses of this slot before
                  go = mbar_wait_warp(&tempty[slot], (use & 1) ^ 1, abort_flag, wd);
                }
                bs = s, bx = x, bsph = ph, bxph = xph;
                for (int b = 0; b < n && go; ++b) {
                  if (pass == 0) {
                    go = mbar_wait_warp(&ofull[bs], bsph, abort_flag, wd);
                    go = go && mbar_wait_warp(&xfull[bx], bxph, abort_flag, wd);
                    if (!go) break;
                  }
                  tc_fence_after();
                  const bool last = in_chunk + b == C::CHUNK - 1 || kb + b + 1 == kb_end;
                  if (elect_one()) {
                    // rows of this half in each CTA's tile: the MMA's N is split between the CTAs
                    const uint32_t xa = smem_u32(x_buf + bx * C::X_BYTES) + half * (C::HALF / 2) * 128;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                      tc_mma_f16_pair_ts(tmem + (low + half) * C::HALF, tmem + C::A_COL + bs * 64 + kk * 8,
                                         desc_sw128(xa + (kk >> 2) * (C::X_BYTES / 2)) + 2 * (kk & 3), idesc,
                                         in_chunk + b != 0 || kk != 0);
                    if (!apart || pass == 1) {
                      tc_commit_pair(&oempty[bs], 3u << lead);
                      tc_commit_pair(&xempty[bx], 3u << lead);
                      if (last) {
                        tc_commit_pair(&tfull[low], 3u << lead);
                        tc_commit_pair(&tfull[low + 1], 3u << lead);
                      }
                    }
                  }
                  __syncwarp();
                  if (++bs == OPS) {
                    bs = 0;
                    bsph ^= 1;
                  }
                  if (++bx == XS) {
                    bx = 0;
                    bxph ^= 1;
                  }
                }
              }
              if (!go) break;
              s = bs, x = bx, ph = bsph, xph = bxph;
              kb += n;
              if (in_chunk + n == C::CHUNK || kb == kb_end) ++chunk;
            }
          }
        }
        if (elect_one()) tc_commit_pair(drain, 1u << lead);
        __syncwarp();
        volatile int32_t dummy = 0;
        mbar_wait_warp(drain, 0, &dummy, wd);
      }
    } else if (WIDE && warp == 2) {
      const uint64_t pol = policy_evict_last();
      int s = 0;
      uint32_t ph = 0;
      uint32_t used = 0, phases = 0;
      for (int t = first; t < tiles && !*abort_flag; t += step) {
        const Int8Tile tl = int8_tile(p, t, NT);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!mbar_wait_warp(&xempty[s], ph ^ 1, abort_flag, wd)) break;
          if (elect_one()) {
            uint8_t* st = x_buf + s * C::X_BYTES;
            const uint32_t bar = mapa_shared(smem_u32(&xfull[s]), lead);
            if (leader) mbar_arrive_expect_tx(&xfull[s], 2 * C::X_BYTES);
            // [64 of K][two boxes of 64 tokens]. The MMA takes the even CTA's rows as its first columns: 128 of 256,
            // or 64 of 128 where the halves are summed apart.
            const bool apart = (kb - kb_begin) % C::CHUNK < C::APART;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tma_load_2d_pair(st + i * (C::X_BYTES / 4), &tmX, bar, kb * 128 + (i >> 1) * 64,
                               tl.m0 + (apart ? (i & 1) * 128 + static_cast<int>(rank) * 64 : static_cast<int>(rank) * 128 + (i & 1) * 64),
                               pol);
          }
          __syncwarp();
          used |= 1u << s;
          phases = (phases & ~(1u << s)) | ph << s;
          if (++s == XS) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (leader)  // its barriers count both CTAs' bytes: let them all land
        for (int i = 0; i < XS; ++i)
          if (used >> i & 1) {
            volatile int32_t dummy = 0;
            mbar_wait_warp(&xfull[i], phases >> i & 1, &dummy, wd);
          }
    } else if (warp >= 4) {
      // converters: a lane takes a channel's 128 bytes, then its share of the tokens
      const int q = warp & 3, group = (warp - 4) >> 2;
      const uint32_t ofull_leader = mapa_shared(smem_u32(ofull), lead);
      // this group's blocks of all of the pair's tiles, one after the other
      const int blocks = first < tiles ? ((tiles - 1 - first) / step + 1) * (kb_end - kb_begin) : 0;
      int r = group, s = group;
      uint32_t rph = 0, ph = 0;
      const int row = q * 32 + lane;
      // token rows that exist (one tile: the others' columns are never stored)
      const int xrows = p.mt == 1 ? min(C::XROWS, max(0, M - static_cast<int>(rank) * C::XROWS)) : C::XROWS;
      for (int block = group; block < blocks; block += C::CONV_GROUPS) {
        if (!mbar_wait_warp(&rfull[r], rph, abort_flag, wd)) break;
        if (!mbar_wait_warp(&oempty[s], ph ^ 1, abort_flag, wd)) break;
        tc_fence_after();
        const uint32_t raw = smem_u32(smem + r * C::RAW_BYTES);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 w = ld_shared_v4(raw + row * 128 + (((half * 4 + c) ^ (row & 7)) << 4));
            widen4(w.x, v[8 * c], v[8 * c + 1]);
            widen4(w.y, v[8 * c + 2], v[8 * c + 3]);
            widen4(w.z, v[8 * c + 4], v[8 * c + 5]);
            widen4(w.w, v[8 * c + 6], v[8 * c + 7]);
          }
          tmem_st32(tmem + (static_cast<uint32_t>(q * 32) << 16) + C::A_COL + s * 64 + half * 32, v);
        }
        if (!WIDE) {
          // 16-byte pieces of the XROWS x 128 bytes, 16 rows at a time: piece c of a row becomes two of the fp16 tile,
          // whose two boxes hold 64 of K each
          const uint32_t xsrc = raw + C::W_BYTES, xdst = smem_u32(x_buf + s * C::X_BYTES);
          const int c = row & 7, piece = 2 * (c & 3);
#pragma unroll
          for (int i = 0; i < C::XROWS / 16; ++i) {
            if (i * 16 >= xrows) break;
            const int xrow = i * 16 + (row >> 3);
            const uint4 w = ld_shared_v4(xsrc + xrow * 128 + ((c ^ (xrow & 7)) << 4));
            uint32_t v[8];
            widen4(w.x, v[0], v[1]);
            widen4(w.y, v[2], v[3]);
            widen4(w.z, v[4], v[5]);
            widen4(w.w, v[6], v[7]);
            const uint32_t to = xdst + (c >> 2) * (C::X_BYTES / 2) + xrow * 128;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((piece + k) ^ (xrow & 7)) << 4)),
                           "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                           : "memory");
          }
          fence_proxy_async_shared();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&rempty[r]);
          mbar_arrive_operands(ofull_leader + 8 * s);
        }
        r += C::CONV_GROUPS;
        if (r >= RAW) {
          r -= RAW;
          rph ^= 1;
        }
        s += C::CONV_GROUPS;
        if (s >= OPS) {
          s -= OPS;
          ph ^= 1;
        }
      }
    }
    if (split > 1) {  // the epilogue warps' two barriers around the exchange of the parts
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

// Tokens' codes to fp16: 8 of them a thread, so that loads and stores are whole lines, four such pieces under way.
__global__ void __launch_bounds__(256) k_int8_widen(const uint2* a, uint4* out, int64_t n) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += 4 * step) {
    uint2 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * step < n) w[j] = a[i + j * step];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j * step >= n) break;
      uint4 v;
      widen4(w[j].x, v.x, v.y);
      widen4(w[j].y, v.z, v.w);
      out[i + j * step] = v;
    }
  }
}

template <int NT, int OUT>
cudaError_t launch_int8(const CUtensorMap& tmW, const CUtensorMap& tmX, const Int8GemmArgs& p, int sms, cudaStream_t st) {
  using C = Int8Cfg<NT>;
  auto kernel = k_int8_gemm<NT, OUT>;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.mt) * p.nt;
  const int64_t pairs = p.split > 1 ? tiles * p.split : (tiles < sms / 2 ? tiles : sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int NT>
cudaError_t launch_int8_out(const CUtensorMap& tmW, const CUtensorMap& tmX, const Int8GemmArgs& p, int sms, cudaStream_t st) {
  if (p.out == kInt8OutF32) return launch_int8<NT, kInt8OutF32>(tmW, tmX, p, sms, st);
  if (p.out == kInt8OutF16) return launch_int8<NT, kInt8OutF16>(tmW, tmX, p, sms, st);
  return launch_int8<NT, kInt8OutBf16>(tmW, tmX, p, sms, st);
}

}  // namespace

cudaError_t launch_int8_gemm(const CUtensorMap& tmW, const CUtensorMap& tmX, const Int8GemmArgs& p, int tile_tokens, int sms,
                             cudaStream_t st) {
  if (tile_tokens == 64) return launch_int8_out<64>(tmW, tmX, p, sms, st);
  if (tile_tokens == 128) return launch_int8_out<128>(tmW, tmX, p, sms, st);
  return launch_int8_out<256>(tmW, tmX, p, sms, st);
}

cudaError_t launch_int8_widen(const uint8_t* a, void* out, int64_t n, int sms, cudaStream_t st) {
  const int64_t groups = n / 8, blocks = (groups + 1023) / 1024, most = 8 * static_cast<int64_t>(sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_int8_widen, reinterpret_cast<const uint2*>(a), static_cast<uint4*>(out), groups);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace nvfp4

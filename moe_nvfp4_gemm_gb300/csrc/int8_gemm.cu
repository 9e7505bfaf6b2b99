// Product of 8-bit integers with a scale for each token and each channel:
//   y[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k],  the sum exact.
//
// sm_103a has no integer kind of tcgen05.mma, so the sums run through kind::f16: an 8-bit integer is exact in
// fp16, a product of two in fp32, and a sum of 1,024 products, at most 1,024 * 128^2 = 2^24, too. After every
// 1,024 of K (a chunk) the epilogue warps read the sums back, convert them and add them as 32-bit integers.
//
// A CTA pair (cta_group::2) takes 256 channels as the MMA's M and NT tokens as N. The weights stay 8-bit integers up
// to the SM: a TMA ring brings blocks of 128 of K, and a warpgroup turns each channel's 128 bytes into
// fp16 in registers (byte order 0x64uu is 1024 + u; u = b + 128; minus 1152) and stores them to TMEM, from
// where the MMA takes its A operand: the fp16 weights never pass through shared memory, whose bandwidth
// they would fill (four blocks of 64 columns). Tokens: up to 128 are converted by two warps into
// the swizzled shared-memory tile that the MMA reads; tiles of 256 come as fp16 from the workspace, converted
// once by k_int8_widen.
//
// Few tiles: the pairs of a cluster (p.split of them) sum a tile's parts of K, exchange the integer sums through
// distributed shared memory and store a share of the tokens each.
#include <stdint.h>

#include <cuda_fp16.h>

#include "ffn.cuh"
#include "kernels.h"
#include "nvfp4_quant.cuh"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

template <int NT>
struct Int8Cfg {
  // warps 0-3: weights' producer, MMA issuer, two for the tokens (converters; with NT = 256 one loads them);
  // then one or two warpgroups that convert weights, two or one of epilogue warps. 512 x 128 registers at launch.
  static constexpr int THREADS = 512;
  static constexpr bool WIDE = NT == 256;  // tokens come as fp16
  // converting groups take blocks in turn. Few tokens: bound by the weights' bytes, which one group (a block of 16 KB
  // in about 500 cycles) just keeps up with. With 256 tokens a block's MMAs take 1,024 cycles.
  static constexpr int CONV_GROUPS = WIDE ? 1 : 2;
  static constexpr int EPI_WARP = 4 + 4 * CONV_GROUPS;  // first epilogue warp
  static constexpr int EPI_WARPS = 16 - EPI_WARP;
  static constexpr int CONTROL_REGS = WIDE ? 72 : 96, EPILOGUE_REGS = WIDE ? 184 : 200;
  static_assert(32 * EPI_WARP * CONTROL_REGS + 32 * EPI_WARPS * EPILOGUE_REGS <= 512 * 128, "register shares");
  static constexpr int XROWS = NT / 2;                  // token rows of a CTA
  static constexpr int W_BYTES = 128 * 128;             // 128 channels x 128 of K
  static constexpr int RAW_BYTES = W_BYTES + (WIDE ? 0 : XROWS * 128);
  static constexpr int RAW = WIDE ? 4 : (NT == 128 ? 5 : 7);  // stages of 8-bit operands
  static constexpr int OPS = 4;                         // operand buffers: TMEM columns 256 + 64 i, X tile i
  static constexpr int X_BYTES = XROWS * 256;           // two boxes of XROWS x 64 of K, fp16
  static constexpr int BUFS = WIDE ? 1 : 2;             // TMEM buffers of sums
  static constexpr int CHUNK = 8;                       // blocks of 128 between two readings of the sums
  static constexpr int COLS = NT * 4 / EPI_WARPS;       // tokens of an epilogue warp
  static constexpr int OUT_BYTES = EPI_WARPS * 4096;            // a box for each epilogue warp
  static constexpr int SMEM_BYTES = RAW * RAW_BYTES + OPS * X_BYTES + OUT_BYTES + 1024 + 512;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  // The exchange of split sums, [part][own token][132] words, in the place of the operand rings. Tokens are owned in
  // groups of eight.
  __host__ __device__ static constexpr int own(int split) { return (NT / 8 + split - 1) / split * 8; }
  static constexpr int EXCHANGE_BYTES = (4 * own(4) > 3 * own(3) ? 4 * own(4) : 3 * own(3)) * 132 * 4;
  static_assert(EXCHANGE_BYTES <= RAW * RAW_BYTES + OPS * X_BYTES, "exchange area");
};

struct Int8Tile {
  int m0, n0;
};

DEVI Int8Tile int8_tile(const Int8GemmArgs& p, int t, int nt_tokens) {
  // tokens fastest: the pairs that run at one time share the weights
  return {t % p.mt * nt_tokens, t / p.mt * 256};
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
  constexpr int RAW = C::RAW, OPS = C::OPS, BUFS = C::BUFS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* x_buf = smem + RAW * C::RAW_BYTES;
  uint8_t* out_buf = x_buf + OPS * C::X_BYTES;
  uint64_t* rfull = reinterpret_cast<uint64_t*>(out_buf + C::OUT_BYTES);  // [RAW] 8-bit operands have landed
  uint64_t* rempty = rfull + RAW;                                         // [RAW] and have been read
  uint64_t* ofull = rempty + RAW;   // [OPS] fp16 operands are in place (leader)
  uint64_t* oempty = ofull + OPS;   // [OPS] and have been used
  uint64_t* xfull = oempty + OPS;   // [OPS] WIDE: the tokens' tile has landed (leader)
  uint64_t* tfull = xfull + OPS;    // [BUFS] a chunk's sums are complete
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
      mbar_init(&rempty[s], WIDE ? 4 : 6);  // the warps that read it
    }
    for (int s = 0; s < OPS; ++s) {
      mbar_init(&ofull[s], WIDE ? 8 : 12);  // the converting warps of both CTAs
      mbar_init(&oempty[s], 1);
      mbar_init(&xfull[s], 1);
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
    int buf = 0;
    uint32_t bph = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const Int8Tile tl = int8_tile(p, t, NT);
      const int own = C::own(split);  // split: tokens that this CTA stores
      const int row0 = tl.m0 + (split > 1 ? part * own : h * C::COLS);
      const int col0 = tl.n0 + static_cast<int>(rank) * 128 + q * 32;
      // A lane holds the scales of tokens 32 c + lane of those that its warp stores, and of channel `lane` of the
      // warp's 32: requested here, so that no load waits behind the sums.
      constexpr int SA = NT / 32 < 4 ? NT / 32 : 4;
      float sa[SA];
#pragma unroll
      for (int c = 0; c < SA; ++c) sa[c] = row0 + 32 * c + lane < M ? p.sa[row0 + 32 * c + lane] : 0.0f;
      const float sb_lane = col0 + lane < N ? p.sb[col0 + lane] : 0.0f;
      // acc[32 c + 16 i + 4 g + 2 j + u]: channel 16 i + 8 j + lane / 4 of the warp's 32, token
      // 32 c + 8 g + 2 (lane % 4) + u of its COLS
      int acc[C::COLS];
#pragma unroll
      for (int i = 0; i < C::COLS; ++i) acc[i] = 0;
#pragma unroll 1
      for (int kb = kb_begin; kb < kb_end; kb += C::CHUNK) {
        ok = mbar_wait_warp(&tfull[buf], bph, abort_flag, wd);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT + h * C::COLS;
#pragma unroll
        for (int c = 0; c < C::COLS / 32; ++c) {
          uint32_t r[32];
          tmem_ld_frag32(at + c * 32, r);
          tmem_ld_frag32(at + c * 32 + (16u << 16), r + 16);
          tmem_ld_wait32(r);
          if (c + 1 == C::COLS / 32) {
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive_cluster(tempty_leader + 8 * buf);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[32 * c + j] += __float2int_rn(__uint_as_float(r[j]));
        }
        if (++buf == BUFS) {
          buf = 0;
          bph ^= 1;
        }
      }
      if (split > 1) {
        // All roles of all the cluster's CTAs are done with the rings; also after an abort (then garbage, not
        // stored), so that the cluster's barriers pair. CTA `part` of its half stores tokens [part, part + 1) own.
        uint32_t* recv = reinterpret_cast<uint32_t*>(smem);
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int c = 0; c < C::COLS / 32; ++c)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int tok = h * C::COLS + 32 * c + 8 * g + 2 * (lane & 3);  // a group of 8 has one owner
            const int o = tok / own;
            const uint32_t dst = mapa_shared(smem_u32(recv + (part * own + tok - o * own) * 132 + q * 32 + (lane >> 2)), 2 * o + rank);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                st_shared_cluster_b32(dst + (u * 132 + 8 * i) * 4, acc[32 * c + 16 * (i >> 1) + 4 * g + 2 * (i & 1) + u]);
          }
        __syncwarp();
        cluster_sync();
        if (ok && !*abort_flag) {
          // a lane: one channel; a warp: every other token where two have the same channels
          const int n = col0 + lane;
          constexpr int STEP = C::EPI_WARPS / 4;
          const int rows = min(min(own, NT - part * own), M - row0);
          const uint32_t* src = recv + q * 32 + lane;
#pragma unroll
          for (int c = 0; c < SA; ++c)
#pragma unroll 4
            for (int j = h; j < 32; j += STEP) {
              const float sa_j = __shfl_sync(0xffffffffu, sa[c], j);
              const int i = 32 * c + j;
              if (i >= rows) break;
              uint32_t v = 0;
              for (int s = 0; s < split; ++s) v += src[(s * own + i) * 132];
              const float f = static_cast<float>(static_cast<int>(v)) * sa_j * sb_lane;
              const int64_t to = static_cast<int64_t>(row0 + i) * N + n;
              if (n < N) {
                if (OUT == kInt8OutF32)
                  static_cast<float*>(p.y)[to] = f;
                else
                  static_cast<uint16_t*>(p.y)[to] = static_cast<uint16_t>(pack16<OUT == kInt8OutF16>(f, 0.0f) & 0xFFFFu);
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
        // 32 tokens x 32 channels at a time through the warp's box
#pragma unroll
        for (int c = 0; c < C::COLS / 32; ++c) {
          const int rows = min(32, M - row0 - 32 * c);
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
          const int64_t at = static_cast<int64_t>(row0 + 32 * c) * N + col0;
          if (OUT == kInt8OutF32) {
            float* y = static_cast<float*>(p.y) + at;
            if (N % 4 == 0) {  // 16 bytes a lane, four tokens at a time
              if (col0 + 4 * (lane & 7) < N)
                for (int i = lane >> 3; i < rows; i += 4)
                  *reinterpret_cast<uint4*>(y + static_cast<int64_t>(i) * N + 4 * (lane & 7)) =
                      *reinterpret_cast<const uint4*>(box + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
            } else if (col0 + lane < N) {
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
        const uint32_t idesc = idesc_f16(256, NT, false);
        int s = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        for (int t = first; t < tiles && !*abort_flag; t += step) {
          for (int kb = kb_begin; kb < kb_end; ++kb) {
            const int in_chunk = (kb - kb_begin) % C::CHUNK;
            if (!mbar_wait_warp(&ofull[s], ph, abort_flag, wd)) break;
            if (WIDE && !mbar_wait_warp(&xfull[s], ph, abort_flag, wd)) break;
            if (in_chunk == 0 && !mbar_wait_warp(&tempty[buf], bph ^ 1, abort_flag, wd)) break;
            tc_fence_after();
            const bool last = in_chunk == C::CHUNK - 1 || kb + 1 == kb_end;
            if (elect_one()) {
              const uint32_t xa = smem_u32(x_buf + s * C::X_BYTES);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_f16_pair_ts(tmem + buf * NT, tmem + 256 + s * 64 + kk * 8,
                                   desc_sw128(xa + (kk >> 2) * (C::X_BYTES / 2)) + 2 * (kk & 3), idesc, in_chunk != 0 || kk != 0);
              tc_commit_pair(&oempty[s], 3u << lead);
              if (last) tc_commit_pair(&tfull[buf], 3u << lead);
            }
            __syncwarp();
            if (++s == OPS) {
              s = 0;
              ph ^= 1;
            }
            if (last && ++buf == BUFS) {
              buf = 0;
              bph ^= 1;
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
          if (!mbar_wait_warp(&oempty[s], ph ^ 1, abort_flag, wd)) break;
          if (elect_one()) {
            uint8_t* st = x_buf + s * C::X_BYTES;
            const uint32_t bar = mapa_shared(smem_u32(&xfull[s]), lead);
            if (leader) mbar_arrive_expect_tx(&xfull[s], 2 * C::X_BYTES);
            tma_load_2d_pair(st, &tmX, bar, kb * 128, tl.m0 + rank * C::XROWS, pol);
            tma_load_2d_pair(st + C::X_BYTES / 2, &tmX, bar, kb * 128 + 64, tl.m0 + rank * C::XROWS, pol);
          }
          __syncwarp();
          used |= 1u << s;
          phases = (phases & ~(1u << s)) | ph << s;
          if (++s == OPS) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (leader)  // its barriers count both CTAs' bytes: let them all land
        for (int i = 0; i < OPS; ++i)
          if (used >> i & 1) {
            volatile int32_t dummy = 0;
            mbar_wait_warp(&xfull[i], phases >> i & 1, &dummy, wd);
          }
    } else if (warp >= 4 || !WIDE) {
      // converters: a lane takes a channel's 128 bytes (warps 4-7), or with the other token warp the
      // tokens', a row or half a row each
      const bool weights = warp >= 4;
      const int q = warp & 3, group = (warp - 4) >> 2;
      const uint32_t ofull_leader = mapa_shared(smem_u32(ofull), lead);
      int r = 0, s = 0;
      uint32_t rph = 0, ph = 0, block = 0;
      for (int t = first; t < tiles && !*abort_flag; t += step) {
        for (int kb = kb_begin; kb < kb_end; ++kb, ++block) {
          const bool turn = !weights || C::CONV_GROUPS == 1 || static_cast<int>(block & 1) == group;
          if (turn && !mbar_wait_warp(&rfull[r], rph, abort_flag, wd)) break;
          if (turn && !mbar_wait_warp(&oempty[s], ph ^ 1, abort_flag, wd)) break;
          tc_fence_after();
          const uint32_t raw = smem_u32(smem + r * C::RAW_BYTES);
          if (!turn) {
          } else if (weights) {
            const int row = q * 32 + lane;
            const uint32_t src = raw + row * 128;
            const uint32_t dst = tmem + (static_cast<uint32_t>(q * 32) << 16) + 256 + s * 64;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t v[32];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint4 w = ld_shared_v4(src + (((half * 4 + c) ^ (row & 7)) << 4));
                widen4(w.x, v[8 * c], v[8 * c + 1]);
                widen4(w.y, v[8 * c + 2], v[8 * c + 3]);
                widen4(w.z, v[8 * c + 4], v[8 * c + 5]);
                widen4(w.w, v[8 * c + 6], v[8 * c + 7]);
              }
              tmem_st32(dst + half * 32, v);
            }
            tmem_st_wait();
            tc_fence_before();
          } else {
            // 16-byte pieces of the XROWS x 128 bytes: piece c of row i becomes two of the fp16 tile, whose two
            // boxes hold 64 of K each
            const uint32_t src = raw + C::W_BYTES, dst = smem_u32(x_buf + s * C::X_BYTES);
#pragma unroll 4
            for (int i = (warp - 2) * 32 + lane; i < C::XROWS * 8; i += 64) {
              const int row = i >> 3, c = i & 7;
              const uint4 w = ld_shared_v4(src + row * 128 + ((c ^ (row & 7)) << 4));
              uint32_t v[8];
              widen4(w.x, v[0], v[1]);
              widen4(w.y, v[2], v[3]);
              widen4(w.z, v[4], v[5]);
              widen4(w.w, v[6], v[7]);
              const uint32_t to = dst + (c >> 2) * (C::X_BYTES / 2) + row * 128;
              const int piece = 2 * (c & 3);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((piece + k) ^ (row & 7)) << 4)),
                             "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                             : "memory");
            }
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (turn && lane == 0) {
            mbar_arrive(&rempty[r]);
            mbar_arrive_operands(ofull_leader + 8 * s);
          }
          if (++r == RAW) {
            r = 0;
            rph ^= 1;
          }
          if (++s == OPS) {
            s = 0;
            ph ^= 1;
          }
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

// Tokens' codes to fp16, 16 a thread.
__global__ void __launch_bounds__(256) k_int8_widen(const uint4* a, uint4* out, int64_t n) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    const uint4 w = a[i];
    uint4 lo, hi;
    widen4(w.x, lo.x, lo.y);
    widen4(w.y, lo.z, lo.w);
    widen4(w.z, hi.x, hi.y);
    widen4(w.w, hi.z, hi.w);
    out[2 * i] = lo;
    out[2 * i + 1] = hi;
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
  const int64_t groups = n / 16, blocks = (groups + 255) / 256, most = 8 * static_cast<int64_t>(sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_int8_widen, reinterpret_cast<const uint4*>(a), static_cast<uint4*>(out), groups);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace nvfp4

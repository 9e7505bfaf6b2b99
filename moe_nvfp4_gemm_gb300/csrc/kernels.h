// Launch interfaces shared by the C ABI (capi.cu) and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace nvfp4 {

struct DenseArgs {
  const uint8_t* sfa;
  const uint8_t* sfb;
  const float* ga;
  const float* gb;
  uint16_t* y;
  int M, N, K;
  int32_t* status;
  // NVFP4 output (k_gemm_dense_pair<true>): codes [M, N/2], tiled scales of [M, N], with
  // the caller's global scale; y is not written
  uint8_t* q_out;
  uint8_t* sf_out;
  const float* g_out;
  uint64_t watchdog_ns;  // limit of every pipeline wait
  int drop_stage;        // test hook: k >= 1 withholds the k-th stage CTA 0 loads (0: none)
  // tile order: 0 m-blocks fastest; -1 n-blocks fastest; G > 0 bands of G m-blocks, m fastest
  // inside a band (the band's B tiles are read by G CTA pairs at about the same time)
  int raster;
};

// Tile t of an mt x nt grid of output tiles in the order `raster` selects.
__host__ __device__ inline void tile_coords(int t, int mt, int nt, int raster, int& m_blk, int& n_blk) {
  if (raster < 0) {
    m_blk = t / nt;
    n_blk = t % nt;
  } else if (raster == 0 || raster >= mt) {
    m_blk = t % mt;
    n_blk = t / mt;
  } else {
    const int band = t / (raster * nt);
    const int first = band * raster;
    const int rows = mt - first < raster ? mt - first : raster;
    const int local = t - band * raster * nt;
    m_blk = first + local % rows;
    n_blk = local / rows;
  }
}

struct StreamArgs {
  const uint8_t* sfw;      // weight scales (grouped: expert e at sfw + e * sfw_stride)
  int64_t sfw_stride;
  const uint8_t* sfx;      // dense: token scales; grouped: scale slabs per token tile
  const float* ga;
  const float* gb;         // grouped: gb[e]
  uint16_t* y;
  const int4* tiles;       // grouped: (expert, first row, rows, slab)
  const int32_t* n_tiles;  // grouped: device count of tiles
  int32_t* status;
  int M;                   // dense: tokens; grouped: M_total
  int N, K;
  int split;               // dense: cluster size along K
  int stages;
  int x_rows;              // token rows reserved per stage (multiple of 16)
  int acc_cols;            // TMEM columns per accumulator buffer
  int acc_bufs;
  int tmem_cols;
  int pdl;                 // launched with programmatic stream serialization
  int swiglu;              // grouped: weight rows interleave gate/up; y[t, c] = silu(gate) * up, N / 2 wide
  const int32_t* row_token;  // grouped: routed row r reads token row row_token[r] of x (null: row r)
  int T;                     // grouped with row_token: rows of x
  int w_keep;                // weights loaded L2 evict_last (kept resident across calls), else evict_first
  uint64_t watchdog_ns;      // limit of every pipeline wait
  int drop_stage;            // test hook: k >= 1 withholds the k-th stage CTA 0 loads (0: none)
  const uint8_t* meta;       // pair-wise 2:4 sparse weights: tiled metadata (null: dense weights)
  int64_t meta_stride;       // grouped: bytes of metadata per expert
  int l2_prefetch;           // dense: K blocks of the CTA's weight slice prefetched into L2 at entry
  // grouped SwiGLU emitting NVFP4: codes [M, N/4] and tiled scales of [M, N/2] with the
  // caller's global scale g_out; y is not written
  uint8_t* q_out;
  uint8_t* sf_out;
  const float* g_out;
};


// A batched decode launch: up to kMaxBatch GEMMs sharing M (and the launch's split-K,
// stage count and token rows); tensor maps and pointers per GEMM, passed as kernel
// parameters.
constexpr int kMaxBatch = 8;
struct BatchParams {
  CUtensorMap w[kMaxBatch];  // weights [N, K/2], 128-row boxes
  CUtensorMap x[kMaxBatch];  // activations [M, K/2], 16-row boxes
  const uint8_t* sfw[kMaxBatch];
  const uint8_t* sfx[kMaxBatch];
  const float* ga[kMaxBatch];
  const float* gb[kMaxBatch];
  uint16_t* y[kMaxBatch];
  int N[kMaxBatch], K[kMaxBatch];
  int cta_base[kMaxBatch + 1];  // first CTA of each GEMM; cta_base[count] = grid
  int count;
};

// Token rows of one expert per grouped work item: up to 128 (MMA N <= 128); 64 bounds the
// tile count that the workspace is sized for, so either size fits the same workspace.
constexpr int kGroupTile = 64;
constexpr int kGroupTileMax = 128;

cudaError_t launch_amax(const uint16_t* x, int64_t n, float* amax_out, float* g_out, float* partial,
                        int max_partials, cudaStream_t st);
cudaError_t launch_quantize(const uint16_t* x, int64_t M, int64_t K, const float* g, uint8_t* q, uint8_t* sf,
                            cudaStream_t st);
cudaError_t launch_encode(int which, const float* v, int64_t n, uint8_t* out, cudaStream_t st);
cudaError_t launch_prune_pairs(const uint16_t* w, int64_t N, int64_t K, uint16_t* c, uint8_t* meta, int sms,
                               cudaStream_t st);
cudaError_t launch_quantize_b32(const uint16_t* x, int64_t M, int64_t K, const float* g, uint8_t* q, uint8_t* sf,
                                cudaStream_t st);
cudaError_t launch_dense(const CUtensorMap& tmA, const CUtensorMap& tmB, const DenseArgs& a, int bn, int grid,
                         cudaStream_t st);
cudaError_t launch_dense_pair(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmSFA,
                              const CUtensorMap& tmSFB, const CUtensorMap& tmY, const DenseArgs& a, int grid,
                              cudaStream_t st, bool quantized_out = false);
cudaError_t launch_stream(const CUtensorMap& tmW, const CUtensorMap& tmX, const StreamArgs& a, bool grouped,
                          int grid, cudaStream_t st);
cudaError_t launch_batched(const BatchParams& bp, const StreamArgs& a, int grid, cudaStream_t st);
cudaError_t launch_grouped_prep(const int32_t* offsets, const int32_t* row_token, int T, int E, int M_total, int K,
                                int kc4, int tile_rows, const uint8_t* sfx,
                                int32_t* n_tiles, int4* tiles, uint8_t* slabs, int32_t* status, int grid,
                                cudaStream_t st, const uint8_t* x_tok = nullptr, uint8_t* xg = nullptr);

// ---- MoE router ---------------------------------------------------------------------------
constexpr int kRouteBlocks = 304;  // most CTAs that share the tokens (two per SM)
struct RouteArgs {
  const void* logits;     // [T, E], fp32 or bf16
  const uint8_t* valid;   // [T] or null
  int64_t T;
  int E, k;
  int bf16, renorm;
  int vec;                // rows can be read a lane's values at a time
  int32_t* topk_idx;      // [T, k]
  float* topk_w;          // [T, k]
  int32_t* slot_row;      // [T, k]
  int32_t* counts;        // [E]
  int32_t* expert_offsets;  // [E + 1]
  int32_t* row_token;     // [T * k]
  float* mean_prob;       // [E]
  float* loss;            // [1]
  int32_t* routed_tokens;  // [1]
  int32_t* ws_hist;       // [blocks][E + 1]
  float* ws_psum;         // [blocks][E]
};
struct RouteBwdArgs {
  const void* logits;
  const uint8_t* valid;
  int64_t T;
  int E, k;
  int bf16, renorm;
  int vec;
  const int32_t* topk_idx;
  const float* topk_w;
  const int32_t* counts;
  const int32_t* routed_tokens;
  const float* d_w;       // [T, k] or null
  const float* d_loss;    // [1] or null
  void* d_logits;         // [T, E], the logits' type
};
int route_blocks(int64_t T, int E);
cudaError_t launch_moe_route(RouteArgs a, cudaStream_t st, int* launches);
cudaError_t launch_moe_route_bwd(RouteBwdArgs a, int sms, cudaStream_t st);

// ---- FP8 block-128 operators --------------------------------------------------------------
struct Fp8QuantArgs {
  const uint16_t* x;         // bf16 [M_x, K]
  const int32_t* row_token;  // [M] rows of x, or null (row r)
  int64_t M_x, M, K;
  uint8_t* q;                // [M, K] or null
  float* s;                  // [ceil(K/128), M], square blocks [ceil(M/128), ceil(K/128)]
  uint8_t* qt;               // [K, M rounded up to 16] or null
  float* st;                 // [ceil(M/128), K], square blocks [ceil(K/128), ceil(M/128)]
};
cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int block_rows, cudaStream_t st);

struct Fp8GemmArgs {
  const float* sa;
  const float* sb;
  void* y;
  int64_t M, N, K;
  int b_rows;              // rows of b that share a scale: 128 or 1
  int f32;                 // y fp32 instead of bf16
  const int4* tiles;       // grouped: (expert, first row, rows, -), else null
  const int32_t* n_tiles;
  int max_tiles;           // grouped: most tiles the list can hold
  int32_t* status;
  uint64_t watchdog_ns;    // limit of every pipeline wait
  int drop_stage;          // test hook: k >= 1 withholds the k-th stage CTA 0 loads (0: none)
  int split;               // streaming kernel, dense: cluster size along K
  int stages;              // streaming kernel: ring depth (set by its launcher)
  int l2_prefetch;         // streaming kernel, dense: blocks of K prefetched into L2 at entry
};
cudaError_t launch_fp8_stream(const CUtensorMap& tmW, const CUtensorMap& tmX, const Fp8GemmArgs& p, int tile_rows,
                              int sms, cudaStream_t st);
cudaError_t launch_fp8_tiles(const int32_t* offsets, int E, int M, int tile_rows, int4* tiles, int32_t* n_tiles,
                             int32_t* status, cudaStream_t st);
// grid: an even number of CTAs (two per 256 x 256 tile in flight)
cudaError_t launch_fp8_gemm_pair(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmY,
                                 const Fp8GemmArgs& p, int grid, cudaStream_t st);
// grid: an even number of CTAs (two per tile of 256 weight rows and up to 128 tokens in flight);
// dense without p.tiles. tmW has 128-row boxes, tmX 32.
cudaError_t launch_fp8_narrow(const CUtensorMap& tmW, const CUtensorMap& tmX, const Fp8GemmArgs& p, int grid,
                                    cudaStream_t st);

// ---- 16-bit gated feed-forward block ------------------------------------------------------
// Forward: a[0] x, b gate and up, y h, gate, up; boxes of 64 x 128. Gradients: a dg and du, b w_gate, w_up and x, y dx and
// the weights' gradients; boxes of 64 x 64. part: the sums of a product in parts, fp32.
struct FfnTileMaps {
  CUtensorMap a[2], b[3], y[3], part[2];
};
struct FfnProduct {
  int M, N;     // rows and columns of a result
  int mt, nt;   // 256 x 256 tiles of sums (forward: 128 columns of h each)
  int kblocks;  // blocks of 64 of the contraction
  int split;    // its parts
  int items;    // tiles x parts x results
  int raster;   // tile order, see tile_coords
  float* ws;    // split > 1: fp32 [results][split][mt * 256][nt * 256]
};
struct FfnTileArgs {
  FfnProduct in[2];  // forward: one; gradients: of the input and of the weights (no items: not wanted)
  int act, save;     // forward: activation; also write gate and up
  int up_first;      // gradients: the weights' first result is w_up's
  int half;          // fp16 instead of bf16
  int drop_stage;    // test hook: k >= 1 withholds the k-th stage CTA 0 loads (0: none)
  int32_t* status;
  uint64_t watchdog_ns;  // limit of every pipeline wait
  void* y[3];        // the results, as maps.y, written by the kernel that joins parts
  int64_t ldy;       // forward: row stride of h
};
cudaError_t launch_ffn_tile(const FfnTileMaps& maps, const FfnTileArgs& p, bool forward, int sms, cudaStream_t st);
// Forward pass for up to 128 tokens. w: gate and up, boxes of 64 x 64; x: boxes of 64 x 32.
struct FfnStreamMaps {
  CUtensorMap w[2], x;
};
struct FfnStreamArgs {
  uint16_t* h;     // rows ldh apart
  float* gate;     // [M, N], with up: also written, or null
  float* up;
  int64_t ldh;
  int M, N;
  int kblocks;     // blocks of 64 of K
  int split;       // cluster size along K
  int act, half;
  int l2_prefetch;  // blocks of K prefetched into L2 at entry
  int drop_stage;   // test hook: k >= 1 withholds the k-th stage CTA 0 loads (0: none)
  int32_t* status;
  uint64_t watchdog_ns;  // limit of every pipeline wait
};
cudaError_t launch_ffn_stream(const FfnStreamMaps& maps, const FfnStreamArgs& p, cudaStream_t st);
struct FfnGradArgs {
  const float* gate;     // [M, I]
  const float* up;       // [M, I]
  const uint16_t* dh;    // rows lddh apart
  uint16_t* dg;          // [M, I]
  uint16_t* du;          // [M, I]
  int64_t M, lddh;
  int I, act, half;
};
cudaError_t launch_ffn_grad(const FfnGradArgs& p, int sms, cudaStream_t st);

// ---- 8-bit integers with a scale for each row ----------------------------------------------
struct Int8QuantArgs {
  const uint16_t* x;  // rows ldx apart
  int64_t M, K, ldx;
  uint8_t* q;         // [M, K]
  float* s;           // [M]
  int half;           // fp16 instead of bf16
};
enum { kInt8OutBf16 = 0, kInt8OutF32 = 1, kInt8OutF16 = 2 };
struct Int8GemmArgs {
  const float* sa;  // [M]
  const float* sb;  // [N]
  void* y;          // [M, N]
  int64_t M, N, K;
  int mt, nt;       // tiles: tokens, 256 channels
  int split;        // pairs of a cluster, along K
  int raster;       // tile order, see tile_coords
  int out;
  int drop_stage;   // test hook: k >= 1 withholds the k-th stage CTA 0 loads (0: none)
  int32_t* status;
  uint64_t watchdog_ns;  // limit of every pipeline wait
};
// tile_tokens 64 or 128: tmX over the codes [M, K], boxes of 128 x tile_tokens / 2; 256: over their fp16 values,
// boxes of 64 x 64. tmW: boxes of 128 x 128.
cudaError_t launch_int8_gemm(const CUtensorMap& tmW, const CUtensorMap& tmX, const Int8GemmArgs& p, int tile_tokens, int sms,
                             cudaStream_t st);
constexpr int kInt8FewTokens = 8;  // most tokens of the kernel without tensor cores
constexpr int kInt8FewRows = 32;   // channels of one of its CTAs, over split
constexpr int int8_few_resident(int64_t M) { return M <= 2 ? 4 : (M <= 4 ? 3 : 2); }  // its CTAs on an SM, by their registers
struct Int8FewArgs {
  const int8_t* a;  // [M, K]
  const int8_t* b;  // [N, K]
  const float* sa;
  const float* sb;
  void* y;
  int64_t M, N, K;
  int split;        // warps that share a channel: 1, 2, 4 or 8
  int out;
};
cudaError_t launch_int8_few(const Int8FewArgs& p, cudaStream_t st);
// n codes (a multiple of 16) to fp16
cudaError_t launch_int8_widen(const uint8_t* a, void* out, int64_t n, int sms, cudaStream_t st);
cudaError_t launch_int8_quantize(const Int8QuantArgs& p, int sms, cudaStream_t st);

// ---- gradient norm and clipping -----------------------------------------------------------
constexpr int kClipChunk = 16384;  // values that a block takes at a time
constexpr int kClipGroup = 960;    // gradients a launch takes (its parameters hold the list)
constexpr int kClipBlocks = 608;   // blocks of a launch at most: four on each SM
constexpr int kClipCluster = 8;    // CTAs that take a short list, of up to kClipFew chunks, in one launch
constexpr int kClipFew = 16;
enum { kClipBf16 = 0, kClipF32 = 1, kClipF16 = 2 };
struct ClipEntry {
  const void* src;
  void* dst;
  int64_t numel;
  int first;  // its first chunk
  int type;
};
struct ClipArgs {
  const void* const* src;  // host arrays
  void* const* dst;        // null: in place
  const int64_t* numel;
  const int32_t* types;
  double* partial;         // a sum of squares for each block of the first kernels
  float* norm;
  int slots;               // of them
  float max_norm;
  int scale;               // also write the scaled gradients
};
struct ClipGroup {
  int first, end;  // gradients of this launch
  int chunks;
  int slot0, grid;
};
// Entry i of the list; false where it has no values.
inline bool clip_list_entry(const ClipArgs& a, int i, ClipEntry& e) {
  e.src = a.src[i];
  e.dst = a.dst ? a.dst[i] : const_cast<void*>(a.src[i]);
  e.numel = a.numel[i];
  e.type = a.types[i];
  return e.numel > 0;
}
// The sums of squares; the kernel that joins them and scales; or both, for a list of few chunks.
enum ClipStep { kClipNorm, kClipScale, kClipAll };
cudaError_t launch_clip_group(const ClipArgs& a, const ClipGroup& g, ClipStep step, cudaStream_t st);

int stream_smem_bytes(int stages, int x_rows, int recv_bytes, bool sparse = false);
// shared memory after the ring for one tile's token indices (and with qout the epilogue's
// NVFP4 transpose tiles, 1 KB per epilogue warp)
__host__ __device__ inline int grouped_extra_bytes(int x_rows, bool qout = false) {
  return (x_rows * 4 > 256 ? x_rows * 4 : 256) + (qout ? 4 * 1024 : 0);
}
int stream_recv_bytes(int M, int split);

// Raises `func`'s dynamic shared-memory limit to the opt-in maximum, once per
// (kernel, device); later calls only look the pair up.
cudaError_t allow_max_smem(const void* func);

}  // namespace nvfp4

// ff_internal.h -- host-side interface of the feed-forward operators: kernel
// arguments, launches, and the tile shapes ff_api.cu chooses from.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv_cache_internal.h"   // api_*: what the C ABI's translation units share

namespace gemm_tn_dev {

// Kernel arguments of the products with whole tiles (sm103_ff_gemm.cuh) and of
// those with few rows of A (sm103_ff_skinny.cu).
struct FfArgs {
  CUtensorMap tmap_a;   // 128-byte-swizzled boxes, 128 bytes along the contiguous dimension
  CUtensorMap tmap_b;
  CUtensorMap tmap_as;  // e4m3 in whole tiles: A's scales {m, k blocks}, boxes {128, 1}
  CUtensorMap tmap_bs;  // B's {n, k blocks}, boxes {MMA N, 1}; or, of 128 rows, {k blocks, n / 128}, boxes {4, MMA N / 128}
  void* c;              // [m, n], element type out_kind
  int64_t ldc;
  void* pre;            // gated: [m, 2n] the two projections, or NULL
  int64_t ldp;
  const float* a_scale;   // e4m3 with few rows: [m, k blocks], strides in elements
  const float* b_scale;   // [n or ceil(n / 128), k blocks]
  int64_t as_row, as_blk, bs_row, bs_blk;
  int32_t b_block_rows;   // rows of B that share a scale: 1 or 128
  int32_t m, n;         // of C
  int32_t num_k_blocks;
  int32_t num_m_tiles, num_n_tiles, num_tiles;
  int32_t group_m;      // tile rows that run together (whole tiles)
  int32_t activation;   // 1 relu, 2 gelu, 3 silu
  int32_t out_kind;     // 0 fp16, 1 bf16, 2 fp32
  int32_t accumulate;   // fp32: C's contents are added to
  int32_t splits;       // nt: parts that K is cut into, each summed into an [m, n] array of its own (fp32, part_stride apart)
  int64_t part_stride;
  int32_t alone;        // nothing may start early while this runs (a workspace is freed behind it)
  int* status;
  uint64_t timeout_ns;
  int32_t drop_load_kb; // test hook: k-block of the first tile whose loads are skipped (-1: none)
};

struct GatedGradArgs {
  const void* grad;     // [m, n]
  const void* pre;      // [m, 2n]
  void* out;            // [m, 2n]
  int64_t ldg, ldp, ldo;
  int64_t m, n;
  int32_t activation;
};

struct QuantizeArgs {
  const void* x;        // [rows, cols]
  int64_t ldx;
  uint8_t* q;           // [rows, cols], or [cols, rows] transposed
  int64_t ldq;
  float* scale;
  int64_t s_line, s_blk;   // strides of the scales: lines (or blocks of 128 lines) of q, and blocks along a line
  int64_t rows, cols;
};

}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

enum FfKind : int { kFfGated = 0, kFfNt = 1, kFfE4m3 = 2, kFfE4m3Rows = 3 };
// Whole-tile shapes: rows x columns of the MMA, and the CTAs that share it.
enum FfTile : int { kFfPair256 = 0, kFfPair128 = 1, kFfSingle128 = 2, kNumFfTiles = 3 };
struct FfTileInfo {
  int cta_group, tile_m, block_n;
};
constexpr FfTileInfo kFfTiles[kNumFfTiles] = {{2, 256, 256}, {2, 256, 128}, {1, 128, 128}};

cudaError_t launch_ff_gated(int tile, bool bf16, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream);
cudaError_t launch_ff_nt(int tile, bool bf16, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream);
cudaError_t launch_ff_e4m3(int tile, bool b_rows, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream);
// CTA pairs that run at once on the current device (0 on error): every form of
// a tile takes an SM's shared memory whole.
int ff_resident_pairs(int sms);

// Clusters of `splits` CTAs with an SM each that run at once on the current device (0 on error).
int ff_resident_clusters(int splits, int sms);
// Few rows of A: `rows` (16, 32, 64 or 128) of them against 128 rows of B a CTA, K split over clusters of `splits`
// CTAs with an SM each (0: whole, two CTAs to an SM).
// Up to 32 rows it runs whatever K; more pay where a long K is cut. Beside whole
// tiles, us: e4m3, 64 rows, 4096 x 8192 11.7 and 18.2, x 1024 6.3 and 5.0; 256
// rows cut in four, 1024 x 8192 15.9 and 18.4, x 4096 11.8 and 10.8; 200 rows cut
// in eight, 512 x 4096 8.7 and 10.5; gated, 128 rows, 4096 x 4096 14.9 and 17.8, x
// 1024 9.1 and 7.5; 256 rows, 512 x 4096 10.0 and 17.0.
constexpr bool ff_skinny_has(int kind, int rows, int splits) {
  return rows <= 32 || splits >= (rows == 128 && kind != kFfGated ? 4 : 2);
}
constexpr bool ff_skinny_pays(int kind, int rows, int splits, int64_t k_blocks) {
  return rows <= 32 || k_blocks >= (rows == 64 ? 16 : kind == kFfGated || splits == 8 ? 32 : 64);
}
cudaError_t launch_ff_skinny(int kind, bool bf16, int rows, int splits, const gemm_tn_dev::FfArgs& args, int grid,
                             cudaStream_t stream);

// C [m, n] = the sum of `parts` fp32 arrays (pitch a multiple of 4), in order, as out_kind; or added to C.
struct JoinRequest {
  const float* parts;
  int64_t pitch, part_stride;
  int splits;
  void* c;
  int64_t ldc, m, n;
  int out_kind, accumulate;
};
cudaError_t launch_join_parts(const JoinRequest& req, int num_sms, cudaStream_t stream);

// launch_repack2's copies of 16-bit rows, made by pieces through all rows (a
// block to a row leaves most of it idle where rows are short).
cudaError_t launch_pad_rows(const RepackRequest (&req)[2], cudaStream_t stream);

// dst[i * pitch + j] = src[i * s_i + j * s_j] for i < rows, j < cols; up to two at once (rows 0: none).
struct PackRequest {
  const float* src;
  float* dst;
  int64_t rows, cols, s_i, s_j, pitch;
};
cudaError_t launch_pack_scales(const PackRequest (&req)[2], cudaStream_t stream);

cudaError_t launch_gated_grad(bool bf16, const gemm_tn_dev::GatedGradArgs& args, int num_sms, cudaStream_t stream);
cudaError_t launch_quantize(int src_kind, int block_rows, bool transpose, const gemm_tn_dev::QuantizeArgs& args,
                            cudaStream_t stream);

}  // namespace gemm_tn_impl

// sm103_ff_gemm.cuh -- the feed-forward products in whole tiles, one kernel in
// three forms:
//  * gated: H = act(A Bg^T) * (A Bu^T), with B's rows [0, n) the gate's and
//    [n, 2n) the other projection's. A tile multiplies the same rows of A by
//    as many rows of either, side by side as one N of the tensor core's
//    instruction, so that an epilogue thread finds both values of an output
//    in its own row of tensor memory and the two projections never leave the
//    chip (unless `pre` asks for them).
//  * nt: C = A^T B, both operands stored with the summed dimension outermost
//    (a weight's gradient, summed over tokens): read in place through
//    MN-major descriptors, no transposed copies.
//  * e4m3: C[i][j] = sum over blocks of 128 of sa[i][b] sb[j][b] (A_b B_b^T)[i][j].
//    The scales differ from block to block, so the tensor core's sum ends at
//    each block of 128: the block's product lands in one of the tensor
//    memory's buffers, and the epilogue warps fold it, scaled, into fp32 sums
//    in registers while the next block multiplies.
//
// One persistent CTA (or pair: cta_group::2, 256 rows) per SM: warps 0 and 2
// move A's and B's tiles with the TMA into a ring, warp 1 issues the MMAs, warps
// 4 to 11 are the epilogue, two for each quarter of tensor memory.
//
// What bounds them, and what they measured, stands at the instantiations
// (sm103_ff_gated.cu, sm103_ff_nt.cu, sm103_ff_e4m3.cu).
#pragma once

#include <atomic>

#include "sm103_ff.cuh"

namespace gemm_tn_dev {
namespace ff {

constexpr uint32_t kLoadA = 0, kMultiply = 1, kLoadB = 2;   // warps
constexpr int kFirstEpilogueWarp = 4;
// e4m3: an epilogue thread holds 128 sums and the values being added; the first
// warpgroup gives up registers for it (128 x 72 + 256 x 216 = 384 x 168, what
// the block is launched with)
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 32 * (kFirstEpilogueWarp + kEpilogueWarps);
constexpr uint32_t kFewRegisters = 72, kManyRegisters = 216;
static_assert(128 * kFewRegisters + 256 * kManyRegisters <= kThreads * 168, "register split");
constexpr int kGated = 0, kNt = 1, kE4m3 = 2, kE4m3Rows = 3;   // kE4m3Rows: a scale for each row of B, else for 128 rows

template <int kForm_, int kCtaGroup_, int kBlockN_, int kStages_, bool kBf16_>
struct Tile {
  static constexpr int kForm = kForm_;
  static constexpr int kCtaGroup = kCtaGroup_;
  static constexpr int kBlockN = kBlockN_;               // columns of products to a tile
  static constexpr int kStages = kStages_;
  static constexpr bool kBf16 = kBf16_;
  static constexpr bool kScaled = kForm == kE4m3 || kForm == kE4m3Rows;
  static constexpr int kBlockM = 128;                    // rows per CTA
  static constexpr int kTileM = kBlockM * kCtaGroup;     // MMA M
  static constexpr int kOutN = kForm == kGated ? kBlockN / 2 : kBlockN;   // columns of C
  static constexpr int kBlockK = kScaled ? 128 : 64;     // 128 bytes
  static constexpr int kBRows = kBlockN / kCtaGroup;     // rows of B this CTA loads
  static constexpr uint32_t kStageA = kBlockM * 128;
  static constexpr uint32_t kStageB = kBRows * 128;
  static constexpr uint32_t kBoxBytes = 64 * 64 * 2;     // nt: 64 x 64 boxes
  static constexpr int kBuffers = kScaled ? 512 / kBlockN : 2;   // of tensor memory
  static constexpr uint32_t kTmemCols = kBuffers * kBlockN;
  // kE4m3 pairs of 256 columns: a block is multiplied in two halves of N, each
  // handed over and back by itself, so that the tensor core has three halves to
  // go on with while one is being added (8192^3 391 us whole, 374 halved; with the
  // columns' own scales, whose sums take longer than the products, no faster).
  // A half is 64 of each CTA's rows of B: of the tile's columns the h-th 64 and
  // the h-th 64 after 128.
  static constexpr int kHalves = kForm == kE4m3 && kBlockN == 256 ? 2 : 1;
  static constexpr int kMmaN = kBlockN / kHalves;
  // e4m3: warps 1 and 3 multiply, every other block each
  static constexpr int kMultiplyWarps = kScaled ? 2 : 1;
  // e4m3: a ring of the blocks' scales. A block's are loaded with its operands.
  // Its slot is free once its sums are made; when the stage of block i is
  // loaded anew (with block i + kStages), block i has been multiplied, so the
  // one kBuffers before it has left tensor memory and the one before that has
  // been added: at most kStages + kBuffers + 1 blocks' scales are alive.
  static constexpr int kScaleSlots = kStages + kBuffers + 1;
  static constexpr uint32_t kAScaleBytes = kBlockM * 4;
  static constexpr uint32_t kBScaleBytes = kForm == kE4m3Rows ? kBlockN * 4 : (kBlockN + 127) / 128 * 16;
  static constexpr uint32_t kScaleStride = kForm == kE4m3Rows ? kAScaleBytes + kBScaleBytes : kAScaleBytes + 128;
  static constexpr uint32_t kStageScales = kScaled ? kAScaleBytes + kBScaleBytes : 0;
  static constexpr uint32_t kOffA = 0;
  static constexpr uint32_t kOffB = kOffA + kStages * kStageA;
  static constexpr uint32_t kOffStaging = kOffB + kStages * kStageB;
  static constexpr uint32_t kOffScale = kOffStaging + kEpilogueWarps * kStagingBytes;
  static constexpr uint32_t kOffBar = kOffScale + (kScaled ? kScaleSlots * kScaleStride : 0);
  static constexpr int kNumBars = 2 * kStages + 2 * kBuffers * kHalves + 1;   // full, empty, sum full, sum empty, drain
  static constexpr uint32_t kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
  static constexpr uint32_t kSmemBytes = kOffAbort + 4 + 1024;
  static constexpr uint32_t kIdesc = mma_idesc_f16(!kScaled && kBf16, kTileM, kMmaN, kForm == kNt) |
                                     (kForm == kNt ? 1u << 15 : 0u);
  static_assert(kStages <= 32, "issued phases fit a 32-bit mask");
  static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM columns");
  static_assert(kStageB % 1024 == 0 && kOffStaging % 1024 == 0, "swizzle atoms stay 1024-aligned");
  static_assert(kForm != kNt || kBRows % 64 == 0, "boxes of 64 columns");
  static_assert(kSmemBytes <= 232448, "fits the opt-in shared memory of one CTA");
};

// Tiles in groups of group_m tile rows, so that those running together share
// rows of A and of B in L2.
__device__ __forceinline__ void tile_at(const FfArgs& a, int tile, int& tm, int& tn) {
  const int per_group = a.group_m * a.num_n_tiles;
  const int first = tile / per_group * a.group_m;
  const int in = tile - first * a.num_n_tiles;
  const int rows = min(a.group_m, a.num_m_tiles - first);
  tn = in / rows;
  tm = first + in - tn * rows;
}

// A CTA's units of work: tiles over all of K, or (nt) parts of K of a tile.
struct Unit {
  int tm, tn, kb0, kb1, part;
};
template <bool kCut>
__device__ __forceinline__ Unit unit_at(const FfArgs& a, int unit) {
  Unit u;
  u.part = 0;
  u.kb0 = 0;
  u.kb1 = a.num_k_blocks;
  if (kCut && a.splits > 1) {
    const int tile = unit / a.splits;
    u.part = unit - tile * a.splits;
    u.kb0 = static_cast<int>(static_cast<int64_t>(u.part) * a.num_k_blocks / a.splits);
    u.kb1 = static_cast<int>(static_cast<int64_t>(u.part + 1) * a.num_k_blocks / a.splits);
    unit = tile;
  }
  tile_at(a, unit, u.tm, u.tn);
  return u;
}

// H of a chunk of 32 columns from its two projections (32 fp32 values a lane).
template <int kAct>
__device__ __forceinline__ void gate(const uint32_t (&g)[32], const uint32_t (&u)[32], float (&h)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) h[j] = act<kAct>(__uint_as_float(g[j])) * __uint_as_float(u[j]);
}

template <class T>
__global__ void __launch_bounds__(kThreads, 1) ff_gemm_kernel(const __grid_constant__ FfArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t base = smem_addr(smem);

  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = T::kCtaGroup == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  auto a_tile = [&](int s) { return base + T::kOffA + s * T::kStageA; };
  auto b_tile = [&](int s) { return base + T::kOffB + s * T::kStageB; };
  auto scales_at = [&](int s) { return base + T::kOffScale + static_cast<uint32_t>(s) * T::kScaleStride; };
  auto full_bar = [&](int s) { return base + T::kOffBar + 8u * s; };
  auto empty_bar = [&](int s) { return base + T::kOffBar + 8u * (T::kStages + s); };
  auto sum_full = [&](int b) { return base + T::kOffBar + 8u * (2 * T::kStages + b); };
  auto sum_empty = [&](int b) { return base + T::kOffBar + 8u * (2 * T::kStages + T::kBuffers * T::kHalves + b); };
  const uint32_t drain_bar = base + T::kOffBar + 8u * (2 * T::kStages + 2 * T::kBuffers * T::kHalves);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + T::kOffAbort);

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < T::kBuffers * T::kHalves; ++b) {
      mbar_init(sum_full(b), 1);
      mbar_init(sum_empty(b), T::kCtaGroup * kEpilogueWarps / T::kHalves);
    }
    mbar_init(drain_bar, T::kMultiplyWarps);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_descriptor(&args.tmap_a);
    tma_prefetch_descriptor(&args.tmap_b);
    if constexpr (T::kScaled) {
      tma_prefetch_descriptor(&args.tmap_as);
      tma_prefetch_descriptor(&args.tmap_bs);
    }
  }
  if (warp == kMultiply) {
    tmem_alloc<T::kCtaGroup>(smem_addr(tmem_slot), T::kTmemCols);
    tmem_relinquish<T::kCtaGroup>();
  }
  tc_fence_before_sync();
  if constexpr (T::kCtaGroup == 2) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // set-up may overlap the previous kernel in the stream; memory waits for it
  griddep_wait();
  if (args.alone == 0) griddep_launch_dependents();

  const Waiter<T::kCtaGroup> wd{args.status, args.timeout_ns, abort_flag};
  const int first_tile = static_cast<int>(blockIdx.x) / T::kCtaGroup;
  const int tile_step = static_cast<int>(gridDim.x) / T::kCtaGroup;

  if (warp < static_cast<uint32_t>(kFirstEpilogueWarp)) {
    if constexpr (T::kScaled) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kFewRegisters));
    const uint32_t elected = elect_one();
    if (warp == kLoadA || warp == kLoadB) {
      // ---------------------------------------------------------------- TMA producers, one for each operand
      int stage = 0, slot = 0;
      uint32_t phase = 0;
      Issued issued;
      bool ok = true;
      for (int tile = first_tile; ok && tile < args.num_tiles; tile += tile_step) {
        const Unit u = unit_at<T::kForm == kNt>(args, tile);
        const int tn = u.tn;
        const int a_row = u.tm * T::kTileM + static_cast<int>(rank) * T::kBlockM;
        const int b_row = tn * T::kOutN + static_cast<int>(rank) * T::kBRows;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!wd.warp_wait(empty_bar(stage), phase ^ 1u)) {
            ok = false;
            break;
          }
          const uint32_t bar = T::kCtaGroup == 2 ? map_to_cta(full_bar(stage), 0u) : full_bar(stage);
          auto load = [&](const CUtensorMap* map, uint32_t dst, int x, int y) {
            load_warp<T::kCtaGroup>(elected, map, dst, bar, x, y);
          };
          const int k0 = kb * T::kBlockK;
          const bool skip = kb == args.drop_load_kb && tile == first_tile;
          if (warp == kLoadA) {
            // the bytes of both operands, and of both CTAs of a pair
            if (leader && elected != 0) mbar_arrive_expect_tx(full_bar(stage), T::kCtaGroup * (T::kStageA + T::kStageB + T::kStageScales));
            __syncwarp();
            if (!skip) {
              if constexpr (T::kForm == kNt) {
#pragma unroll
                for (int j = 0; j < T::kBlockM / 64; ++j)
                  load(&args.tmap_a, a_tile(stage) + j * T::kBoxBytes, a_row + 64 * j, k0);
              } else {
                load(&args.tmap_a, a_tile(stage), k0, a_row);
                if constexpr (T::kScaled) load(&args.tmap_as, scales_at(slot), a_row, kb);
              }
            }
          } else if (!skip) {
            if constexpr (T::kForm == kNt) {
#pragma unroll
              for (int j = 0; j < T::kBRows / 64; ++j)
                load(&args.tmap_b, b_tile(stage) + j * T::kBoxBytes, b_row + 64 * j, k0);
            } else if constexpr (T::kForm != kGated) {
              load(&args.tmap_b, b_tile(stage), k0, b_row);
              // every CTA takes the scales of all the tile's columns
              if constexpr (T::kForm == kE4m3Rows) {
                load(&args.tmap_bs, scales_at(slot) + T::kAScaleBytes, tn * T::kOutN, kb);
              } else {
                load(&args.tmap_bs, scales_at(slot) + T::kAScaleBytes, kb & ~3, tn * (T::kBlockN / 128));
              }
            } else if constexpr (T::kCtaGroup == 2) {
              // the pair's halves of N: the gate's rows, the other projection's
              load(&args.tmap_b, b_tile(stage), k0, tn * T::kOutN + static_cast<int>(rank) * args.n);
            } else {
              load(&args.tmap_b, b_tile(stage), k0, b_row);
              load(&args.tmap_b, b_tile(stage) + T::kStageB / 2, k0, b_row + args.n);
            }
          }
          issued.record(stage, phase);
          if (++stage == T::kStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (T::kScaled && ++slot == T::kScaleSlots) slot = 0;
        }
      }
      // loads may still be landing if another role gave up
      for (int s = 0; s < T::kStages; ++s)
        if (leader && ((issued.issued >> s) & 1u)) wd.drain(full_bar(s), (issued.parity >> s) & 1u);
    } else if (leader && (warp == kMultiply || T::kMultiplyWarps == 2)) {
      // ---------------------------------------------------------------- MMA issuers
      // with two, each takes every other block (of all the CTA's tiles), and
      // the waits of one run beside the other's
      int stage = static_cast<int>(warp) >> 1, buf = static_cast<int>(warp) >> 1;   // warp 1: 0, warp 3: 1
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      int first_kb = stage;
      for (int tile = first_tile; ok && tile < args.num_tiles; tile += tile_step) {
        int kb = first_kb, begin = 0, end = args.num_k_blocks;
        if constexpr (T::kForm == kNt) {
          const Unit u = unit_at<true>(args, tile);
          kb = begin = u.kb0;
          end = u.kb1;
        }
        for (; kb < end; kb += T::kMultiplyWarps) {
          // a step along K: 32 bytes of a K-major row, or two 8-row groups of an MN-major tile
          constexpr uint32_t kStep = T::kForm == kNt ? 2048u >> 4 : 2u;
          const uint64_t a_desc = T::kForm == kNt ? sw128_mnmajor_desc(a_tile(stage), T::kBoxBytes)
                                                  : sw128_kmajor_desc(a_tile(stage));
          const uint64_t b_desc = T::kForm == kNt ? sw128_mnmajor_desc(b_tile(stage), T::kBoxBytes)
                                                  : sw128_kmajor_desc(b_tile(stage));
#pragma unroll
          for (int h = 0; h < T::kHalves; ++h) {
            const int sum = buf * T::kHalves + h;
            if (ok && (T::kScaled || kb == begin)) ok = wd.warp_wait(sum_empty(sum), buf_phase ^ 1u);
            if (ok && h == 0) ok = wd.warp_wait(full_bar(stage), phase);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + static_cast<uint32_t>(sum * T::kMmaN);
            constexpr uint32_t kHalfRows = T::kBRows / T::kHalves * 128u >> 4;   // of this CTA's rows of B
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_warp<T::kCtaGroup, T::kScaled>(elected, d, a_desc + kStep * kk, b_desc + kHalfRows * h + kStep * kk, T::kIdesc,
                                                 kk > 0 || (!T::kScaled && kb > begin) ? 1u : 0u);
            if (h == T::kHalves - 1) commit_warp<T::kCtaGroup>(elected, empty_bar(stage), 0x3);
            if (T::kScaled || kb == end - 1) commit_warp<T::kCtaGroup>(elected, sum_full(sum), 0x3);
          }
          if (!ok) break;
          stage += T::kMultiplyWarps;
          if (stage >= T::kStages) {
            stage -= T::kStages;
            phase ^= 1u;
          }
          if (T::kScaled || kb == end - 1) {
            buf += T::kMultiplyWarps;
            if (buf >= T::kBuffers) {
              buf -= T::kBuffers;
              buf_phase ^= 1u;
            }
          }
        }
        first_kb = kb - args.num_k_blocks;
      }
      // what was issued here finishes before tensor memory is freed
      commit_warp<T::kCtaGroup>(elected, drain_bar, 0x1);
      wd.drain(drain_bar, 0);
    }
    __syncwarp();
  } else {
    if constexpr (T::kScaled) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kManyRegisters));
    // ------------------------------------------------------------------ epilogue
    const uint32_t quarter = warp & 3u;
    const int epilogue_warp = static_cast<int>(warp) - kFirstEpilogueWarp;
    const int half = epilogue_warp >> 2;
    uint8_t* staging = smem + T::kOffStaging + static_cast<uint32_t>(epilogue_warp) * kStagingBytes;
    const uint32_t sum_empty0 = T::kCtaGroup == 2 ? map_to_cta(sum_empty(0), 0u) : sum_empty(0);
    int buf = 0, slot = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    // this warp's sums: all of a buffer's, or the half that is its own
    auto my_sum = [&]() { return T::kHalves == 2 ? 2 * buf + half : buf; };
    auto hand_back = [&]() {   // they are in registers: the MMA warp may write them again
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (T::kCtaGroup == 2) {
          arrive_remote(sum_empty0 + 8u * my_sum());
        } else {
          mbar_arrive(sum_empty(my_sum()));
        }
      }
      if (++buf == T::kBuffers) {
        buf = 0;
        buf_phase ^= 1u;
      }
    };
    for (int tile = first_tile; ok && tile < args.num_tiles; tile += tile_step) {
      const Unit unit = unit_at<T::kForm == kNt>(args, tile);
      const int row0 = unit.tm * T::kTileM + static_cast<int>(rank) * T::kBlockM + static_cast<int>(quarter) * 32;
      const int col0 = unit.tn * T::kOutN;
      const uint32_t t_quarter = tmem_base + ((quarter * 32u) << 16);

      if constexpr (T::kScaled) {
        // this warp's half of the columns; a thread's sums: its row's, two to a register pair
        constexpr int kCols = T::kBlockN / 2;
        // column of the tile of the thread's x-th sum
        auto column = [&](int x) {
          if constexpr (T::kHalves == 2) return half * 64 + (x < 64 ? x : x + 64);
          return half * kCols + x;
        };
        const uint32_t t_mine = t_quarter + static_cast<uint32_t>(half * kCols);
        uint64_t sum[kCols / 2];
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) sum[j] = 0;
#pragma unroll 1
        for (int kb = 0; kb < args.num_k_blocks; ++kb) {
          if (!wd.warp_wait(sum_full(my_sum()), buf_phase)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t t = t_mine + static_cast<uint32_t>(buf * T::kBlockN);
          uint32_t v[2][16];
          tmem_load_32x16(t, v[0]);
          // (the block has been multiplied, so its scales have landed too)
          const float* scales = reinterpret_cast<const float*>(smem + T::kOffScale + static_cast<uint32_t>(slot) * T::kScaleStride);
          const float* cols = scales + T::kBlockM;
          if (++slot == T::kScaleSlots) slot = 0;
          const float row_scale = scales[quarter * 32u + lane];
          uint64_t scale2[T::kHalves];   // kE4m3: by the columns' 128-row block of B
#pragma unroll
          for (int x = 0; x < T::kHalves; ++x) {
            const float scale = T::kForm == kE4m3 ? row_scale * cols[x * 4 + (kb & 3)] : row_scale;
            scale2[x] = f32x2_pack(scale, scale);
          }
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            uint64_t both[8];   // the columns' scales times the row's, while tensor memory answers
            if constexpr (T::kForm == kE4m3Rows) {
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(cols + column(c * 16) + 2 * j);
                both[j] = f32x2_mul(b.x, scale2[0]);
                both[j + 1] = f32x2_mul(b.y, scale2[0]);
              }
            }
            uint32_t(&x)[16] = v[c & 1];
            tmem_loaded(x);
            if (c + 1 < kCols / 16) {
              tmem_load_32x16(t + 16u * (c + 1), v[(c + 1) & 1]);
            } else {
              hand_back();
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint64_t p = f32x2_pack(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
              sum[c * 8 + j] = f32x2_fma(p, T::kForm == kE4m3 ? scale2[c * 16 * T::kHalves / kCols] : both[j], sum[c * 8 + j]);
            }
          }
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          float out[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) f32x2_unpack(sum[c * 16 + j], out[2 * j], out[2 * j + 1]);
          if (col0 + column(c * 32) < args.n) store_block(args, row0, col0 + column(c * 32), out, staging);
        }
      } else {
        // chunks of 32 columns of C, alternately this warp's and its partner's
        constexpr int kChunks = T::kOutN / 32;
        if (!__all_sync(0xffffffffu, wd.wait(sum_full(buf), buf_phase))) break;
        tc_fence_after_sync();
        const uint32_t t = t_quarter + static_cast<uint32_t>(buf * T::kBlockN);
#pragma unroll 1
        for (int c = half; c < kChunks; c += 2) {
          const int col = col0 + c * 32;
          uint32_t v[32];
          tmem_load_32x32(t + 32u * c, v);
          if constexpr (T::kForm == kGated) {
            uint32_t u[32];
            tmem_load_32x32(t + T::kOutN + 32u * c, u);
            tmem_loaded(v);
            tmem_loaded(u);
            if (c + 2 >= kChunks) hand_back();
            if (col >= args.n) continue;
            if (args.pre != nullptr) {
              uint32_t p[16];
              uint16_t* pre = static_cast<uint16_t*>(args.pre) + static_cast<int64_t>(row0) * args.ldp + col;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                p[j] = pack16<T::kBf16>(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
              store_rows<2>(pre, args.ldp, args.m - row0, args.n - col, p, false, staging);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                p[j] = pack16<T::kBf16>(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
              store_rows<2>(pre + args.n, args.ldp, args.m - row0, args.n - col, p, false, staging);
            }
            float h[32];
            if (args.activation == kSilu) {
              gate<kSilu>(v, u, h);
            } else if (args.activation == kGelu) {
              gate<kGelu>(v, u, h);
            } else {
              gate<kRelu>(v, u, h);
            }
            store_block(args, row0, col, h, staging);
          } else {
            tmem_loaded(v);
            if (c + 2 >= kChunks) hand_back();
            if (col >= args.n) continue;
            float out[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) out[j] = __uint_as_float(v[j]);
            store_block(args, row0, col, out, staging, unit.part * args.part_stride);
          }
        }
      }
    }
    __syncwarp();
  }

  // ------------------------------------------------------------------ teardown
  tc_fence_before_sync();
  if constexpr (T::kCtaGroup == 2) {
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == kMultiply) {
    tc_fence_after_sync();
    tmem_dealloc<T::kCtaGroup>(tmem_base, T::kTmemCols);
  }
}

}  // namespace ff
}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

template <class T>
struct FfLauncher {
  static cudaError_t fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int grid, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> done_mask{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done_mask.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(gemm_tn_dev::ff::ff_gemm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(T::kSmemBytes));
      if (e != cudaSuccess) return e;
      done_mask.fetch_or(bit, std::memory_order_acq_rel);
    }
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(gemm_tn_dev::ff::kThreads);
    cfg.dynamicSmemBytes = T::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (T::kCtaGroup == 2) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attr[cfg.numAttrs].val.clusterDim.x = 2;
      attr[cfg.numAttrs].val.clusterDim.y = 1;
      attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    return cudaSuccess;
  }

  static cudaError_t launch(const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    cudaError_t e = fill(cfg, attr, grid, stream);
    if (e != cudaSuccess) return e;
    if (dependent_launch_enabled()) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, gemm_tn_dev::ff::ff_gemm_kernel<T>, args);
  }

  static int resident(int sms) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    if (fill(cfg, attr, sms - sms % T::kCtaGroup, nullptr) != cudaSuccess) return 0;
    if (T::kCtaGroup == 1) return sms;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, gemm_tn_dev::ff::ff_gemm_kernel<T>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return clusters;
  }
};

}  // namespace gemm_tn_impl

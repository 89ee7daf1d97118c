// sm103_cache_weigh.cu -- accumulated attention weight of cached keys
// (include/kv_cache.h: kv_cache_weigh):
//
//   weight_out[b][h][s] = weight[b][h][s]
//       + sum over counted tokens i and the query heads x of KV head h of
//         exp(scale * q_(i,x) . k_s - lse_(i,x)),     s seen by i
//
// The transposed product S^T = K Q^T puts a key on each TMEM lane and the query
// rows on its columns: a thread owns one key, sums its columns in registers and
// is the only one that writes the key's weight. No maximum is needed (lse is
// given), no reduction crosses threads, no atomics are used, and what lies
// behind the last key stays on its own lanes.
//
// Keys are read once (dim * 2 bytes each) per 256 query rows against one
// exponential per key and row: up to about 150 rows HBM bounds the kernel,
// past that the exponentials do. GB300: 32 tokens of 32 heads over 8 KV heads
// (128 rows), dim 128, 8 sequences of 9001 to 16384 slots, 231 MB: 43.7 us, 5.3
// TB/s; one token of 16 heads of dim 64, 4 sequences of 300 to 1024 slots: 7.3.
//
// Work: an item is (sequence, KV head); the items' 128-key tiles, laid end to end
// a change of items apart, are cut into equal contiguous chunks, one per CTA
// (sm103_cache.cuh). Per segment of an item the query rows come in blocks of at
// most 256, each block walking the segment's tiles.
//   warp 0      TMA producer (lane l copies the tile's l-th page)
//   warp 1      MMA issuer: S^T (128 keys x up to 128 rows) into one of the two
//               TMEM buffers of the group that takes the tile, so that the next
//               product runs while the group sums the one before
//   warps 2-9   two groups of four taking every other tile; all eight gather a
//               block's query rows into shared memory first, but
//   warp 10     gathers those of blocks of up to 128 rows behind another such: these
//               lie in the buffer's halves in turn, and are there when the block
//               before ends (in between, the gathering's two round trips to memory
//               stand still for 4 us: 40 sequences of up to 1000 slots 29.5 -> 23.5)
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "kv_cache_internal.h"
#include "sm103_cache.cuh"

namespace gemm_tn_dev {

namespace cw {

using cache::kTileKeys;
constexpr int kProducerWarp = 0;
constexpr int kMmaWarp = 1;
constexpr int kFirstSumWarp = 2;
constexpr int kSumWarps = 8;
constexpr int kGatherWarp = kFirstSumWarp + kSumWarps;
constexpr int kMaxRows = 256;      // query rows per block
constexpr int kHalf = 128;         // query rows per product (columns of one of the four TMEM buffers)
constexpr float kLog2e = 1.4426950408889634f;

template <int kDim_, bool kBf16_>
struct Cfg {
  static constexpr int kDim = kDim_;
  static constexpr bool kBf16 = kBf16_;
  static constexpr int kNumThreads = 32 * (kGatherWarp + 1);
  static constexpr int kDimBoxes = kDim / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;        // 128 keys x 128 bytes
  static constexpr uint32_t kTileBytes = kDimBoxes * kBoxBytes;
  static constexpr uint32_t kQBoxBytes = kMaxRows * 128u;   // 256 query rows x 128 bytes
  static constexpr int kStages = kDim == 64 ? 8 : 4;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kOffQ + kDimBoxes * kQBoxBytes;
  static constexpr uint32_t kOffLse = kOffK + kStages * kTileBytes;   // [256] -log2e lse, rounded; [256] 2^ what that left
  // q_full[2], q_free[2], k_full[S], k_empty[S], s_full[2][2], s_empty[2][2], drain
  static constexpr int kNumBars = 4 + 2 * kStages + 8 + 1;
  static constexpr uint32_t kOffBar = kOffLse + 8u * kMaxRows;
  static constexpr uint32_t kOffTmemSlot = kOffBar + 8u * kNumBars;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4u;
  static constexpr uint32_t kOffStart = kOffAbort + 4u;   // the chunk's first Walk
  static constexpr uint32_t kOffSums = kOffStart + 32u;   // 32 words of the search for it
  static constexpr uint32_t kSmemBytes = kOffSums + 128u + 1024u;   // + slack to align the base to 1024
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdesc = mma_idesc_f16(kBf16, kTileKeys, 0, false);   // N is set per block
  static_assert(kSmemBytes <= 227u * 1024u, "shared memory budget");
  static_assert(kOffBar % 8u == 0, "64-bit shared words");
};

__device__ __forceinline__ int cached_len(const WeighArgs& a, int b) {
  return min(max(__ldg(a.lens + b), 0), a.capacity);
}
__device__ __forceinline__ int row_count(const WeighArgs& a, int b) {
  return a.counts == nullptr ? a.max_rows : min(max(__ldg(a.counts + b), 0), a.max_rows);
}

// Which of the query buffer's halves the blocks take: those of up to 128 rows one
// in turn, wider ones both. Every role that uses the buffer keeps one of these.
// (One word: it lives across the tile loop, which has no registers to spare.)
struct Halves {
  // bits 0, 1: parity of the blocks that have taken each half; 2: whose turn it
  // is; 3: the block at hand is wide (as none is before the first); 4: the one before was
  uint32_t state = 8u;

  __device__ __forceinline__ void take(int cols) {
    state = (state & 7u) | (cols > kHalf ? 8u : 0u) | ((state & 8u) << 1);
  }
  __device__ __forceinline__ bool wide() const { return (state & 8u) != 0; }
  __device__ __forceinline__ int turn() const { return static_cast<int>(state >> 2) & 1; }
  __device__ __forceinline__ int first() const { return wide() ? 0 : turn() * kHalf; }   // buffer row
  __device__ __forceinline__ bool has(int half) const { return wide() || half == turn(); }
  __device__ __forceinline__ uint32_t phase(int half) const { return (state >> half) & 1u; }
  // Whether the block's half is free while the block before is used.
  __device__ __forceinline__ bool ahead() const { return (state & 24u) == 0; }
  __device__ __forceinline__ void leave() { state ^= wide() ? 3u : 4u | (1u << turn()); }
};

// Walks a chunk: runs of one (sequence, KV head)'s key tiles.
struct Walk {
  int b, h, j0, len, n, tiles, left, count;

  // The walk that begins at place `off` of sequence b: each of its items' tiles
  // lie behind `gap` places that stand for the time a change of items costs.
  __device__ __forceinline__ void start(const WeighArgs& a, int b_, int off, int left_) {
    b = b_;
    load(a);
    h = off / (tiles + a.gap);
    j0 = off - (tiles + a.gap) * h - a.gap;
    left = left_ + min(j0, 0);
    j0 = max(j0, 0);
    count = min(tiles - j0, left);
  }
  __device__ __forceinline__ void load(const WeighArgs& a) {
    len = cached_len(a, b);
    n = row_count(a, b);
    tiles = (len + kTileKeys - 1) / kTileKeys;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const WeighArgs& a) {
    left -= count;
    if (left <= 0) return;
    j0 = 0;
    if (++h == a.kv_heads) {
      h = 0;
      do {
        ++b;
        load(a);
      } while (tiles == 0);
    }
    left -= a.gap;
    count = min(tiles, left);
  }
  // blocks of query rows; one empty block where no token counts (the weights are still copied)
  __device__ __forceinline__ int blocks(const WeighArgs& a) const {
    return max(1, (n + a.block_tokens - 1) / a.block_tokens);
  }
  __device__ __forceinline__ int block_rows(const WeighArgs& a, int block) const {
    return max(0, min(a.block_tokens, n - block * a.block_tokens)) * a.group;
  }
};

}  // namespace cw

template <class C>
__global__ void __launch_bounds__(C::kNumThreads, 1) cache_weigh_kernel(const __grid_constant__ WeighArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t base = smem_addr(smem);
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();

  auto k_tile = [&](int s) { return base + C::kOffK + s * C::kTileBytes; };
  auto bar = [&](int i) { return base + C::kOffBar + 8u * i; };
  auto q_full = [&](int half) { return bar(half); };
  auto q_free = [&](int half) { return bar(2 + half); };
  auto k_full = [&](int s) { return bar(4 + s); };
  auto k_empty = [&](int s) { return bar(4 + C::kStages + s); };
  auto s_full = [&](int g, int buf) { return bar(4 + 2 * C::kStages + 2 * g + buf); };
  auto s_empty = [&](int g, int buf) { return bar(8 + 2 * C::kStages + 2 * g + buf); };
  const uint32_t drain_bar = bar(12 + 2 * C::kStages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
  cw::Walk* start_walk = reinterpret_cast<cw::Walk*>(smem + C::kOffStart);
  int* sums = reinterpret_cast<int*>(smem + C::kOffSums);
  float* row_ref = reinterpret_cast<float*>(smem + C::kOffLse);
  float* row_factor = row_ref + cw::kMaxRows;

  if (threadIdx.x == 0) {
    for (int half = 0; half < 2; ++half) {
      mbar_init(q_full(half), cw::kSumWarps + 1);   // whoever gathers, all of them arrive
      mbar_init(q_free(half), cw::kSumWarps);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(s_full(x >> 1, x & 1), 1);
      mbar_init(s_empty(x >> 1, x & 1), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    start_walk->left = 0;
    fence_barrier_init();
  }
  if (warp == cw::kProducerWarp && lane == 0) tma_prefetch_descriptor(&args.tmap_k);
  if (warp == cw::kMmaWarp) {
    tmem_alloc<1>(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish<1>();
  }
  griddep_wait();
  griddep_launch_dependents();
  cache::find_start(
      args.batch, args.chunks, args.min_chunk, args.gap, static_cast<int>(blockIdx.x), sums,
      [&](int b) {
        const int tiles = (cw::cached_len(args, b) + cw::kTileKeys - 1) / cw::kTileKeys;
        return tiles > 0 ? (tiles + args.gap) * args.kv_heads : 0;
      },
      [&](int b, int, int off, int left, int) {
        cw::Walk w;
        w.start(args, b, off, left);
        *start_walk = w;
      });
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const cache::Watch<false> wd{args.status, args.timeout_ns, abort_flag};
  cw::Walk w = *start_walk;

  if (warp == cw::kProducerWarp) {
    // -------------------------------------------------------------- TMA producer
    cache::Issued issued;
    const int box_rows = min(args.page_size, cw::kTileKeys);
    const int tile_pages = cw::kTileKeys / box_rows;
    int it = 0;
    bool ok = true;
    for (; ok && w.more(); w.next(args)) {
      const int32_t* table = args.page_table + static_cast<int64_t>(w.b) * args.table_stride;
      auto page_of = [&](int j) {   // the page that this lane copies of tile j
        const int first = j * cw::kTileKeys + static_cast<int>(lane) * box_rows;
        if (static_cast<int>(lane) >= tile_pages || first >= w.len) return 0;
        int page = __ldg(table + first / args.page_size);
        if (page < 0 || page >= args.num_pages) {   // not a page: the copy fills zeros, the caller is told
          cache::report(args.status, cache::kStatusInvalid);
          page = args.num_pages;
        }
        return page;
      };
      const int blocks = w.blocks(args);
      for (int block = 0; ok && block < blocks; ++block) {
        int page = page_of(w.j0);
        for (int j = w.j0; j < w.j0 + w.count; ++j, ++it) {
          const int valid = min(cw::kTileKeys, w.len - j * cw::kTileKeys);
          const int boxes = (valid + box_rows - 1) / box_rows;
          const int slot0 = tile_pages == 1 ? (j * cw::kTileKeys) % args.page_size : 0;
          const int next_page = j + 1 < w.j0 + w.count ? page_of(j + 1) : 0;
          const int s = it % C::kStages;
          const uint32_t ph = static_cast<uint32_t>(it / C::kStages) & 1u;
          if (!(ok = wd.warp_wait(k_empty(s), ph ^ 1u))) break;
          if (lane == 0) mbar_arrive_expect_tx(k_full(s), static_cast<uint32_t>(boxes * box_rows) * 128u * C::kDimBoxes);
          __syncwarp();
          if (static_cast<int>(lane) < boxes && !(blockIdx.x == 0 && it == args.drop_load_block)) {
            for (int c = 0; c < C::kDimBoxes; ++c)
              tma_load_4d(&args.tmap_k, k_tile(s) + c * C::kBoxBytes + lane * box_rows * 128u, k_full(s), 64 * c, w.h,
                          slot0, page);
          }
          issued.note(s, ph);
          page = next_page;
        }
      }
    }
    // wait (bounded) for every copy issued before the CTA may exit
    issued.drain(wd, C::kStages, k_full);
  } else if (warp == cw::kMmaWarp) {
    {
      // ------------------------------------------------------------ MMA issuer
      // (the whole warp runs this, one lane issues)
      const uint32_t leader = elect_one();
      int it = 0;       // tiles issued
      cw::Halves halves;
      int used[2] = {0, 0};   // products of each group so far
      bool ok = true;
      for (; ok && w.more(); w.next(args)) {
        const int blocks = w.blocks(args);
        for (int block = 0; ok && block < blocks; ++block, halves.leave()) {
          const int cols = max(1, (w.block_rows(args, block) + 31) / 32) * 32;
          halves.take(cols);
          for (int half = 0; half < 2 && ok; ++half)
            if (halves.has(half)) ok = wd.warp_wait(q_full(half), halves.phase(half));
          for (int j = 0; ok && j < w.count; ++j, ++it) {
            const int s = it % C::kStages, g = it & 1;
            if (!(ok = wd.warp_wait(k_full(s), static_cast<uint32_t>(it / C::kStages) & 1u))) break;
            for (int c0 = 0; c0 < cols; c0 += cw::kHalf) {   // halves of the query rows
              const int buf = used[g] & 1;
              if (!(ok = wd.warp_wait(s_empty(g, buf), (static_cast<uint32_t>(used[g] >> 1) & 1u) ^ 1u))) break;
              tc_fence_after_sync();
              const uint32_t idesc = C::kIdesc | ((static_cast<uint32_t>(min(cols - c0, cw::kHalf)) >> 3) << 17);
              const uint32_t t_s = tmem_base + 256u * static_cast<uint32_t>(g) + cw::kHalf * static_cast<uint32_t>(buf);
#pragma unroll
              for (int c = 0; c < C::kDimBoxes; ++c) {
                const uint64_t a_desc = sw128_kmajor_desc(k_tile(s) + c * C::kBoxBytes);
                const uint64_t b_desc = sw128_kmajor_desc(base + C::kOffQ + c * C::kQBoxBytes + static_cast<uint32_t>(halves.first() + c0) * 128u);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_f16_warp(leader, t_s, a_desc + 2u * kk, b_desc + 2u * kk, idesc, (c | kk) != 0 ? 1u : 0u);
              }
              mma_commit_warp(leader, s_full(g, buf));
              ++used[g];
            }
            if (ok) mma_commit_warp(leader, k_empty(s));
          }
        }
      }
      // every MMA issued here must finish before TMEM is freed
      mma_commit_warp(leader, drain_bar);
      wd.drain(drain_bar, 0);
    }
  } else if (warp == cw::kGatherWarp) {
    // -------------------------------------------------------------- query rows
    // K-major with the 128-byte swizzle. A lane looks up the rows of its number,
    // four at a time; the warp then copies them, 16 bytes a lane.
    constexpr int kPieces = C::kDim / 8;   // 16-byte pieces per row
    constexpr int kAtOnce = 32 / kPieces;  // rows that the warp copies at a time
    const int piece = static_cast<int>(lane) % kPieces, sub = static_cast<int>(lane) / kPieces;
    cw::Halves halves;
    bool ok = true;
    for (; ok && w.more(); w.next(args)) {
      const int blocks = w.blocks(args);
      const uint16_t* q = static_cast<const uint16_t*>(args.q) + w.b * args.q_batch + w.h * args.group * args.q_head + 8 * piece;
      for (int block = 0; ok && block < blocks; ++block, halves.leave()) {
        const int rows = w.block_rows(args, block);
        const int cols = max(1, (rows + 31) / 32) * 32;
        halves.take(cols);
        for (int half = 0; half < 2 && ok; ++half)   // every sum warp is done with the block that was there
          if (halves.has(half)) ok = wd.patient_wait(q_free(half), halves.phase(half) ^ 1u);
        if (!ok) break;
        if (halves.ahead()) {   // at most 128 rows
          int token[4];
          int64_t from[4];   // where the row begins, in elements; -1: a row that does not count
          float lse[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 32 * x + static_cast<int>(lane);
            token[x] = -1;
            if (row < rows) {
              token[x] = block * args.block_tokens + row / args.group;   // of the counted tokens
              if (args.rows != nullptr) token[x] = __ldg(args.rows + static_cast<int64_t>(w.b) * args.max_rows + token[x]);
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 32 * x + static_cast<int>(lane), head = row % args.group;
            from[x] = -1;
            lse[x] = INFINITY;   // rows that do not count weigh nothing
            if (row < rows) {
              if (token[x] < 0 || token[x] >= args.tokens) {
                cache::report(args.status, cache::kStatusInvalid);
              } else {
                from[x] = token[x] * args.q_token + head * args.q_head;
                lse[x] = __ldg(args.lse + (static_cast<int64_t>(w.b) * args.tokens + token[x]) * args.heads + w.h * args.group + head);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (32 * x >= cols) break;
#pragma unroll 4
            for (int r = sub; r < 32; r += kAtOnce) {
              const int64_t at = __shfl_sync(0xffffffffu, from[x], r);
              const int row = halves.first() + 32 * x + r;
              const uint32_t to = base + C::kOffQ + (piece / 8) * C::kQBoxBytes + row * 128u + (((piece & 7) ^ (row & 7)) * 16u);
              if (at >= 0) cp_async_16(to, q + at);
              else st_shared_v4(to, 0u, 0u, 0u, 0u);
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (32 * x >= cols) break;
            // lse * log2e as a rounded part and the factor that makes up for the rounding
            const int row = halves.first() + 32 * x + static_cast<int>(lane);
            const float hi = lse[x] * cw::kLog2e;
            const float lo = fmaf(lse[x], cw::kLog2e, -hi);
            row_ref[row] = isinf(hi) ? -INFINITY : -hi;
            row_factor[row] = isinf(hi) ? 0.0f : ex2_approx(-lo);
          }
        }
        cp_async_wait_all();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0)
          for (int half = 0; half < 2; ++half)
            if (halves.has(half)) mbar_arrive(q_full(half));
      }
    }
  } else {
    // -------------------------------------------------------------- sums
    const int g = (static_cast<int>(warp) - cw::kFirstSumWarp) >> 2;   // group: tiles it & 1 == g
    const uint32_t quarter = warp & 3u;
    const int key_lane = static_cast<int>(quarter * 32u + lane);
    const uint32_t t_s = tmem_base + ((quarter * 32u) << 16) + 256u * static_cast<uint32_t>(g);
    const float c_log2 = args.scale_log2;
    const int sum_thread = static_cast<int>(threadIdx.x) - 64;
    cw::Halves halves;
    int it = 0;
    int used = 0;   // products of this group so far
    bool ok = true;
    for (; ok && w.more(); w.next(args)) {
      const int blocks = w.blocks(args);
      const int64_t weight_row = (static_cast<int64_t>(w.b) * args.kv_heads + w.h) * args.capacity;
      for (int block = 0; ok && block < blocks; ++block, halves.leave()) {
        const int cols = max(1, (w.block_rows(args, block) + 31) / 32) * 32;
        const int first_row = block * args.block_tokens;   // of the counted tokens
        halves.take(cols);
        const bool ahead = halves.ahead();
        if (!ahead) {
          // every sum warp is done with the block that was there: between them they
          // have seen all its products complete and read its rows' references
          for (int half = 0; half < 2 && ok; ++half)
            if (halves.has(half)) ok = wd.warp_wait(q_free(half), halves.phase(half) ^ 1u);
          if (!ok) break;
          const int rows = w.block_rows(args, block);
          // query rows -> shared memory, K-major with the 128-byte swizzle, four or
          // eight pieces a thread at a time: their loads are in flight together
          // (eight where four would take two rounds: 128 rows of dim 128 over 8
          // sequences of up to 16384 slots 44.5 -> 44.0 us; eight always makes 32
          // rows 1 to 12% slower, whose code it lengthens)
          constexpr int kPieces = C::kDim / 8;   // 16-byte pieces per row
          constexpr int kRowStep = 32 * cw::kSumWarps / kPieces;
          const int piece = sum_thread % kPieces;
          auto gather = [&](auto batch) {
            constexpr int kBatch = batch.value;
            for (int row0 = sum_thread / kPieces; row0 < cols; row0 += kBatch * kRowStep) {
              int token[kBatch], head[kBatch];
              uint4 v[kBatch];
              float lse[kBatch];
#pragma unroll
              for (int x = 0; x < kBatch; ++x) {
                const int row = row0 + x * kRowStep, i = row / args.group;
                head[x] = w.h * args.group + row - i * args.group;
                token[x] = first_row + i;
                if (row >= rows) token[x] = -1;
                else if (args.rows != nullptr) {
                  token[x] = __ldg(args.rows + static_cast<int64_t>(w.b) * args.max_rows + token[x]);
                  if (token[x] < 0 || token[x] >= args.tokens) {
                    cache::report(args.status, cache::kStatusInvalid);
                    token[x] = -1;
                  }
                }
              }
#pragma unroll
              for (int x = 0; x < kBatch; ++x) {
                v[x] = make_uint4(0u, 0u, 0u, 0u);
                lse[x] = INFINITY;   // rows that do not count weigh nothing
                if (token[x] >= 0) {
                  v[x] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(args.q) + w.b * args.q_batch +
                                                              token[x] * args.q_token + head[x] * args.q_head) + piece);
                  if (piece == 0)
                    lse[x] = __ldg(args.lse + (static_cast<int64_t>(w.b) * args.tokens + token[x]) * args.heads + head[x]);
                }
              }
#pragma unroll
              for (int x = 0; x < kBatch; ++x) {
                const int row = row0 + x * kRowStep;
                if (row >= cols) break;
                st_shared_v4(base + C::kOffQ + (piece / 8) * C::kQBoxBytes + (halves.first() + row) * 128u + (((piece & 7) ^ (row & 7)) * 16u),
                             v[x].x, v[x].y, v[x].z, v[x].w);
                if (piece == 0) {
                  // lse * log2e as a rounded part and the factor that makes up for the rounding
                  const float hi = lse[x] * cw::kLog2e;
                  const float lo = fmaf(lse[x], cw::kLog2e, -hi);
                  row_ref[halves.first() + row] = isinf(hi) ? -INFINITY : -hi;
                  row_factor[halves.first() + row] = isinf(hi) ? 0.0f : ex2_approx(-lo);
                }
              }
            }
          };
          if (cols > 4 * kRowStep) gather(std::integral_constant<int, 8>{});
          else gather(std::integral_constant<int, 4>{});
          fence_proxy_async_shared();
        }
        __syncwarp();
        if (lane == 0)
          for (int half = 0; half < 2; ++half)
            if (halves.has(half)) mbar_arrive(q_full(half));
        for (int half = 0; half < 2 && ok; ++half)
          if (halves.has(half)) ok = wd.warp_wait(q_full(half), halves.phase(half));
        if (!ok) break;
        const float* block_ref = row_ref + halves.first();   // and as far behind it as row_factor is
        for (int j = w.j0; ok && j < w.j0 + w.count; ++j, ++it) {
          if ((it & 1) != g) continue;
          const int key = j * cw::kTileKeys + key_lane;
          const bool live = key < w.len;
          float acc = 0.0f;
          if (live) acc = block == 0 ? args.weight[weight_row + key] : args.weight_out[weight_row + key];
          // causal: counted token i sees the key from i = key - (len - n) on;
          // low: the first column of this block that does
          const int first_token = args.causal ? key - (w.len - w.n) - first_row : 0;
          const int low = first_token > 0 ? min(first_token, args.block_tokens) * args.group : 0;
          const bool masked = __any_sync(0xffffffffu, live && low > 0);
          // two columns an instruction: p = 2^(s c - ref), sum += p factor. The next
          // 32 columns come from tensor memory while these are worked on.
          const uint64_t cc = f32x2_pack(c_log2, c_log2);
          uint64_t sum01, sum23;
          uint32_t raw[2][32];
          auto columns = [&](const uint32_t (&x)[32], int c0, auto mask) {
            uint32_t hidden = 0;   // columns that weigh nothing (factor 0), and that do not see the key
            if constexpr (mask.value)
              hidden = __ballot_sync(0xffffffffu, block_ref[cw::kMaxRows + c0 + static_cast<int>(lane)] == 0.0f) | cache::low_bits(low - c0);
            const ulonglong2* refs = reinterpret_cast<const ulonglong2*>(block_ref + c0);
            const ulonglong2* factors = reinterpret_cast<const ulonglong2*>(block_ref + cw::kMaxRows + c0);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const ulonglong2 ref = refs[e / 4], f = factors[e / 4];
              float p0, p1, p2, p3;
              f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), cc, ref.x), p0, p1);
              f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), cc, ref.y), p2, p3);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              p2 = ex2_approx(p2);
              p3 = ex2_approx(p3);
              if constexpr (mask.value) {
                if ((hidden >> e) & 1u) p0 = 0.0f;
                if ((hidden >> (e + 1)) & 1u) p1 = 0.0f;
                if ((hidden >> (e + 2)) & 1u) p2 = 0.0f;
                if ((hidden >> (e + 3)) & 1u) p3 = 0.0f;
              }
              sum01 = f32x2_fma(f32x2_pack(p0, p1), f.x, sum01);
              sum23 = f32x2_fma(f32x2_pack(p2, p3), f.y, sum23);
            }
          };
          // this key's sum over the columns c0 .. of a half, end - c0 of them
          auto half = [&](uint32_t t_buf, int c0, int end, auto mask) {
            sum01 = sum23 = f32x2_pack(0.0f, 0.0f);
            tmem_load_32x32(t_buf, raw[0]);
            for (; c0 < end; c0 += 64, t_buf += 64u) {
              tmem_load_wait();
              if (c0 + 32 < end) tmem_load_32x32(t_buf + 32u, raw[1]);
              columns(raw[0], c0, mask);
              if (c0 + 32 < end) {
                tmem_load_wait();
                if (c0 + 64 < end) tmem_load_32x32(t_buf + 64u, raw[0]);
                columns(raw[1], c0 + 32, mask);
              }
            }
            float sum0, sum1, sum2, sum3;
            f32x2_unpack(sum01, sum0, sum1);
            f32x2_unpack(sum23, sum2, sum3);
            return (sum0 + sum1) + (sum2 + sum3);
          };
          float total = 0.0f;
          for (int c0 = 0; c0 < cols; c0 += cw::kHalf, ++used) {
            const int buf = used & 1;
            if (!(ok = wd.warp_wait(s_full(g, buf), static_cast<uint32_t>(used >> 1) & 1u))) break;
            tc_fence_after_sync();
            const uint32_t t_buf = t_s + cw::kHalf * static_cast<uint32_t>(buf);
            // Rows that weigh nothing (the padding, queries that are none) are zeros with
            // a factor of 0, which is enough but for a key with an infinity or a NaN:
            // where a sum is none, it is taken again without them. (Leaving them out at
            // once, by a bit a column wherever there are some, took 256 rows over 8
            // sequences of up to 8192 slots from 42.8 us to 43.9, one row of 4 heads over
            // 40 of up to 1000 from 16.1 to 16.5; this way takes 44.4 and 16.1.)
            float sum = 0.0f;
            bool again = masked;
            if (!masked) {
              sum = half(t_buf, c0, min(cols, c0 + cw::kHalf), std::false_type{});
              again = __any_sync(0xffffffffu, sum != sum);
            }
            if (again) sum = half(t_buf, c0, min(cols, c0 + cw::kHalf), std::true_type{});
            total += sum;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_empty(g, buf));
          }
          if (!ok) break;
          if (live) args.weight_out[weight_row + key] = acc + total;
        }
        __syncwarp();
        if (lane == 0)
          for (int half = 0; half < 2; ++half)
            if (halves.has(half)) mbar_arrive(q_free(half));
        __syncwarp();
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == cw::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem_base, C::kTmemCols);
  }
}

}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

namespace {

template <class C>
cudaError_t launch_cfg(const gemm_tn_dev::WeighArgs& args, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(gemm_tn_dev::cache_weigh_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmemBytes));
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(args.chunks), 1, 1);
  cfg.blockDim = dim3(C::kNumThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent_launch_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gemm_tn_dev::cache_weigh_kernel<C>, args);
}

}  // namespace

cudaError_t launch_cache_weigh(int head_dim, bool bf16, const gemm_tn_dev::WeighArgs& args, cudaStream_t stream) {
  using namespace gemm_tn_dev::cw;
  if (head_dim == 64)
    return bf16 ? launch_cfg<Cfg<64, true>>(args, stream) : launch_cfg<Cfg<64, false>>(args, stream);
  if (head_dim == 128)
    return bf16 ? launch_cfg<Cfg<128, true>>(args, stream) : launch_cfg<Cfg<128, false>>(args, stream);
  return cudaErrorInvalidValue;
}

}  // namespace gemm_tn_impl

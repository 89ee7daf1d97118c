// sm103_decode_attn.cu -- attention over a paged cache for few query rows: at
// most 32 per KV head (one token of a group of 8, a small tree), the decode
// step of tree_attn_fwd (include/kv_cache.h; the schedule, the parts of cut
// items and their join are sm103_tree_attn.cu's).
//
// With rows on the tensor memory's lanes, as in sm103_tree_attn.cu, a tile of
// 128 keys costs its one or two busy warps 128 exponentials however few rows
// there are, all on one of the SM's four sub-partitions: 0.9 us a tile, with
// 64 KB a tile due from memory every 1.5 us. Here both products are transposed:
//   S^T = K Q^T   (M = 128 keys, N = 16 or 32 rows, K = dim)
//   O^T += V^T P^T  (M = dim, N = rows, K = 128 keys; V's tile as it lies is an
//                    MN-major A operand, P is the K-major B operand in shared memory)
// A thread has one key: it computes one exponential per row, 16 or 32 a tile,
// four warps a tile on four sub-partitions, and the tensor cores' work falls
// with N as well. What the row-wise form gets for free has to cross threads:
// a row's maximum (taken from the first tile, and again only when a probability
// passes 2^8) and, once per segment, its sum. Every thread of a unit holds the
// same row references; the four warps of a unit agree through an mbarrier once
// a tile whether a reference has to move. The epilogue has dim on the lanes, so
// rows go out in contiguous pieces.
//
// Bound by HBM once a CTA has some ten tiles: one token of 32 heads over 8 KV
// heads of dim 128 for 64 sequences of 900 to 8192 slots reads 1.2 GB in 190 us
// (6.3 TB/s, 0.93 of the measured copy bandwidth; this change of layout alone
// took 223 us to 202). A few short sequences are bound by latency: the start, one
// round trip to memory for a table entry, another for its page, the tiles one
// after another (0.9 us each) and the way out. There the CTAs of a cluster share
// an item's tiles and join their results through shared memory: one sequence of
// 517 slots, 8 heads of dim 64, takes 8.1 us (on one CTA per head 3.7 more).
//
// Roles: warp 0 TMA producer (lane l copies the tile's l-th page), warp 1 MMA
// issuer, warps 2-5 and 6-9 two units that take every other key tile and are
// joined at the end of a segment.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kv_cache_internal.h"
#include "sm103_tree_attn.cuh"

namespace gemm_tn_dev {

namespace da {

using cache::kTileKeys;
constexpr int kProducerWarp = 0;
constexpr int kMmaWarp = 1;
constexpr int kFirstSoftmaxWarp = 2;
constexpr int kMaxRows = 32;

template <int kDim_, bool kBf16_, int kRows_>
struct Cfg {
  static constexpr int kDim = kDim_;
  static constexpr bool kBf16 = kBf16_;
  static constexpr int kRows = kRows_;                    // N of both products
  static constexpr int kNumThreads = 64 + 256;
  static constexpr int kDimBoxes = kDim / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;      // 128 keys x 128 bytes
  static constexpr uint32_t kTileBytes = kDimBoxes * kBoxBytes;
  static constexpr uint32_t kQBoxBytes = kRows * 128u;    // rows x 64 elements of dim
  static constexpr uint32_t kQBytes = kDimBoxes * kQBoxBytes;
  static constexpr uint32_t kPBoxBytes = kRows * 128u;    // rows x 64 keys
  static constexpr uint32_t kPBytes = 2 * kPBoxBytes;
  static constexpr int kStages = kDim == 64 ? 6 : 3;      // of K and of V
  static constexpr uint32_t kOffK = 0;
  static constexpr uint32_t kOffV = kOffK + kStages * kTileBytes;
  static constexpr uint32_t kOffP = kOffV + kStages * kTileBytes;   // one per unit
  static constexpr uint32_t kOffQ = kOffP + 2 * kPBytes;            // two slots
  static constexpr uint32_t kOffWarps = kOffQ + 2 * kQBytes;          // [2 units][4 warps][32 rows]: a tile's maxima, a segment's sums
  static constexpr uint32_t kOffRef = kOffWarps + 2u * 4u * 32u * 4u; // [2 units][32 rows]
  static constexpr uint32_t kOffShare = kOffRef + 2u * 32u * 4u;      // [32 rows] (max, sum) of this CTA's share of an item
  static constexpr uint32_t kOffBar = kOffShare + 32u * 8u;
  // q_full[2], q_empty[2], k_full[S], k_empty[S], v_full[S], v_empty[S],
  // s_full[2], p_full[2], o_done[2], agree[2], xch_full, xch_empty, drain
  static constexpr int kNumBars = 4 + 4 * kStages + 8 + 3;
  static constexpr uint32_t kOffVote = kOffBar + 8u * kNumBars;     // [2 units][3]
  static constexpr uint32_t kOffTmemSlot = kOffVote + 24u;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4u;
  static constexpr uint32_t kOffStart = kOffAbort + 4u;   // the chunk's first Walk, the second; then the segments' in turn
  static constexpr uint32_t kOffWalkSums = kOffStart + 72u;
  static constexpr uint32_t kSmemBytes = kOffWalkSums + 128u + 1024u;   // + slack to align the base to 1024
  static constexpr uint32_t kTmemCols = 4 * kRows;        // S_0, S_1, O_0, O_1
  static constexpr uint32_t kIdescS = mma_idesc_f16(kBf16, kTileKeys, kRows, false);
  // A is V^T, MN-major (bit 15). Dim 64 runs with M = 128: the lanes from 64 on
  // multiply whatever lies 8 KB further on and are not looked at.
  static constexpr uint32_t kIdescO = mma_idesc_f16(kBf16, 128, kRows, false) | (1u << 15);
  static constexpr uint32_t kVBlockBytes = kDim == 128 ? kBoxBytes : 8192u;
  static_assert(kRows == 16 || kRows == 32, "rows");
  static_assert(kSmemBytes <= 227u * 1024u, "shared memory budget");
  static_assert(kOffBar % 8u == 0, "64-bit shared words");
};

// Reduces kRows values over the 32 lanes: lane r (and r + 16 with 16 rows) gets
// row r's. Halves the rows at every exchange: 31 shuffles for 32 rows.
template <int kRows, class Op>
__device__ __forceinline__ float warp_rows(float (&x)[kRows], uint32_t lane, Op op) {
#pragma unroll
  for (int half = kRows / 2; half >= 1; half /= 2) {
    const bool upper = (lane & static_cast<uint32_t>(half)) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? x[i + half] : x[i], give = upper ? x[i] : x[i + half];
      x[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, half));
    }
  }
  if constexpr (kRows == 16) x[0] = op(x[0], __shfl_xor_sync(0xffffffffu, x[0], 16));
  return x[0];
}

template <int kRows>
__device__ __forceinline__ void tmem_load_rows(uint32_t taddr, float (&v)[kRows]) {
  if constexpr (kRows == 32) {
    uint32_t raw[32];
    tmem_load_32x32(taddr, raw);
    tmem_load_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(raw[e]);
  } else {
    uint32_t raw[16];
    tmem_load_32x16(taddr, raw);
    tmem_load_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(raw[e]);
  }
}

template <int kRows>
__device__ __forceinline__ void tmem_store_rows(uint32_t taddr, const float (&v)[kRows]) {
  uint32_t raw[kRows];
#pragma unroll
  for (int e = 0; e < kRows; ++e) raw[e] = __float_as_uint(v[e]);
  if constexpr (kRows == 32) tmem_store_32x32(taddr, raw);
  else tmem_store_32x16(taddr, raw);
}

// Joins the shares of an item that the CTAs of a cluster have in shared memory,
// in the order of their tiles: each CTA joins and writes a part of the rows'
// 4-column pieces.
template <class C>
__device__ __forceinline__ void join_shares(const TreeArgs& args, const ta::Walk& w, uint32_t base) {
  constexpr int kPieces = C::kDim / 4, kMost = 8;   // CTAs of a cluster
  const int rows = w.tl * args.group;
  const uint32_t rank = cluster_ctarank();
#pragma unroll 1
  for (int x = static_cast<int>(rank) * C::kNumThreads + static_cast<int>(threadIdx.x); x < rows * kPieces;
       x += args.spread * C::kNumThreads) {
    const int r = x / kPieces, piece = x - r * kPieces;
    float2 ml[kMost];
    float4 y[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      ml[i] = make_float2(0.0f, 0.0f);
      if (i >= args.spread) continue;
      const uint32_t at = map_to_cta(base, static_cast<uint32_t>(i));
      ml[i] = ld_cluster_f2(at + C::kOffShare + 8u * r);
      y[i] = ld_cluster_f4(at + C::kOffK + 16u * x);
    }
    // a sum of zero has no maximum and nothing in its row
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMost; ++i) m = ml[i].y != 0.0f ? fmaxf(m, ml[i].x) : m;
    float sum = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (ml[i].y == 0.0f) continue;
      const float f = ex2_approx(ml[i].x - m);
      sum += ml[i].y * f;
      o0 += y[i].x * f;
      o1 += y[i].y * f;
      o2 += y[i].z * f;
      o3 += y[i].w * f;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int token = r / args.group;
    const int64_t out_row = (static_cast<int64_t>(w.b) * args.tokens + token) * args.heads + w.h * args.group + (r - token * args.group);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(args.o) + out_row * C::kDim + 4 * piece) =
        make_uint2(cache::pack2<C::kBf16>(o0 * inv, o1 * inv), cache::pack2<C::kBf16>(o2 * inv, o3 * inv));
    if (piece == 0 && args.lse != nullptr) args.lse[out_row] = sum == 0.0f ? -INFINITY : (m * ta::kLn2 + logf(sum));
  }
}

}  // namespace da

template <class C>
__global__ void __launch_bounds__(C::kNumThreads, 1) decode_attn_kernel(const __grid_constant__ TreeArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t base = smem_addr(smem);
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();

  auto q_slot = [&](int s) { return base + C::kOffQ + s * C::kQBytes; };
  auto k_tile = [&](int s) { return base + C::kOffK + s * C::kTileBytes; };
  auto v_tile = [&](int s) { return base + C::kOffV + s * C::kTileBytes; };
  auto p_tile = [&](int u) { return base + C::kOffP + u * C::kPBytes; };
  auto bar = [&](int i) { return base + C::kOffBar + 8u * i; };
  constexpr int kKBar = 4, kVBar = kKBar + 2 * C::kStages, kUBar = kVBar + 2 * C::kStages;
  auto q_full = [&](int s) { return bar(s); };
  auto q_empty = [&](int s) { return bar(2 + s); };
  auto k_full = [&](int s) { return bar(kKBar + s); };
  auto k_empty = [&](int s) { return bar(kKBar + C::kStages + s); };
  auto v_full = [&](int s) { return bar(kVBar + s); };
  auto v_empty = [&](int s) { return bar(kVBar + C::kStages + s); };
  auto s_full = [&](int u) { return bar(kUBar + u); };
  auto p_full = [&](int u) { return bar(kUBar + 2 + u); };
  auto o_done = [&](int u) { return bar(kUBar + 4 + u); };
  auto agree = [&](int u) { return bar(kUBar + 6 + u); };
  const uint32_t xch_full = bar(kUBar + 8), xch_empty = bar(kUBar + 9), drain_bar = bar(kUBar + 10);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
  ta::Walk* start_walk = reinterpret_cast<ta::Walk*>(smem + C::kOffStart);
  int* sums = reinterpret_cast<int*>(smem + C::kOffWalkSums);
  float* warp_maxima = reinterpret_cast<float*>(smem + C::kOffWarps);
  float* warp_sums = warp_maxima;
  float* unit_refs = reinterpret_cast<float*>(smem + C::kOffRef);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);   // one arrival per softmax warp of the unit
      mbar_init(o_done(s), 1);
      mbar_init(agree(s), 4);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    mbar_init(xch_full, 8);
    mbar_init(xch_empty, 4);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    start_walk->left = 0;
    start_walk->b = -1;
    fence_barrier_init();
  }
  if (warp == da::kProducerWarp && lane == 0) {
    tma_prefetch_descriptor(&args.tmap_q);
    tma_prefetch_descriptor(&args.tmap_k);
    tma_prefetch_descriptor(&args.tmap_v);
  }
  if (warp == da::kMmaWarp) {
    tmem_alloc<1>(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish<1>();
  }
  // rows of Q past the item's stay zero
  for (uint32_t x = threadIdx.x; x < 2 * C::kQBytes / 16; x += C::kNumThreads)
    st_shared_v4(base + C::kOffQ + 16u * x, 0u, 0u, 0u, 0u);
  if (threadIdx.x < 6) reinterpret_cast<uint32_t*>(smem + C::kOffVote)[threadIdx.x] = 0u;
  if (threadIdx.x < 32) reinterpret_cast<float2*>(smem + C::kOffShare)[threadIdx.x] = make_float2(0.0f, 0.0f);
  fence_proxy_async_shared();
  // The set-up above may overlap the end of the previous kernel in the
  // stream; global memory is touched only once that kernel has completed.
  griddep_wait();
  griddep_launch_dependents();
  ta::find_walk(args, start_walk, sums);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const cache::Watch<false> wd{args.status, args.timeout_ns, abort_flag};
  const bool has_new = args.has_new != 0;
  ta::Walk w = *start_walk;
  if (threadIdx.x == 0) ta::note_no_cut(args, w);

  if (warp == da::kProducerWarp) {
    // -------------------------------------------------------------- TMA producer
    cache::Issued issued_q, issued_k, issued_v;
    const int box_rows = min(args.page_size, da::kTileKeys);
    const int tile_pages = da::kTileKeys / box_rows;   // pages (or parts of one) per tile
    const uint32_t q_bytes = static_cast<uint32_t>(args.tokens * args.group) * 128u * C::kDimBoxes;
    int s = 0;             // ring stage and phase of the next tile
    uint32_t ph = 0;
    int it = 0, seg = 0;
    bool ok = true;
    for (; ok && w.more(); w.next(args), ++seg) {
      const int32_t* table = args.page_table + static_cast<int64_t>(w.b) * args.table_stride;
      auto page_of = [&](int j) {
        return ta::page_of(args, table, ta::tile_of(w.len, w.tl, has_new, j), box_rows, static_cast<int>(lane));
      };
      int page = page_of(w.j0);
      const int slot = seg & 1;
      const uint32_t q_ph = static_cast<uint32_t>(seg >> 1) & 1u;
      if (!(ok = wd.warp_wait(q_empty(slot), q_ph ^ 1u))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full(slot), q_bytes);
        for (int c = 0; c < C::kDimBoxes; ++c)
          tma_load_4d(&args.tmap_q, q_slot(slot) + c * C::kQBoxBytes, q_full(slot), 64 * c, w.h * args.group, 0, w.b);
      }
      issued_q.note(slot, q_ph);
      for (int j = w.j0; j < w.j0 + w.count; ++j, ++it) {
        const ta::Tile t = ta::tile_of(w.len, w.tl, has_new, j);
        const int boxes = t.fresh ? (t.valid > 0 ? 1 : 0) : (t.valid + box_rows - 1) / box_rows;
        const uint32_t bytes = static_cast<uint32_t>(boxes * (t.fresh ? da::kTileKeys : box_rows)) * 128u * C::kDimBoxes;
        const int slot0 = t.fresh ? t.index * da::kTileKeys
                                  : (tile_pages == 1 ? (t.index * da::kTileKeys) % args.page_size : 0);
        const bool mine = static_cast<int>(lane) < boxes;
        if (!(ok = wd.warp_wait(k_empty(s), ph ^ 1u))) break;
        if (lane == 0) mbar_arrive_expect_tx(k_full(s), bytes);
        __syncwarp();
        if (mine && !(blockIdx.x == 0 && it == args.drop_load_block)) {
          for (int c = 0; c < C::kDimBoxes; ++c)
            tma_load_4d(t.fresh ? &args.tmap_k_new : &args.tmap_k, k_tile(s) + c * C::kBoxBytes + lane * box_rows * 128u,
                        k_full(s), 64 * c, w.h, slot0, t.fresh ? w.b : page);
        }
        issued_k.note(s, ph);
        if (!(ok = wd.warp_wait(v_empty(s), ph ^ 1u))) break;
        if (lane == 0) mbar_arrive_expect_tx(v_full(s), bytes);
        __syncwarp();
        if (mine) {
          for (int c = 0; c < C::kDimBoxes; ++c)
            tma_load_4d(t.fresh ? &args.tmap_v_new : &args.tmap_v, v_tile(s) + c * C::kBoxBytes + lane * box_rows * 128u,
                        v_full(s), 64 * c, w.h, slot0, t.fresh ? w.b : page);
        }
        issued_v.note(s, ph);
        if (j + 1 < w.j0 + w.count) page = page_of(j + 1);
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // Loads may still be landing if another role gave up: wait (bounded) for
    // every phase issued before the CTA may exit.
    issued_q.drain(wd, 2, q_full);
    issued_k.drain(wd, C::kStages, k_full);
    issued_v.drain(wd, C::kStages, v_full);
  } else if (warp == da::kMmaWarp) {
    {
      // ------------------------------------------------------------ MMA issuer
      // (the whole warp runs this, one lane issues)
      const uint32_t leader = elect_one();
      int it0 = 0;                    // ring number of the segment's first tile
      int seg = 0;
      int done[2] = {0, 0};           // tiles of each unit whose P has been asked for
      bool ok = true;
      for (; ok && w.more(); it0 += w.count, w.next(args), ++seg) {
        const int slot = seg & 1;
        auto issue_s = [&](int u, int i) {   // i: tile of the segment
          const int x = it0 + i, s = x % C::kStages;
          if (!wd.warp_wait(k_full(s), static_cast<uint32_t>(x / C::kStages) & 1u)) return false;
          tc_fence_after_sync();
#pragma unroll
          for (int c = 0; c < C::kDimBoxes; ++c) {
            const uint64_t a_desc = sw128_kmajor_desc(k_tile(s) + c * C::kBoxBytes);
            const uint64_t b_desc = sw128_kmajor_desc(q_slot(slot) + c * C::kQBoxBytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 16 elements of dim = 32 bytes = 2 descriptor units
              mma_f16_warp(leader, tmem_base + static_cast<uint32_t>(C::kRows * u), a_desc + 2u * kk, b_desc + 2u * kk, C::kIdescS,
                         (c | kk) != 0 ? 1u : 0u);
          }
          mma_commit_warp(leader, s_full(u));
          mma_commit_warp(leader, k_empty(s));
          if (i == w.count - 1) mma_commit_warp(leader, q_empty(slot));   // Q has been read for the last time
          return true;
        };
        if (!(ok = wd.warp_wait(q_full(slot), static_cast<uint32_t>(seg >> 1) & 1u))) break;
        ok = issue_s(0, 0) && (w.count < 2 || issue_s(1, 1));
        for (int i = 0; ok && i < w.count; ++i) {
          const int x = it0 + i, s = x % C::kStages, u = i & 1;
          if (!(ok = wd.warp_wait(v_full(s), static_cast<uint32_t>(x / C::kStages) & 1u))) break;
          if (!(ok = wd.warp_wait(p_full(u), static_cast<uint32_t>(done[u]) & 1u))) break;
          ++done[u];
          tc_fence_after_sync();
          const int steps = (ta::tile_of(w.len, w.tl, has_new, w.j0 + i).valid + 15) / 16;
          const uint64_t a_desc = sw128_mnmajor_desc(v_tile(s), C::kVBlockBytes);
          const uint64_t b_desc = sw128_kmajor_desc(p_tile(u));
          const uint32_t t_o = tmem_base + static_cast<uint32_t>(C::kRows * (2 + u));
          auto pv = [&](int kk) {   // 16 keys: 16 rows of 128 bytes of V; 32 bytes of P's rows, 64 keys a box
            mma_f16_warp(leader, t_o, a_desc + ((static_cast<uint32_t>(kk) * 2048u) >> 4),
                       b_desc + ((static_cast<uint32_t>(kk >> 2) * C::kPBoxBytes) >> 4) + 2u * static_cast<uint32_t>(kk & 3),
                       C::kIdescO, i < 2 && kk == 0 ? 0u : 1u);
          };
          if (steps == 8) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) pv(kk);
          } else {
            for (int kk = 0; kk < steps; ++kk) pv(kk);
          }
          mma_commit_warp(leader, v_empty(s));
          if (i + 2 < w.count) ok = issue_s(u, i + 2);
          else mma_commit_warp(leader, o_done(u));
        }
      }
      // every MMA issued here must finish before TMEM is freed
      mma_commit_warp(leader, drain_bar);
      wd.drain(drain_bar, 0);
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int u = (static_cast<int>(warp) - da::kFirstSoftmaxWarp) >> 2;   // unit
    const uint32_t quarter = warp & 3u;                                    // TMEM lanes 32*quarter ..
    const int key = static_cast<int>(quarter * 32u + lane);                // of the tile; column of O in the end
    const uint32_t lane_off = (quarter * 32u) << 16;
    const uint32_t t_s = tmem_base + lane_off + static_cast<uint32_t>(C::kRows * u);
    const uint32_t t_o = tmem_base + lane_off + static_cast<uint32_t>(C::kRows * (2 + u));
    const float c_log2 = args.scale_log2;
    volatile uint32_t* votes = reinterpret_cast<volatile uint32_t*>(smem + C::kOffVote) + 3 * u;
    float* my_maxima = warp_maxima + (u * 4 + static_cast<int>(quarter)) * 32;
    uint32_t tiles_done = 0;        // tiles of this unit so far
    uint32_t agreed = 0;            // phases of agree(u) so far
    uint32_t voted = 0;             // votes so far
    uint32_t ends[2] = {0, 0};      // o_done phases of the units so far
    uint32_t segs = 0;
    int it0 = 0;
    bool ok = true;
    // the unit's four warps meet (bounded)
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(agree(u));
      return wd.warp_wait(agree(u), agreed++ & 1u);
    };
    for (; ok && w.more(); it0 += w.count, ++segs, w = start_walk[segs & 1u]) {
      if (u == 0 && quarter == 0) {
        // the next segment's, worked out by one warp while the first scores are
        // awaited; the exchange at the end of the segment hands it to the others
        ta::Walk next = w;
        next.next(args);
        if (lane == 0) start_walk[(segs + 1u) & 1u] = next;
      }
      const int rows = w.tl * args.group;   // rows that exist, token-major
      const uint32_t row_bits = cache::low_bits(rows);
      uint32_t unset = row_bits;            // rows that have seen no key yet
      float neg_m[C::kRows], l[C::kRows];   // minus the row's reference, in units of scale * log2e; this key lane's sum
      // Rows that do not exist, whose queries may be anything: a reference of infinity
      // makes their probabilities 0 (or NaN), which call for no new references.
#pragma unroll
      for (int r = 0; r < C::kRows; ++r) {
        neg_m[r] = (row_bits >> r) & 1u ? 0.0f : -INFINITY;
        l[r] = 0.0f;
      }
      for (int i = u; i < w.count && ok; i += 2) {
        // S_u for this tile is complete, and with it O_u += P_u V of the tile before
        if (!(ok = wd.warp_wait(s_full(u), tiles_done & 1u))) break;
        ++tiles_done;
        tc_fence_after_sync();
        const ta::Tile t = ta::tile_of(w.len, w.tl, has_new, w.j0 + i);
        float s[C::kRows];
        da::tmem_load_rows<C::kRows>(t_s, s);
        uint32_t seen = key < t.valid ? 0xffffffffu : 0u;   // rows that see this thread's key
        if (t.fresh) {
          // new token x's rows are bits x * group .. of the word; x sees this key or does not
          const uint64_t* words = args.mask + static_cast<int64_t>(w.b) * args.tokens;   // at most 32 tokens: one word each
          uint32_t word = cache::low_bits(static_cast<int>(lane) + 1);   // lane x: the keys that token x sees
          if (args.mask != nullptr) word = static_cast<int>(lane) < w.tl ? static_cast<uint32_t>(__ldg(words + lane)) : 0u;
          const uint32_t token_rows = cache::low_bits(args.group);
          uint32_t rows_seen = 0;
          for (int x = 0; x < w.tl; ++x) {
            const uint32_t sees = __shfl_sync(0xffffffffu, word, x);
            if ((sees >> (key & 31)) & 1u) rows_seen |= token_rows << (x * args.group);
          }
          if (key < t.valid) seen = rows_seen;
        }
        const bool partial = t.fresh || t.valid < da::kTileKeys;
        auto hide = [&]() {   // scores that their rows do not see
#pragma unroll
          for (int r = 0; r < C::kRows; ++r)
            if (!((seen >> r) & 1u)) s[r] = -INFINITY;
        };
        if (partial) hide();
        bool over = unset != 0;
        if (!over) {
          // probabilities, in the scores' registers, against the references at
          // once; one past 2^8 calls for new references (a NaN does not: its
          // row is lost either way)
          float most = 0.0f;
#pragma unroll
          for (int r = 0; r < C::kRows; ++r) {
            s[r] = ex2_approx(fmaf(s[r], c_log2, neg_m[r]));
            most = fmaxf(most, s[r]);
          }
          const bool mine = most > 256.0f;
          // three words in turn: the next one is cleared before this meeting,
          // after the meeting in which its last vote was read
          const uint32_t word = voted % 3u;
          if (quarter == 0 && lane == 0) votes[(word + 1u) % 3u] = 0u;
          if (__any_sync(0xffffffffu, mine) && lane == 0) votes[word] = 1u;
          if (!(ok = meet())) break;
          over = votes[word] != 0u;
          ++voted;
          if (over) {   // the scores are still in tensor memory
            da::tmem_load_rows<C::kRows>(t_s, s);
            if (partial) hide();
          }
        }
        if (over) {
          // the tile's row maxima over the unit's 128 keys: over the warp, then
          // over the four warps; from there on lane r decides for row r
          float x[C::kRows];
#pragma unroll
          for (int r = 0; r < C::kRows; ++r) x[r] = s[r];
          const float warp_max = da::warp_rows<C::kRows>(x, lane, [](float p, float q) { return fmaxf(p, q); });
          if (lane < C::kRows) my_maxima[lane] = warp_max;
          if (!(ok = meet())) break;
          const uint32_t row = lane % C::kRows;
          const float* all = warp_maxima + u * 128 + row;
          const float mx = fmaxf(fmaxf(all[0], all[32]), fmaxf(all[64], all[96])) * c_log2;
          float neg = 0.0f, alpha = 1.0f;   // the row's reference so far, and O's and l's factor
#pragma unroll
          for (int r = 0; r < C::kRows; ++r)
            if (row == static_cast<uint32_t>(r)) neg = neg_m[r];
          const bool fresh_row = ((unset >> row) & 1u) != 0u && mx != -INFINITY;
          const bool move = ((row_bits & ~unset) >> row & 1u) != 0u && mx > 8.0f - neg;
          if (move) alpha = ex2_approx(-neg - mx);
          if (fresh_row || move) neg = -mx;
          unset &= ~(__ballot_sync(0xffffffffu, fresh_row) & cache::low_bits(C::kRows));
          const bool moved = __any_sync(0xffffffffu, move);   // the same in every warp of the unit
#pragma unroll
          for (int r = 0; r < C::kRows; ++r) {
            neg_m[r] = __shfl_sync(0xffffffffu, neg, r);
            s[r] = ex2_approx(fmaf(s[r], c_log2, neg_m[r]));
          }
          if (moved) {
#pragma unroll
            for (int c = 0; c < C::kRows; c += 16) {
              float o[16];
              da::tmem_load_rows<16>(t_o + static_cast<uint32_t>(c), o);
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const float f = __shfl_sync(0xffffffffu, alpha, c + r);
                o[r] *= f;
                l[c + r] *= f;
              }
              da::tmem_store_rows<16>(t_o + static_cast<uint32_t>(c), o);
            }
            tmem_store_wait();
          }
          // the maxima are not written again before every warp has read them
          if (!(ok = meet())) break;
        }
        // P: row r's 64-key boxes of 128 bytes, 16-byte pieces swizzled by the row
        const uint32_t p_at = p_tile(u) + static_cast<uint32_t>(key >> 6) * C::kPBoxBytes + 2u * static_cast<uint32_t>(key & 7);
        const uint32_t piece = static_cast<uint32_t>(key & 63) >> 3;
#pragma unroll
        for (int r = 0; r < C::kRows; ++r) {
          l[r] += s[r];
          st_shared_u16(p_at + 128u * r + 16u * (piece ^ (r & 7u)), static_cast<uint16_t>(cache::pack2<C::kBf16>(s[r], 0.0f)));
        }
        if (t.valid % 16 != 0) {
          // zero the rows of V behind the last key, up to the end of its 16-key step
          const int x = it0 + i, st = x % C::kStages;
          if (!(ok = wd.warp_wait(v_full(st), static_cast<uint32_t>(x / C::kStages) & 1u))) break;
          const int row_end = (t.valid + 15) / 16 * 16;
          for (int y = t.valid * 8 + key; y < row_end * 8; y += 128)
#pragma unroll
            for (int c = 0; c < C::kDimBoxes; ++c) st_shared_v4(v_tile(st) + c * C::kBoxBytes + 16u * y, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(u));
      }
      if (!ok) break;
      // ---------------------------------------------------------- end of a segment
      // references and sums to shared memory; unit 0 joins the two units' rows
      {
        const float sum = da::warp_rows<C::kRows>(l, lane, [](float p, float q) { return p + q; });
        if (lane < C::kRows) warp_sums[(u * 4 + static_cast<int>(quarter)) * 32 + static_cast<int>(lane)] = sum;
        float neg = 0.0f;   // lane r: row r's (selected, not stored under a branch a row: those took 1 us)
#pragma unroll
        for (int r = 0; r < C::kRows; ++r) neg = lane == static_cast<uint32_t>(r) ? neg_m[r] : neg;
        if (quarter == 0 && lane < C::kRows) unit_refs[u * 32 + static_cast<int>(lane)] = -neg;
        const bool both = w.count > 1;
        if (u < w.count) {
          if (!(ok = wd.warp_wait(o_done(u), ends[u] & 1u))) break;
          ++ends[u];
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(xch_full);
        if (u == 0) {
          if (both) {
            if (!(ok = wd.warp_wait(o_done(1), ends[1] & 1u))) break;
            ++ends[1];
          }
          if (!(ok = wd.warp_wait(xch_full, segs & 1u))) break;
          tc_fence_after_sync();
          // lane r works out row r's factors
          float f0 = 0.0f, f1 = 0.0f;
          const bool shared = args.spread > 1;   // the cluster's CTAs join their shares, once all are there
          const bool whole = w.j0 == 0 && w.count == w.tiles && !shared;
          const int64_t slot = static_cast<int>(blockIdx.x) * 2 + (w.j0 == 0 ? 1 : 0);
          float2* part_ml = shared ? reinterpret_cast<float2*>(smem + C::kOffShare) : args.part_ml + slot * args.part_rows;
          if (static_cast<int>(lane) < rows) {
            const float* x = warp_sums + lane;
            const float l0 = (x[0] + x[32]) + (x[64] + x[96]);
            const float l1 = both ? (x[128] + x[160]) + (x[192] + x[224]) : 0.0f;
            const float m0 = unit_refs[lane], m1 = unit_refs[32 + lane];
            // a part with an empty sum has no reference; NaN sums stay NaN
            const float m = l0 == 0.0f ? m1 : (l1 == 0.0f ? m0 : fmaxf(m0, m1));
            f0 = l0 == 0.0f ? 0.0f : ex2_approx(m0 - m);
            f1 = l1 == 0.0f ? 0.0f : ex2_approx(m1 - m);
            const float sum_all = (l0 == 0.0f ? 0.0f : l0 * f0) + (l1 == 0.0f ? 0.0f : l1 * f1);
            if (whole) {
              const float inv = sum_all == 0.0f ? 0.0f : 1.0f / sum_all;
              f0 *= inv;
              f1 *= inv;
              if (quarter == 0 && args.lse != nullptr) {
                const int token = static_cast<int>(lane) / args.group;
                args.lse[(static_cast<int64_t>(w.b) * args.tokens + token) * args.heads + w.h * args.group +
                         (static_cast<int>(lane) - token * args.group)] =
                    sum_all == 0.0f ? -INFINITY : (m * ta::kLn2 + logf(sum_all));
              }
            } else if (quarter == 0) {
              part_ml[lane] = make_float2(sum_all == 0.0f ? 0.0f : m, sum_all);
            }
          }
          const bool column = key < C::kDim;   // this lane holds a column of O
          uint16_t* out = static_cast<uint16_t*>(args.o) +
                          (static_cast<int64_t>(w.b) * args.tokens * args.heads + w.h * args.group) * C::kDim + key;
          // a share lies over the K ring, which has been read for the last time: row after row
          float* part = shared ? reinterpret_cast<float*>(smem + C::kOffK) + key
                               : args.part_o + (slot * (C::kDim / 4) + key / 4) * args.part_rows * 4 + key % 4;
          const int part_step = shared ? C::kDim : 4;
          const int next_token = (args.heads - args.group) * C::kDim;   // from a token's last row to the next one's first
          int head = 0;
#pragma unroll 1   // once per segment: a loop's instructions are fetched once
          for (int r0 = 0; r0 < rows; r0 += 8) {
            uint32_t o0[8], o1[8];
            tmem_load_32x8(t_o + static_cast<uint32_t>(r0), o0);
            if (both) tmem_load_32x8(t_o + static_cast<uint32_t>(C::kRows + r0), o1);
            tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = r0 + i;
              const float a0 = __shfl_sync(0xffffffffu, f0, r), a1 = __shfl_sync(0xffffffffu, f1, r);
              float v = a0 == 0.0f ? 0.0f : __uint_as_float(o0[i]) * a0;
              if (both && a1 != 0.0f) v += __uint_as_float(o1[i]) * a1;
              if (column && r < rows) {
                if (whole) *out = static_cast<uint16_t>(cache::pack2<C::kBf16>(v, 0.0f));
                else part[part_step * r] = v;
              }
              out += C::kDim;
              if (++head == args.group) {
                head = 0;
                out += next_token;
              }
            }
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(xch_empty);
        }
        // shared sums and the O buffers are free again
        if (!(ok = wd.warp_wait(xch_empty, segs & 1u))) break;
        tc_fence_after_sync();
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == da::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem_base, C::kTmemCols);
  }
  if (args.spread > 1) {
    // every CTA of the cluster comes here, also one that has given up (its
    // waits are bounded) or had no tiles
    cluster_sync_all();
    if (start_walk->b >= 0) da::join_shares<C>(args, *start_walk, base);
    cluster_sync_all();   // no CTA leaves while its shared memory is read
  }
}

}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

namespace {

template <class C>
cudaError_t launch_cfg(const gemm_tn_dev::TreeArgs& args, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(gemm_tn_dev::decode_attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmemBytes));
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(args.chunks * args.spread), 1, 1);
  cfg.blockDim = dim3(C::kNumThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = cache_launch_attributes(attr, args.spread);
  return cudaLaunchKernelEx(&cfg, gemm_tn_dev::decode_attn_kernel<C>, args);
}

template <int kRows>
cudaError_t launch_rows(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream) {
  using namespace gemm_tn_dev::da;
  if (head_dim == 64)
    return bf16 ? launch_cfg<Cfg<64, true, kRows>>(args, stream) : launch_cfg<Cfg<64, false, kRows>>(args, stream);
  if (head_dim == 128)
    return bf16 ? launch_cfg<Cfg<128, true, kRows>>(args, stream) : launch_cfg<Cfg<128, false, kRows>>(args, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

int decode_attn_rows() { return gemm_tn_dev::da::kMaxRows; }

int decode_attn_part_rows(int rows) { return rows <= 16 ? 16 : 32; }

cudaError_t launch_decode_attn(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream) {
  return args.part_rows == 16 ? launch_rows<16>(head_dim, bf16, args, stream) : launch_rows<32>(head_dim, bf16, args, stream);
}

}  // namespace gemm_tn_impl

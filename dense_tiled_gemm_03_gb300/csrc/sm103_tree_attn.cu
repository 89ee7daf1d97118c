// sm103_tree_attn.cu -- attention of new (drafted) tokens over a paged
// key/value cache and over one another (include/kv_cache.h: tree_attn_fwd).
//
//   s(i, k) = scale * q_i . k      k: the sequence's cached keys, then the new
//   o_i     = sum_k softmax(s)_k v_k    tokens that i sees (bit mask or chain)
//
// The query rows of one KV head -- the new tokens times the query heads that
// share it, token-major -- fill 128-row tiles, so one pass over the cache
// serves the whole tree and the whole group: a tile's worth of keys is read
// once for up to 128 rows (256 in pair mode). Per 128 cached keys of dim 128
// that is 64 KB from memory against 8.4 MFLOP on the tensor cores, so up to
// one row tile the kernel is bound by HBM, and past two by the tensor cores.
// GB300, in a replayed graph, second kernel included: trees of 26 tokens, 32
// heads over 8, 8 sequences of 1000 to 4096 slots 33.5 us (2.9 TB/s: few tiles
// a CTA, the start and the join are half of it); trees of 63 tokens, 16 heads
// over 2, 4 sequences of 20011 to 32768 slots 61 us (825 TFLOP/s); 1024
// tokens, 32 heads over 8, after 2 contexts of about 8000 slots 221 us
// (1320 TFLOP/s; 225 to 234 in calls in a row, at the board's power limit).
//
// Work: an item is (sequence, KV head, row unit) and walks its key tiles, the
// cached ones and then the new tokens'. All items' key tiles are laid end to
// end (a change of items apart) and cut into equal contiguous chunks, one per CTA, from the lengths as
// they stand on the device: ragged batches balance to one tile, one long
// sequence spreads over every SM, and a captured launch stays right when the
// lengths change. An item that lies in one chunk is written by its CTA; one
// that is cut leaves each part's unnormalised rows, maxima and sums in a
// workspace and the second kernel joins them in order (repeatable to the bit).
// Where no item can be long, a chunk takes the items that begin in it whole, or a
// cluster's CTAs share one and join its parts through shared memory, and there is
// neither workspace nor second kernel.
//
// One CTA per SM:
//   warp 0      TMA producer. Lane l copies the tile's l-th page (pages of 8 to
//               64 rows; longer pages are copied 128 rows at a time), so page
//               table look-ups and copies of a tile go out together.
//   warp 1      MMA issuer (one thread): S_u = Q_u K_j^T, O_u += P_u V_j, with
//               P_u in tensor memory over the scores it came from.
//   warps 2-9   softmax, four warps per unit u, one thread per row.
// The two units keep the tensor cores busy in turn. With at most 128 rows per
// KV head (parity mode) both units hold the same rows and take every other key
// tile, and their results are joined in tensor memory at the end of a chunk;
// with more (pair mode) each has its own 128 rows and both read every tile.
//
// Rows behind the end of a sequence in its last page (or between its new
// tokens' count and the array's end) may hold anything, NaN included: their
// scores are replaced, not added to, the product P V stops at the 16-key step
// that holds the last key, and the rows of V behind that key are zeroed in
// shared memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kv_cache_internal.h"
#include "sm103_tree_attn.cuh"

namespace gemm_tn_dev {

namespace ta {

constexpr int kProducerWarp = 0;
constexpr int kMmaWarp = 1;
constexpr int kFirstSoftmaxWarp = 2;
constexpr int kTileRows = 128;     // query rows per tile (TMEM lanes)

template <int kDim_, bool kBf16_>
struct Cfg {
  static constexpr int kDim = kDim_;
  static constexpr bool kBf16 = kBf16_;
  static constexpr int kNumThreads = 64 + 256;
  // registers per thread for one CTA per SM (16384 per sub-partition, three warps each)
  static constexpr int kMaxRegs = 168;
  static constexpr int kDimBoxes = kDim / 64;             // 64-element (128-byte) boxes across dim
  static constexpr uint32_t kBoxBytes = 128u * 128u;      // 128 rows x 128 bytes
  static constexpr uint32_t kTileBytes = kDimBoxes * kBoxBytes;
  static constexpr int kKStages = kDim == 64 ? 6 : 3;
  static constexpr int kVStages = kDim == 64 ? 5 : 2;
  static constexpr uint32_t kOffQ = 0;                    // two slots of one row tile
  static constexpr uint32_t kOffK = kOffQ + 2 * kTileBytes;
  static constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
  static constexpr uint32_t kOffXch = kOffV + kVStages * kTileBytes;   // (max, sum) per row of unit 1
  static constexpr uint32_t kOffBar = kOffXch + 8u * kTileRows;
  // q_full[2], q_empty[2], k_full[KS], k_empty[KS], v_full[VS], v_empty[VS],
  // s_full[2], p_full[2], o_done[2], xch_full, xch_empty, drain
  static constexpr int kNumBars = 4 + 2 * kKStages + 2 * kVStages + 6 + 3;
  static constexpr uint32_t kOffTmemSlot = kOffBar + 8u * kNumBars;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4u;
  static constexpr uint32_t kOffStart = kOffAbort + 4u;   // the chunk's first Walk
  static constexpr uint32_t kOffSums = kOffStart + 36u;   // 32 words of the search for it
  static constexpr uint32_t kOffWalks = kOffSums + 128u;   // each softmax warp's Walk, of this segment and the next
  static constexpr uint32_t kSmemBytes = kOffWalks + 16u * 36u + 1024u;   // + slack to align the base to 1024
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;      // S_u: 128 fp32 columns at 128 u (P_u over half of them)
  static constexpr uint32_t kColO = 256;    // O_u: dim fp32 columns at 256 + dim u
  static constexpr uint32_t kIdescS = mma_idesc_f16(kBf16, kTileRows, 0, false);   // N is set per tile
  static constexpr uint32_t kIdescO = mma_idesc_f16(kBf16, kTileRows, kDim, true);
  static_assert(kDim == 64 || kDim == 128, "head dim 64 or 128");
  static_assert(kSmemBytes <= 227u * 1024u, "shared memory budget");
  static_assert(kOffBar % 8u == 0, "64-bit shared words");
};

// Joins the shares of an item that the CTAs of a cluster have in shared memory,
// in the order of their tiles: each CTA joins and writes a part of the rows'
// 8-column pieces. A function of its own, to leave the kernel's registers alone.
template <class C>
static __device__ __noinline__ void join_shares(const TreeArgs& args, const Walk& w, uint32_t base) {
  constexpr int kPieces = C::kDim / 8, kMost = 8;   // CTAs of a cluster
  const uint32_t rank = cluster_ctarank();
#pragma unroll 1
  for (int x = static_cast<int>(rank) * C::kNumThreads + static_cast<int>(threadIdx.x); x < kTileRows * kPieces;
       x += args.spread * C::kNumThreads) {
    const int r = x % kTileRows, piece = x / kTileRows;
    const int r_token = r / args.group, token = w.ru * args.tile_tokens + r_token;
    if (r_token >= args.tile_tokens || token >= w.tl) continue;
    float2 ml[kMost];
    float m = -INFINITY;   // a sum of zero has no maximum and nothing in its row
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      ml[i] = make_float2(0.0f, 0.0f);
      if (i < args.spread) ml[i] = ld_cluster_f2(map_to_cta(base, static_cast<uint32_t>(i)) + C::kOffXch + 8u * r);
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) m = ml[i].y != 0.0f ? fmaxf(m, ml[i].x) : m;
    float sum = 0.0f, o[8] = {};
#pragma unroll
    for (int i0 = 0; i0 < kMost; i0 += 4) {
      float4 y[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i >= args.spread) continue;
        const uint32_t at = map_to_cta(base, static_cast<uint32_t>(i0 + i)) + C::kOffK + 16u * (2 * piece * kTileRows + r);
        y[i][0] = ld_cluster_f4(at);
        y[i][1] = ld_cluster_f4(at + 16u * kTileRows);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 part = ml[i0 + i];
        if (part.y == 0.0f) continue;
        const float f = ex2_approx(part.x - m);
        sum += part.y * f;
        const float v[8] = {y[i][0].x, y[i][0].y, y[i][0].z, y[i][0].w, y[i][1].x, y[i][1].y, y[i][1].z, y[i][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += v[e] * f;
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t out_row = (static_cast<int64_t>(w.b) * args.tokens + token) * args.heads + w.h * args.group + (r - r_token * args.group);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.o) + out_row * C::kDim + 8 * piece) =
        make_uint4(pack2<C::kBf16>(o[0] * inv, o[1] * inv), pack2<C::kBf16>(o[2] * inv, o[3] * inv),
                   pack2<C::kBf16>(o[4] * inv, o[5] * inv), pack2<C::kBf16>(o[6] * inv, o[7] * inv));
    if (piece == 0 && args.lse != nullptr) args.lse[out_row] = sum == 0.0f ? -INFINITY : (m * kLn2 + logf(sum));
  }
}

}  // namespace ta

template <class C>
__global__ void __launch_bounds__(C::kNumThreads) __maxnreg__(C::kMaxRegs)
    tree_attn_kernel(const __grid_constant__ TreeArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t base = smem_addr(smem);
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = lane_id();

  auto q_tile = [&](int s) { return base + C::kOffQ + s * C::kTileBytes; };
  auto k_tile = [&](int s) { return base + C::kOffK + s * C::kTileBytes; };
  auto v_tile = [&](int s) { return base + C::kOffV + s * C::kTileBytes; };
  auto bar = [&](int i) { return base + C::kOffBar + 8u * i; };
  constexpr int kKBar = 4, kVBar = kKBar + 2 * C::kKStages, kUBar = kVBar + 2 * C::kVStages;
  auto q_full = [&](int s) { return bar(s); };
  auto q_empty = [&](int s) { return bar(2 + s); };
  auto k_full = [&](int s) { return bar(kKBar + s); };
  auto k_empty = [&](int s) { return bar(kKBar + C::kKStages + s); };
  auto v_full = [&](int s) { return bar(kVBar + s); };
  auto v_empty = [&](int s) { return bar(kVBar + C::kVStages + s); };
  auto s_full = [&](int u) { return bar(kUBar + u); };
  auto p_full = [&](int u) { return bar(kUBar + 2 + u); };
  auto o_done = [&](int u) { return bar(kUBar + 4 + u); };
  const uint32_t xch_full = bar(kUBar + 6), xch_empty = bar(kUBar + 7), drain_bar = bar(kUBar + 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
  ta::Walk* start_walk = reinterpret_cast<ta::Walk*>(smem + C::kOffStart);
  int* sums = reinterpret_cast<int*>(smem + C::kOffSums);
  float2* xch = reinterpret_cast<float2*>(smem + C::kOffXch);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);   // one arrival per softmax warp of the unit
      mbar_init(o_done(s), 1);
    }
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    mbar_init(xch_full, 4);
    mbar_init(xch_empty, 4);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    start_walk->left = 0;
    start_walk->b = -1;
    fence_barrier_init();
  }
  if (warp == ta::kProducerWarp && lane == 0) {
    tma_prefetch_descriptor(&args.tmap_q);
    tma_prefetch_descriptor(&args.tmap_k);
    tma_prefetch_descriptor(&args.tmap_v);
  }
  if (warp == ta::kMmaWarp) {
    tmem_alloc<1>(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish<1>();
  }
  if (threadIdx.x < ta::kTileRows) xch[threadIdx.x] = make_float2(0.0f, 0.0f);   // a share without tiles stays so
  // The set-up above may overlap the end of the previous kernel in the
  // stream; global memory is touched only once that kernel has completed.
  griddep_wait();
  griddep_launch_dependents();
  ta::find_walk(args, start_walk, sums);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const cache::Watch<true> wd{args.status, args.timeout_ns, abort_flag};
  const bool parity_mode = args.units == 1;
  const bool has_new = args.has_new != 0;
  ta::Walk w = *start_walk;
  if (threadIdx.x == 0) ta::note_no_cut(args, w);

  if (warp == ta::kProducerWarp) {
    // -------------------------------------------------------------- TMA producer
    cache::Issued issued_q, issued_k, issued_v;
    const int box_rows = min(args.page_size, ta::kTileKeys);
    const int tile_pages = ta::kTileKeys / box_rows;   // pages (or parts of one) per tile
    const uint32_t q_bytes = static_cast<uint32_t>(args.tile_tokens * args.group) * 128u * C::kDimBoxes;
    int it = 0;     // tiles issued
    int seg = 0;    // segments begun
    bool ok = true;
    for (; ok && w.more(); w.next(args), ++seg) {
      const int32_t* table = args.page_table + static_cast<int64_t>(w.b) * args.table_stride;
      auto page_of = [&](int j) {
        return ta::page_of(args, table, ta::tile_of(w.len, w.tl, has_new, j), box_rows, static_cast<int>(lane));
      };
      int page = page_of(w.j0);
      for (int j = w.j0; j < w.j0 + w.count; ++j, ++it) {
        const ta::Tile t = ta::tile_of(w.len, w.tl, has_new, j);
        const int boxes = t.fresh ? (t.valid > 0 ? 1 : 0) : (t.valid + box_rows - 1) / box_rows;
        const int rows = t.fresh ? ta::kTileKeys : box_rows;
        const uint32_t bytes = static_cast<uint32_t>(boxes * rows) * 128u * C::kDimBoxes;
        const int slot0 = t.fresh ? t.index * ta::kTileKeys
                                  : (tile_pages == 1 ? (t.index * ta::kTileKeys) % args.page_size : 0);
        const int next_page = j + 1 < w.j0 + w.count ? page_of(j + 1) : 0;
        const bool mine = static_cast<int>(lane) < boxes;
        const int s = it % C::kKStages;
        const uint32_t ph = static_cast<uint32_t>(it / C::kKStages) & 1u;
        if (!(ok = wd.warp_wait(k_empty(s), ph ^ 1u))) break;
        if (lane == 0) mbar_arrive_expect_tx(k_full(s), bytes);
        __syncwarp();
        if (mine && !(blockIdx.x == 0 && it == args.drop_load_block)) {
          for (int c = 0; c < C::kDimBoxes; ++c)
            tma_load_4d(t.fresh ? &args.tmap_k_new : &args.tmap_k, k_tile(s) + c * C::kBoxBytes + lane * box_rows * 128u,
                        k_full(s), 64 * c, w.h, slot0, t.fresh ? w.b : page);
        }
        issued_k.note(s, ph);
        if (j == w.j0) {
          // the segment's queries, behind its first keys: their slots are free
          // only once the segment before has multiplied its last keys
          for (int u = 0; u < args.units && ok; ++u) {
            const int slot = parity_mode ? seg & 1 : u;
            const uint32_t q_ph = static_cast<uint32_t>(parity_mode ? seg >> 1 : seg) & 1u;
            ok = wd.warp_wait(q_empty(slot), q_ph ^ 1u);
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(q_full(slot), q_bytes);
              for (int c = 0; c < C::kDimBoxes; ++c)
                tma_load_4d(&args.tmap_q, q_tile(slot) + c * C::kBoxBytes, q_full(slot), 64 * c, w.h * args.group,
                            (w.ru * args.units + u) * args.tile_tokens, w.b);
            }
            if (ok) issued_q.note(slot, q_ph);
          }
          if (!ok) break;
        }
        const int sv = it % C::kVStages;
        const uint32_t phv = static_cast<uint32_t>(it / C::kVStages) & 1u;
        if (!(ok = wd.warp_wait(v_empty(sv), phv ^ 1u))) break;
        if (lane == 0) mbar_arrive_expect_tx(v_full(sv), bytes);
        __syncwarp();
        if (mine) {
          for (int c = 0; c < C::kDimBoxes; ++c)
            tma_load_4d(t.fresh ? &args.tmap_v_new : &args.tmap_v, v_tile(sv) + c * C::kBoxBytes + lane * box_rows * 128u,
                        v_full(sv), 64 * c, w.h, slot0, t.fresh ? w.b : page);
        }
        issued_v.note(sv, phv);
        page = next_page;
      }
    }
    // Loads may still be landing if another role gave up: wait (bounded) for
    // every phase issued before the CTA may exit.
    issued_q.drain(wd, 2, q_full);
    issued_k.drain(wd, C::kKStages, k_full);
    issued_v.drain(wd, C::kVStages, v_full);
  } else if (warp == ta::kMmaWarp) {
    {
      // ------------------------------------------------------------ MMA issuer
      // (the whole warp runs this, one lane issues)
      const uint32_t leader = elect_one();
      int it0 = 0;                    // ring number of the segment's first tile
      int seg = 0;
      int done[2] = {0, 0};           // tiles of each unit whose P has been asked for
      bool ok = true;
      for (; ok && w.more(); it0 += w.count, w.next(args), ++seg) {
        const int end[2] = {w.unit_end(args, 0), w.unit_end(args, 1)};
        const int step = parity_mode ? 2 : 1;
        int products = parity_mode ? w.count : end[0] + end[1] - 2 * w.j0;   // Q K^T still to issue
        // the last unit that reads tile j (pair mode: both read it while both walk it)
        auto last_reader = [&](int u, int j) { return parity_mode || u == 1 || j >= end[1]; };
        auto wait_k = [&](int j) {
          const int i = it0 + j - w.j0;
          return wd.warp_wait(k_full(i % C::kKStages), static_cast<uint32_t>(i / C::kKStages) & 1u);
        };
        auto issue_s = [&](int u, int j) {
          const int s = (it0 + j - w.j0) % C::kKStages;
          const int slot = parity_mode ? seg & 1 : u;
          const int valid = ta::tile_of(w.len, w.tl, has_new, j).valid;
          // N: the key columns that hold keys, in steps of 32
          const uint32_t n = static_cast<uint32_t>(max(1, (valid + 31) / 32)) * 32u;
          const uint32_t idesc = C::kIdescS | ((n >> 3) << 17);
          const uint32_t t_s = tmem_base + C::kColS + 128u * static_cast<uint32_t>(u);
#pragma unroll
          for (int c = 0; c < C::kDimBoxes; ++c) {
            const uint64_t a_desc = sw128_kmajor_desc(q_tile(slot) + c * C::kBoxBytes);
            const uint64_t b_desc = sw128_kmajor_desc(k_tile(s) + c * C::kBoxBytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 16 elements of dim = 32 bytes = 2 descriptor units
              mma_f16_warp(leader, t_s, a_desc + 2u * kk, b_desc + 2u * kk, idesc, (c | kk) != 0 ? 1u : 0u);
          }
          mma_commit_warp(leader, s_full(u));
          if (last_reader(u, j)) mma_commit_warp(leader, k_empty(s));
          if (--products == 0)   // Q has been read for the last time
            for (int x = 0; x < args.units; ++x) mma_commit_warp(leader, q_empty(parity_mode ? seg & 1 : x));
        };
        auto issue_pv = [&](int u, int j, bool first) {
          const int s = (it0 + j - w.j0) % C::kVStages;
          const int steps = (ta::tile_of(w.len, w.tl, has_new, j).valid + 15) / 16;
          const uint64_t v_desc = sw128_mnmajor_desc(v_tile(s), C::kBoxBytes);
          const uint32_t t_p = tmem_base + C::kColS + 128u * static_cast<uint32_t>(u);
          const uint32_t t_o = tmem_base + C::kColO + static_cast<uint32_t>(C::kDim * u);
          auto pv = [&](int kk) {   // 16 keys: 8 columns of P; 16 rows of 128 bytes of V
            mma_f16_tmem_a_warp(leader, t_o, t_p + 64u * static_cast<uint32_t>(kk >> 2) + 8u * static_cast<uint32_t>(kk & 3),
                           v_desc + ((static_cast<uint32_t>(kk) * 2048u) >> 4), C::kIdescO,
                           first && kk == 0 ? 0u : 1u);
          };
          if (steps == 8) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) pv(kk);
          } else {
            for (int kk = 0; kk < steps; ++kk) pv(kk);
          }
          if (last_reader(u, j)) mma_commit_warp(leader, v_empty(s));
        };
        for (int u = 0; u < args.units && ok; ++u) {
          const int slot = parity_mode ? seg & 1 : u;
          ok = wd.warp_wait(q_full(slot), static_cast<uint32_t>(parity_mode ? seg >> 1 : seg) & 1u);
        }
        for (int u = 0; u < 2 && ok; ++u) {
          const int j = w.j0 + (parity_mode ? u : 0);
          if (j >= end[u]) continue;
          if (!(ok = wait_k(j))) break;
          tc_fence_after_sync();
          issue_s(u, j);
        }
        for (int j = w.j0; ok && j < w.j0 + w.count; ++j) {
          const int i = it0 + j - w.j0;
          if (!(ok = wd.warp_wait(v_full(i % C::kVStages), static_cast<uint32_t>(i / C::kVStages) & 1u))) break;
          for (int u = 0; u < 2; ++u) {
            if (j >= end[u] || (parity_mode && ((j - w.j0) & 1) != u)) continue;
            if (!(ok = wd.warp_wait(p_full(u), static_cast<uint32_t>(done[u]) & 1u))) break;
            ++done[u];
            tc_fence_after_sync();
            issue_pv(u, j, j - w.j0 < step);
            if (j + step < end[u]) {
              if (!(ok = wait_k(j + step))) break;
              tc_fence_after_sync();
              issue_s(u, j + step);
            } else {
              mma_commit_warp(leader, o_done(u));
            }
          }
        }
      }
      // every MMA issued here must finish before TMEM is freed
      mma_commit_warp(leader, drain_bar);
      wd.drain(drain_bar, 0);
    }
  } else {
    // -------------------------------------------------------------- softmax
    const int u = (static_cast<int>(warp) - ta::kFirstSoftmaxWarp) >> 2;   // unit
    const uint32_t quarter = warp & 3u;                                    // TMEM lanes 32*quarter ..
    const int r = static_cast<int>(quarter * 32u + lane);                  // row of the tile
    const int r_token = r / args.group, r_head = r - r_token * args.group;
    const uint32_t lane_off = (quarter * 32u) << 16;
    const uint32_t t_s = tmem_base + lane_off + C::kColS + 128u * static_cast<uint32_t>(u);
    auto p_col = [&](int key) { return t_s + static_cast<uint32_t>(64 * (key / 64) + (key % 64) / 2); };
    const uint32_t t_o = tmem_base + lane_off + C::kColO + static_cast<uint32_t>(C::kDim * u);
    const float c_log2 = args.scale_log2;
    const int step = parity_mode ? 2 : 1;
    ta::Walk* walks = reinterpret_cast<ta::Walk*>(smem + C::kOffWalks) + 2 * (warp - ta::kFirstSoftmaxWarp);
    if (lane == 0) walks[0] = w;
    __syncwarp();
    int it0 = 0;                    // ring number of the segment's first tile
    uint32_t tiles_done = 0;        // tiles of this unit so far
    uint32_t ends[2] = {0, 0};      // o_done phases of the units so far
    uint32_t joins = 0;             // exchanges so far (parity mode)
    bool ok = true;
    int seg = 0;
    // A segment's Walk lies in shared memory: its end reads again what the key
    // tiles do not need, which then takes no registers there.
    for (; ok; it0 += w.count, ++seg) {
      w = walks[seg & 1];
      if (!w.more()) break;
      {
        // worked out now, while the first scores are awaited: at the end of the
        // segment its reads of the lengths would queue behind the rows' writes
        // (3 us after a part of 256 rows)
        ta::Walk next = w;
        next.next(args);
        __syncwarp();
        if (lane == 0) walks[(seg + 1) & 1] = next;
        __syncwarp();
      }
      const int end[2] = {w.unit_end(args, 0), w.unit_end(args, 1)};
      const int i0 = (w.ru * args.units + (parity_mode ? 0 : u)) * args.tile_tokens;   // first token of the tile
      const int token = i0 + r_token;
      const bool live = r_token < args.tile_tokens && token < w.tl;          // this row exists
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m_ref = 0.0f;        // reference maximum, in units of scale * log2e
      bool unset = live;         // no key seen yet: there is no reference
      float l = 0.0f;            // row sum of probabilities, against m_ref
      const int first = w.j0 + (parity_mode ? u : 0);
      for (int j = first; j < end[u] && ok; j += step) {
        // S_u for key tile j is complete, and with it P_u V of the tile before: O_u is stable
        if (!wd.warp_wait(s_full(u), tiles_done & 1u)) {
          ok = false;
          break;
        }
        ++tiles_done;
        tc_fence_after_sync();
        const ta::Tile t = ta::tile_of(w.len, w.tl, has_new, j);
        if (warp_live && t.valid > 0) {
          float sv[128];
          {
            uint32_t raw[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_load_32x32(t_s + 32u * c, raw[c]);
            tmem_load_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e) sv[c * 32 + e] = __uint_as_float(raw[c][e]);
          }
          if (t.fresh || t.valid < ta::kTileKeys) {
            uint32_t vis[4];
            int limit = t.valid;   // keys of the tile that this row may see, but for the mask
            if (t.fresh && args.mask == nullptr) limit = min(limit, token + 1 - t.index * ta::kTileKeys);
#pragma unroll
            for (int c = 0; c < 4; ++c) vis[c] = cache::low_bits(limit - 32 * c);
            if (t.fresh && args.mask != nullptr && live) {
              const uint64_t* words = args.mask + (static_cast<int64_t>(w.b) * args.tokens + token) * args.mask_words;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint64_t bits = 2 * t.index + c < args.mask_words ? __ldg(words + 2 * t.index + c) : 0ull;
                vis[2 * c] &= static_cast<uint32_t>(bits);
                vis[2 * c + 1] &= static_cast<uint32_t>(bits >> 32);
              }
            }
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (!((vis[e / 32] >> (e % 32)) & 1u)) sv[e] = -INFINITY;
          }
          // probabilities against neg_m into the P columns; returns their sum
          // (packed fp32 pairs: two values per instruction)
          auto exp_pass = [&](float neg_m) {
            const uint64_t cc = f32x2_pack(c_log2, c_log2), mm = f32x2_pack(neg_m, neg_m);
            uint64_t s01 = f32x2_pack(0.0f, 0.0f), s23 = f32x2_pack(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[16];   // 32 scores -> 16 columns of P
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float* x = sv + 32 * c + e;
                float a0, a1, a2, a3;
                f32x2_unpack(f32x2_fma(f32x2_pack(x[0], x[1]), cc, mm), a0, a1);
                f32x2_unpack(f32x2_fma(f32x2_pack(x[2], x[3]), cc, mm), a2, a3);
                const float p0 = ex2_approx(a0);
                const float p1 = ex2_approx(a1);
                const float p2 = ex2_approx(a2);
                const float p3 = ex2_approx(a3);
                s01 = f32x2_add(s01, f32x2_pack(p0, p1));
                s23 = f32x2_add(s23, f32x2_pack(p2, p3));
                pk[e / 2] = ta::pack2<C::kBf16>(p0, p1);
                pk[e / 2 + 1] = ta::pack2<C::kBf16>(p2, p3);
              }
              tmem_store_32x16(p_col(32 * c), pk);
            }
            float sum0, sum1, sum2, sum3;
            f32x2_unpack(s01, sum0, sum1);
            f32x2_unpack(s23, sum2, sum3);
            return (sum0 + sum1) + (sum2 + sum3);
          };
          auto row_max = [&]() {
            float mx0 = sv[0], mx1 = sv[1], mx2 = sv[2], mx3 = sv[3];
#pragma unroll
            for (int e = 4; e < 128; e += 4) {
              mx0 = fmaxf(mx0, sv[e]);
              mx1 = fmaxf(mx1, sv[e + 1]);
              mx2 = fmaxf(mx2, sv[e + 2]);
              mx3 = fmaxf(mx3, sv[e + 3]);
            }
            return fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
          };
          // A row's reference is the maximum of the first tile in which it sees
          // a key; later tiles are taken against it at once. No probability
          // exceeds 2^8 unless the row's sum over the tile does, so only then is
          // the tile's maximum taken, and the reference moved there (the warp
          // then computes the tile again and rescales O: the same softmax). It
          // moves for the sum, not for a probability past 2^8: keys that all lie
          // a little above the first tile's would else be computed twice, tile
          // after tile (256 tokens over 8192 keys 1 to 7 powers of two above the
          // first tile's: 84 us, and 66 where nothing moves).
          // One copy of the code for both: it is long, and fetched cold.
          float alpha = 1.0f, sum = 0.0f;
          bool take_max = __any_sync(0xffffffffu, unset);
          while (true) {
            if (take_max) {
              const float m_tile = row_max() * c_log2;
              if (unset) {
                if (m_tile != -INFINITY) {
                  m_ref = m_tile;
                  unset = false;
                }
              } else if (live && (m_tile > m_ref + 8.0f || (sum > 256.0f && m_tile > m_ref))) {
                alpha = ex2_approx(m_ref - m_tile);
                m_ref = m_tile;
              }
            }
            sum = exp_pass(-m_ref);
            if (take_max || !__any_sync(0xffffffffu, live && sum > 256.0f)) break;   // (a NaN's row is lost either way)
            take_max = true;
            tmem_store_wait();   // the first pass's stores land before they are overwritten
          }
          l = l * alpha + sum;
          if (__any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
            for (int c = 0; c < C::kDim / 32; ++c) {
              uint32_t o[32];
              tmem_load_32x32(t_o + 32u * c, o);
              tmem_load_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_store_32x32(t_o + 32u * c, o);
            }
          }
          tmem_store_wait();
        }
        if (t.valid % 16 != 0) {
          // zero the rows of V behind the last key, up to the end of its 16-key step
          const int i = it0 + j - w.j0;
          if (!wd.warp_wait(v_full(i % C::kVStages), static_cast<uint32_t>(i / C::kVStages) & 1u)) {
            ok = false;
            break;
          }
          const int row_end = (t.valid + 15) / 16 * 16;
          const uint32_t tile = v_tile(i % C::kVStages);
          for (int x = t.valid * 8 + r; x < row_end * 8; x += 128)
#pragma unroll
            for (int c = 0; c < C::kDimBoxes; ++c) st_shared_v4(tile + c * C::kBoxBytes + 16u * x, 0u, 0u, 0u, 0u);
          fence_proxy_async_shared();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(u));
      }
      if (!ok) break;
      // ---------------------------------------------------------- end of a segment
      asm volatile("" ::: "memory");
      w = walks[seg & 1];
      const bool mine = first < end[u];
      if (mine) {
        if (!(ok = wd.warp_wait(o_done(u), ends[u] & 1u))) break;
        ++ends[u];
      }
      float other_m = 0.0f, other_l = 0.0f;   // the other unit's part of this row
      if (parity_mode && end[0] - w.j0 > 1) {
        if (u == 1) {
          // unit 0 joins the rows: hand over maximum and sum, and leave O_1
          // alone until they have been read
          xch[r] = make_float2(m_ref, l);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(xch_full);
          if (!(ok = wd.warp_wait(xch_empty, joins & 1u))) break;
          tc_fence_after_sync();
          ++joins;
          continue;
        }
        if (!(ok = wd.warp_wait(o_done(1), ends[1] & 1u))) break;
        ++ends[1];
        if (!(ok = wd.warp_wait(xch_full, joins & 1u))) break;
        const float2 x = xch[r];
        other_m = x.x;
        other_l = x.y;
      } else if (!mine) {
        continue;
      }
      tc_fence_after_sync();
      if (warp_live) {
        // a part with an empty sum has no reference and nothing in O
        float m = l > 0.0f ? (other_l > 0.0f ? fmaxf(m_ref, other_m) : m_ref) : other_m;
        const float w0 = l > 0.0f ? ex2_approx(m_ref - m) : 0.0f;
        const float w1 = other_l > 0.0f ? ex2_approx(other_m - m) : 0.0f;
        // NaN sums (NaN or infinite inputs) stay NaN
        const float sum = !(l == 0.0f || other_l == 0.0f) ? l * w0 + other_l * w1 : (l == 0.0f ? other_l : l);
        const bool join = __any_sync(0xffffffffu, other_l != 0.0f);
        const bool shared = args.spread > 1;   // the cluster's CTAs join their shares, once all are there
        const bool whole = w.j0 == 0 && w.count == w.tiles && !shared;
        const float f0 = l == 0.0f ? 0.0f : (l > 0.0f ? w0 : 1.0f);
        const float f1 = other_l == 0.0f ? 0.0f : (other_l > 0.0f ? w1 : 1.0f);
        const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
        const int64_t out_row = (static_cast<int64_t>(w.b) * args.tokens + token) * args.heads + w.h * args.group + r_head;
        const int slot = static_cast<int>(blockIdx.x) * 2 + (w.j0 == 0 ? 1 : 0);
        const int part_unit_row = (parity_mode ? 0 : u) * ta::kTileRows + r;
        const int64_t part_row = static_cast<int64_t>(slot) * args.part_rows + part_unit_row;
        if (live) {
          if (whole) {
            if (args.lse != nullptr)
              args.lse[out_row] = sum == 0.0f ? -INFINITY : (m * ta::kLn2 + logf(sum));
          } else {
            // (this thread has read the other unit's maximum and sum from there)
            *(shared ? xch + r : args.part_ml + part_row) = make_float2(m, sum);
          }
        }
        uint16_t* out = static_cast<uint16_t*>(args.o) + out_row * C::kDim;
        // [slot][dim / 4][row] pieces of four: a warp's 32 rows store 512 contiguous bytes at a time
        // (a share over the K ring, which has been read for the last time)
        float4* part = shared ? reinterpret_cast<float4*>(smem + C::kOffK) + r
                              : reinterpret_cast<float4*>(args.part_o) +
                                    static_cast<int64_t>(slot) * args.part_rows * (C::kDim / 4) + part_unit_row;
        const int part_pitch = args.part_rows;
#pragma unroll 1   // once per segment: short code, which is fetched cold, is faster than unrolled code
        for (int c = 0; c < C::kDim / 32; ++c) {
          uint32_t o[32];
          tmem_load_32x32(t_o + 32u * c, o);
          tmem_load_wait();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = f0 != 0.0f ? __uint_as_float(o[e]) * f0 : 0.0f;
          if (join) {
            tmem_load_32x32(t_o + static_cast<uint32_t>(C::kDim) + 32u * c, o);
            tmem_load_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] += f1 != 0.0f ? __uint_as_float(o[e]) * f1 : 0.0f;
          }
          if (live) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float* y = v + 8 * x;
                dst[x] = make_uint4(ta::pack2<C::kBf16>(y[0] * inv, y[1] * inv), ta::pack2<C::kBf16>(y[2] * inv, y[3] * inv),
                                    ta::pack2<C::kBf16>(y[4] * inv, y[5] * inv), ta::pack2<C::kBf16>(y[6] * inv, y[7] * inv));
              }
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                part[(8 * c + x) * part_pitch] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
            }
          }
        }
      }
      if (parity_mode && end[0] - w.j0 > 1) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(xch_empty);
        ++joins;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == ta::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem_base, C::kTmemCols);
  }
  if (args.spread > 1) {
    // every CTA of the cluster comes here, also one that has given up (its
    // waits are bounded) or had no tiles
    cluster_sync_all();
    if (start_walk->b >= 0) ta::join_shares<C>(args, *start_walk, base);
    cluster_sync_all();   // no CTA leaves while its shared memory is read
  }
}

// Joins the parts of the items that a chunk boundary cut. Block x looks at the
// boundary before chunk x + 1; the first boundary inside an item joins it:
// part 0 lies in the chunk before, the others in the chunks after, in order.
// A warp has 32 rows and two four-column pieces of each (blocks: 32 rows by 64
// columns): it reads 512 contiguous bytes of a part at a time.
// With two groups (few rows, perhaps many parts) each takes every other part,
// as an online softmax, and the second hands its sums to the first in shared
// memory.
template <int kDim, bool kBf16, int kGroups>
__global__ void __launch_bounds__(256 * kGroups, 4 / kGroups) tree_attn_join_kernel(const __grid_constant__ TreeArgs args) {
  constexpr int kPieces = kDim / 4;            // four-column pieces of a row
  constexpr int kPer = 2;                      // pieces per thread
  __shared__ float4 other_o[kGroups == 2 ? kPer : 1][kGroups == 2 ? 256 : 1];
  __shared__ float2 other_ml[kGroups == 2 ? 256 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const int chunk = static_cast<int>(blockIdx.x) + 1;
  const int4* cuts = reinterpret_cast<const int4*>(args.cuts) + 2 * chunk;
  const int4 c0 = __ldg(cuts), c1 = __ldg(cuts + 1);
  const int b = c0.x, h = c0.y, ru = c0.z, j0 = c0.w, tiles = c1.x, len = c1.y, tl = c1.z, per_chunk = c1.w;
  if (b < 0 || j0 > per_chunk) return;
  const int parts = 2 + (tiles - j0 - 1) / per_chunk;
  const int rows_per_part = args.part_rows;
  const int group = static_cast<int>(threadIdx.x) >> 8, tid = static_cast<int>(threadIdx.x) & 255;
  const int piece0 = static_cast<int>(blockIdx.z) * 16 + (tid >> 5) * kPer;
  const int row = static_cast<int>(blockIdx.y) * 32 + (tid & 31);
  const int unit = row / ta::kTileRows, r = row % ta::kTileRows;
  const int r_token = r / args.group;
  const int token = (ru * args.units + unit) * args.tile_tokens + r_token;
  const bool live = row < rows_per_part && r_token < args.tile_tokens && token < tl;
  float m = -INFINITY, sum = 0.0f;
  float4 acc[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) acc[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // adds a part; a sum of zero has no reference and nothing in its row
  auto add = [&](float2 ml, const float4* y) {
    if (ml.y == 0.0f) return;
    const float m_new = fmaxf(m, ml.x);
    const float f0 = sum == 0.0f ? 0.0f : ex2_approx(m - m_new), f1 = ex2_approx(ml.x - m_new);
    m = m_new;
    sum = sum * f0 + ml.y * f1;
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      acc[x] = make_float4(acc[x].x * f0 + y[x].x * f1, acc[x].y * f0 + y[x].y * f1, acc[x].z * f0 + y[x].z * f1,
                           acc[x].w * f0 + y[x].w * f1);
  };
  if (live) {
    // a unit whose keys end before the item's last parts left nothing there
    const int own_tiles = ta::unit_tiles(args, len, tl, ru, unit);
    const int own_parts = own_tiles > j0 ? min(parts, 2 + (own_tiles - j0 - 1) / per_chunk) : 1;
    constexpr int kBatch = 4;   // parts read at a time
#pragma unroll 1
    for (int p0 = group; p0 < own_parts; p0 += kBatch * kGroups) {
      float2 ml[kBatch];
      float4 y[kBatch][kPer];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int p = p0 + i * kGroups;
        ml[i] = make_float2(0.0f, 0.0f);
        if (p >= own_parts) continue;
        const int64_t slot = p == 0 ? (chunk - 1) * 2 + 1 : (chunk + p - 1) * 2;
        ml[i] = __ldg(args.part_ml + slot * rows_per_part + row);
#pragma unroll
        for (int x = 0; x < kPer; ++x)
          y[i][x] = __ldg(reinterpret_cast<const float4*>(args.part_o) + (slot * kPieces + piece0 + x) * rows_per_part + row);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) add(ml[i], y[i]);
    }
  }
  if constexpr (kGroups == 2) {
    if (group == 1) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) other_o[x][tid] = acc[x];
      other_ml[tid] = make_float2(m, sum);
    }
    __syncthreads();
    if (group == 1) return;
    float4 y[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) y[x] = other_o[x][tid];
    add(other_ml[tid], y);
  }
  if (!live) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t out_row = (static_cast<int64_t>(b) * args.tokens + token) * args.heads + h * args.group + (r - r_token * args.group);
  uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.o) + out_row * kDim + piece0 * 4);
#pragma unroll
  for (int x = 0; x < kPer; x += 2)
    out[x / 2] = make_uint4(ta::pack2<kBf16>(acc[x].x * inv, acc[x].y * inv), ta::pack2<kBf16>(acc[x].z * inv, acc[x].w * inv),
                            ta::pack2<kBf16>(acc[x + 1].x * inv, acc[x + 1].y * inv),
                            ta::pack2<kBf16>(acc[x + 1].z * inv, acc[x + 1].w * inv));
  if (piece0 == 0 && args.lse != nullptr) args.lse[out_row] = sum == 0.0f ? -INFINITY : (m * ta::kLn2 + logf(sum));
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
    e = cudaFuncSetAttribute(gemm_tn_dev::tree_attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  return cudaLaunchKernelEx(&cfg, gemm_tn_dev::tree_attn_kernel<C>, args);
}

template <int kDim, bool kBf16, int kGroups>
cudaError_t launch_join(const gemm_tn_dev::TreeArgs& args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  const int rows = args.units == 2 ? args.part_rows
                                   : (args.tokens < args.tile_tokens ? args.tokens : args.tile_tokens) * args.group;
  cfg.gridDim = dim3(static_cast<unsigned>(args.chunks - 1), static_cast<unsigned>((rows + 31) / 32), kDim / 64);
  cfg.blockDim = dim3(256 * kGroups, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent_launch_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gemm_tn_dev::tree_attn_join_kernel<kDim, kBf16, kGroups>, args);
}

}  // namespace

int tree_attn_tile_rows() { return gemm_tn_dev::ta::kTileRows; }

cudaError_t launch_tree_attn(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream) {
  using namespace gemm_tn_dev::ta;
  if (head_dim == 64)
    return bf16 ? launch_cfg<Cfg<64, true>>(args, stream) : launch_cfg<Cfg<64, false>>(args, stream);
  if (head_dim == 128)
    return bf16 ? launch_cfg<Cfg<128, true>>(args, stream) : launch_cfg<Cfg<128, false>>(args, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_attn_join(int head_dim, bool bf16, const gemm_tn_dev::TreeArgs& args, cudaStream_t stream) {
  if (args.part_rows <= 32) {   // the decode kernel's items
    if (head_dim == 64) return bf16 ? launch_join<64, true, 2>(args, stream) : launch_join<64, false, 2>(args, stream);
    if (head_dim == 128) return bf16 ? launch_join<128, true, 2>(args, stream) : launch_join<128, false, 2>(args, stream);
  } else {
    if (head_dim == 64) return bf16 ? launch_join<64, true, 1>(args, stream) : launch_join<64, false, 1>(args, stream);
    if (head_dim == 128) return bf16 ? launch_join<128, true, 1>(args, stream) : launch_join<128, false, 1>(args, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gemm_tn_impl

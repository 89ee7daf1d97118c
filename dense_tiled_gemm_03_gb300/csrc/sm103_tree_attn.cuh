// sm103_tree_attn.cuh -- the schedule of the attention over a paged cache,
// shared by its two kernels (sm103_tree_attn.cu, sm103_decode_attn.cu) and the
// one that joins the parts of cut items.
#pragma once

#include <cstdint>

#include "kv_cache_internal.h"
#include "sm103_cache.cuh"

namespace gemm_tn_dev {

namespace ta {

using cache::kTileKeys;
using cache::pack2;
constexpr float kLn2 = 0.69314718055994531f;

// Cached keys and new tokens of sequence b, as the kernels may use them: the
// arrays on the device are clamped to what the cache and the inputs can hold.
__device__ __forceinline__ int cached_len(const TreeArgs& a, int b) {
  return min(max(__ldg(a.lens + b), 0), a.capacity);
}
__device__ __forceinline__ int new_len(const TreeArgs& a, int b) {
  return a.token_lens == nullptr ? a.tokens : min(max(__ldg(a.token_lens + b), 0), a.tokens);
}

// Key tiles that unit `u` of row unit `ru` walks: all cached ones and the new
// ones up to the last token it may see. At least one where the unit has rows
// (an empty tile writes the empty softmax), none where it has not.
__device__ __forceinline__ int unit_tiles(const TreeArgs& a, int len, int tl, int ru, int u) {
  const int i0 = (ru * a.units + u) * a.tile_tokens;
  if (i0 >= tl) return 0;
  const int fresh = a.has_new == 0 ? 0 : (a.mask == nullptr ? min(tl, i0 + a.tile_tokens) : tl);
  const int n = (len + kTileKeys - 1) / kTileKeys + (fresh + kTileKeys - 1) / kTileKeys;
  return max(n, 1);
}

// Key tiles of an item: what its last unit with rows walks.
__device__ __forceinline__ int item_tiles(const TreeArgs& a, int len, int tl, int ru) {
  const int per_item = a.units * a.tile_tokens, i0 = ru * per_item;
  if (i0 >= tl) return 0;
  const int fresh = a.has_new == 0 ? 0 : (a.mask == nullptr ? min(tl, i0 + per_item) : tl);
  return max((len + kTileKeys - 1) / kTileKeys + (fresh + kTileKeys - 1) / kTileKeys, 1);
}

// Places of all row units of one KV head of a sequence: its items' key tiles,
// each item's behind `gap` places that stand for the time a change of items
// costs. With an item per chunk (whole == 2) every item is one place.
__device__ __forceinline__ int head_places(const TreeArgs& a, int len, int tl) {
  int n = 0;
  const int per_item = a.units * a.tile_tokens;
  if (a.whole == 2) return (tl + per_item - 1) / per_item;
#pragma unroll 1
  for (int ru = 0; ru * per_item < tl; ++ru) n += item_tiles(a, len, tl, ru) + a.gap;
  return n;
}

// Walks a chunk: one segment (a run of one item's key tiles) after another.
struct Walk {
  int b, h, ru, j0;      // item and its first tile in this segment
  int len, tl;           // cached keys and new tokens of b
  int tiles;             // tiles of the item
  int left;              // places of the chunk from this segment's first tile on
  int count;             // tiles of the segment

  // The walk that begins at place `off` of the `all` places of sequence b.
  __device__ __forceinline__ void start(const TreeArgs& a, int b_, int all, int off, int left_) {
    b = b_;
    len = cached_len(a, b);
    tl = new_len(a, b);
    const int per_head = all / a.kv_heads;
    h = off / per_head;
    j0 = off - per_head * h;
    left = left_;
    if (a.whole == 2) {
      ru = j0;
      tiles = item_tiles(a, len, tl, ru);
      // the tiles of the cluster's rank-th CTA (perhaps none)
      const int rank = static_cast<int>(blockIdx.x) % a.spread;
      j0 = (rank * tiles + a.spread - 1) / a.spread;
      count = ((rank + 1) * tiles + a.spread - 1) / a.spread - j0;
      left = count;
      return;
    }
#pragma unroll 1
    for (ru = 0; (tiles = item_tiles(a, len, tl, ru)) + a.gap <= j0; ++ru) j0 -= tiles + a.gap;
    j0 -= a.gap;
    left += min(j0, 0);
    j0 = max(j0, 0);
    count = tiles - j0;
    if (a.whole == 0) {
      count = min(count, left);
    } else if (j0 > 0) {
      next(a);   // this item belongs to the chunk before
    }
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const TreeArgs& a) {
    left -= count;
    if (left <= 0) return;
    j0 = 0;
    do {
      if (++ru == a.row_units) {
        ru = 0;
        if (++h == a.kv_heads) {
          h = 0;
          ++b;
          len = cached_len(a, b);
          tl = new_len(a, b);
        }
      }
      tiles = item_tiles(a, len, tl, ru);
    } while (tiles == 0);
    left -= a.gap;
    count = a.whole != 0 ? tiles : min(tiles, left);
  }
  // Past the last tile of the segment that unit u walks.
  __device__ __forceinline__ int unit_end(const TreeArgs& a, int u) const {
    const int end = j0 + count;
    return a.units == 2 ? max(j0, min(end, unit_tiles(a, len, tl, ru, u))) : end;
  }
};

// Keys of tile j that exist: cached tiles first, then the new tokens'.
struct Tile {
  bool fresh;    // new tokens' keys
  int index;     // tile number among its kind
  int valid;     // keys of the tile that exist
};
__device__ __forceinline__ Tile tile_of(int len, int tl, bool has_new, int j) {
  const int nc = (len + kTileKeys - 1) / kTileKeys;
  Tile t;
  t.fresh = j >= nc;
  t.index = t.fresh ? j - nc : j;
  t.valid = min(kTileKeys, max(0, (t.fresh ? (has_new ? tl : 0) : len) - t.index * kTileKeys));
  return t;
}


// Finds this CTA's chunk (its share of it) and notes, for the kernel that joins parts, the item
// that the chunk begins inside of. Called by the whole block; *start and sums
// (32 words) are shared, start->left is 0 before. The block has to synchronise
// before it reads *start.
__device__ __forceinline__ void find_walk(const TreeArgs& a, Walk* start, int* sums) {
  cache::find_start(
      a.batch, a.chunks, a.min_chunk, a.gap, static_cast<int>(blockIdx.x) / a.spread, sums,   // nothing comes before the first item
      [&](int b) { return head_places(a, cached_len(a, b), new_len(a, b)) * a.kv_heads; },
      [&](int b, int all, int off, int left, int chunk_places) {
        Walk w;
        w.start(a, b, all, off, left);
        *start = w;
        if (a.whole == 0 && w.j0 > 0 && w.more()) {
          int4* to = reinterpret_cast<int4*>(a.cuts) + 2 * blockIdx.x;
          to[0] = make_int4(w.b, w.h, w.ru, w.j0);
          to[1] = make_int4(w.tiles, w.len, w.tl, chunk_places);
        }
      });
}
__device__ __forceinline__ void note_no_cut(const TreeArgs& a, const Walk& w) {   // one thread
  if (a.whole == 0 && (!w.more() || w.j0 == 0)) reinterpret_cast<int4*>(a.cuts)[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
}

// The page that lane `lane` copies of cached tile t, box_rows rows at a time.
__device__ __forceinline__ int page_of(const TreeArgs& a, const int32_t* table, const Tile& t, int box_rows, int lane) {
  if (t.fresh || lane * box_rows >= t.valid) return 0;
  int page = __ldg(table + (t.index * kTileKeys + lane * box_rows) / a.page_size);
  if (page < 0 || page >= a.num_pages) {
    // not a page: nothing is read (the copy fills zeros), and the caller is told
    cache::report(a.status, cache::kStatusInvalid);
    page = a.num_pages;
  }
  return page;
}

}  // namespace ta

}  // namespace gemm_tn_dev

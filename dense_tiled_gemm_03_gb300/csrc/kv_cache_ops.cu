// kv_cache_ops.cu -- the operators on a paged key/value cache that move rows:
// kv_cache_append writes new tokens' keys and values into their slots,
// kv_cache_evict chooses the slots that stay by accumulated attention weight
// and moves kept rows from behind into the holes (include/kv_cache.h).
//
// Both are bound by the bytes they move. Rows go 16 bytes a thread, a row of
// one head on 8 or 16 neighbouring threads. GB300: 2 x 8192 tokens of 8 KV
// heads of dim 128 appended (135 MB) in 25.4 us, 5.3 TB/s; 8 sequences of 12001
// to 16384 slots cut to 8192 (250 MB with the weights) in 65.7 us, 19 of them
// the selection.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "kv_cache_internal.h"
#include "sm103_cache.cuh"

namespace gemm_tn_dev {

namespace {

// Where slot `slot` of sequence b, head h begins in the pools (16-byte units);
// -1 where the page table's entry is not a page.
__device__ __forceinline__ int64_t slot_at(const CacheView& c, int b, int h, int slot) {
  const int page = __ldg(c.page_table + static_cast<int64_t>(b) * c.table_stride + slot / c.page_size);
  if (page < 0 || page >= c.num_pages) return -1;
  return page * c.page_stride + (slot % c.page_size) * c.slot_stride + h * c.head_stride;
}

__device__ __forceinline__ int cached_len(const CacheView& c, const int32_t* lens, int b) {
  return min(max(__ldg(lens + b), 0), c.capacity);
}

__device__ __forceinline__ int new_count(const AppendArgs& a, int b) {
  return a.counts == nullptr ? a.max_rows : min(max(__ldg(a.counts + b), 0), a.max_rows);
}

// The length after n more tokens: n may be any count, so the room is compared and not the sum.
__device__ __forceinline__ int longer(const CacheView& c, int len, int n) { return len + min(n, c.capacity - len); }

__device__ __forceinline__ void advance(const AppendArgs& a, int b) {
  const int n = new_count(a, b);
  const int seen = a.seen_out != nullptr ? a.seen[b] : 0;
  a.lens_out[b] = longer(a.c, cached_len(a.c, a.lens, b), n);
  if (a.seen_out != nullptr) a.seen_out[b] = seen + n;
}

}  // namespace

// One thread per 16 bytes of a new row: its key piece and its value piece.
__global__ void __launch_bounds__(256) cache_append_kernel(const __grid_constant__ AppendArgs a, int write_lens) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int piece = static_cast<int>(x % a.c.vec);
  const int64_t row = x / a.c.vec;
  const int h = static_cast<int>(row % a.c.kv_heads);
  const int64_t bi = row / a.c.kv_heads;
  const int i = static_cast<int>(bi % a.max_rows);
  const int64_t b64 = bi / a.max_rows;
  if (b64 >= a.c.batch) return;
  const int b = static_cast<int>(b64);
  if (write_lens != 0 && i == 0 && h == 0 && piece == 0) advance(a, b);
  if (i >= new_count(a, b)) return;
  const int len = cached_len(a.c, a.lens, b), room = a.c.capacity - len;
  if (i >= room) {   // the sequence's pages are full: one thread says so
    if (i == room && h == 0 && piece == 0) cache::report(a.status, cache::kStatusInvalid);
    return;
  }
  const int slot = len + i;
  const int token = a.rows == nullptr ? i : __ldg(a.rows + static_cast<int64_t>(b) * a.max_rows + i);
  const int64_t to = slot_at(a.c, b, h, slot);
  if (token < 0 || token >= a.tokens || to < 0) {
    cache::report(a.status, cache::kStatusInvalid);
    return;
  }
  a.c.k[to + piece] = __ldg(a.k_new + b * a.kn_batch + token * a.kn_token + h * a.kn_head + piece);
  a.c.v[to + piece] = __ldg(a.v_new + b * a.vn_batch + token * a.vn_token + h * a.vn_head + piece);
  if (piece == 0) {
    const int64_t at = (static_cast<int64_t>(b) * a.c.kv_heads + h) * a.c.capacity + slot;
    if (a.weight != nullptr) a.weight[at] = 0.0f;
    if (a.pos != nullptr) a.pos[at] = (a.seen != nullptr ? __ldg(a.seen + b) : len) + i;
  }
}

__global__ void __launch_bounds__(256) cache_advance_kernel(const __grid_constant__ AppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
  if (b < a.c.batch) {
    // lens_out may be lens: read before written, by this thread alone
    const int len = min(max(a.lens[b], 0), a.c.capacity);
    const int n = new_count(a, b);
    if (a.seen_out != nullptr) a.seen_out[b] = a.seen[b] + n;
    a.lens_out[b] = longer(a.c, len, n);
  }
}

// ------------------------------------------------------------------ evict

namespace ev {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kSmemKeys = 40 * 1024;   // keys that a block holds in shared memory
// Most moves of a list that the selecting block makes itself; more are made by a
// kernel of their own. GB300, us, 8 KV heads of dim 128, one kernel and two: 8
// sequences cut from 544 to 512 slots 7.6 and 9.9, from 1504 to 1024 12.8 and
// 13.8, from 4576 to 4096 17.3 and 18.1; 1 sequence from 1504 to 1024 12.3 and 11.5.
constexpr int kFusedMoves = 512;

// An order-preserving whole number for a slot: the newest slots above
// everything, then NaN, then the weights (-0 and +0 alike).
__device__ __forceinline__ uint32_t key_of(float w, bool newest) {
  if (newest) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  const uint32_t bits = w == 0.0f ? 0u : __float_as_uint(w);
  return (bits >> 31) != 0u ? ~bits : bits | 0x80000000u;
}

// Exclusive sum of one value per warp over the block's warps; every thread of
// a warp passes the same x. `sums` is kWarps words of shared memory.
__device__ __forceinline__ int warp_base(int x, int* sums, int* total) {
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  __syncthreads();
  if (lane == 0) sums[warp] = x;
  __syncthreads();
  int v = sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  *total = __shfl_sync(0xffffffffu, v, 31);
  const int before = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
  return warp == 0 ? 0 : before;
}

}  // namespace ev

// Where the rows of a move lie in the pools (16-byte units; -1 for a page that is none).
__device__ __forceinline__ longlong2 places_of(const EvictArgs& a, int b, int h, int2 m) {
  const longlong2 place = make_longlong2(slot_at(a.c, b, h, m.x), slot_at(a.c, b, h, m.y));
  if (place.x < 0 || place.y < 0) {
    cache::report(a.status, cache::kStatusInvalid);
    return make_longlong2(-1, -1);
  }
  return place;
}

// One block per (sequence, KV head), or for few long lists a cluster of `spread`
// blocks that each hold a run of the slots and add up their counts through shared
// memory. The `keep` largest keys are found by
// counting: the range between the smallest and the largest key is cut into 2048
// equal bins, then the bin that holds the keep-th largest, until a bin is one
// key (three passes at most, usually two; bins of the keys' own range and not
// of fixed leading bits, which weights share: counting those into a few bins of
// shared memory one after the other took 20 us of 37 for 64 lists of 16384).
// Ties go to the lowest slots. Then the holes before `keep` and the kept slots
// behind it are numbered in ascending order and paired. Keys are held in shared
// memory where they fit and recomputed from the arrays where they do not.
// kFused: the block moves its rows itself, from a list in shared memory, and
// writes lens_out.
template <bool kFused>
__global__ void __launch_bounds__(ev::kThreads) cache_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ __align__(8) int hist[2][ev::kBins];   // a round's, and the one before's while other blocks read it
  __shared__ int sums[ev::kWarps];
  __shared__ uint32_t extremes[2][ev::kWarps];
  __shared__ uint32_t shared_words[8];   // what the cluster's other blocks read of this one, each word once
  __shared__ int chosen[3];
  __shared__ int2 list[kFused ? ev::kFusedMoves : 1];
  __shared__ longlong2 places[kFused ? ev::kFusedMoves : 1];
  __shared__ uint32_t smem_words[ev::kSmemKeys / 32];
  __shared__ int smem_ranks[2][ev::kSmemKeys / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int spread = kFused ? 1 : a.spread;
  const int bh = static_cast<int>(blockIdx.x) / spread, rank = static_cast<int>(blockIdx.x) - bh * spread;
  const int b = bh / a.c.kv_heads, h = bh - b * a.c.kv_heads;
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int len = cached_len(a.c, a.lens, b);
  const int keep = a.keep;
  const int64_t base = static_cast<int64_t>(bh) * a.c.capacity;
  const float* weight = a.weight + base;
  const int32_t* pos = a.pos != nullptr ? a.pos + base : nullptr;
  const int stay = min(len, keep);
  if (kFused && h == 0 && tid == 0) a.lens_out[b] = stay;
  const int thread = rank * ev::kThreads + tid, threads = spread * ev::kThreads;   // of the list
  if (len <= keep) {
    if (!kFused && thread == 0) a.counts[bh] = 0;
    if (a.weight_out != a.weight)
      for (int s = thread; s < stay; s += threads) a.weight_out[base + s] = weight[s];
    if (a.pos_out != nullptr && a.pos_out != a.pos)
      for (int s = thread; s < stay; s += threads) a.pos_out[base + s] = pos[s];
    return;
  }
  // this block's run of slots: whole words of 32
  const int per_block = ((len + spread - 1) / spread + 31) / 32 * 32;
  const int s0 = min(len, rank * per_block), s1 = min(len, s0 + per_block);
  auto sync = [&] {
    if (spread > 1) cluster_sync_all();
    else __syncthreads();
  };
  // word `at` of the cluster's block i, after a sync
  auto word_of = [&](int i, int at) {
    return spread > 1 ? ld_cluster_u32(map_to_cta(smem_addr(shared_words + at), static_cast<uint32_t>(i))) : shared_words[at];
  };
  // the blocks' values of word `at` before this one's, and of all of them
  auto before_and_all = [&](int at, int* all) {
    int before = 0;
    *all = 0;
    for (int i = 0; i < spread; ++i) {
      if (i == rank) before = *all;
      *all += static_cast<int>(word_of(i, at));
    }
    return before;
  };
  const int first_new = a.recent > 0 ? a.seen[b] - a.recent : 0;   // positions from here on are the newest
  auto load_key = [&](int s) { return ev::key_of(weight[s], a.recent > 0 && pos[s] >= first_new); };
  const bool in_smem = s1 - s0 <= a.smem_keys;
  auto key = [&](int s) { return in_smem ? smem_keys[s - s0] : load_key(s); };
  const int word_pitch = (a.c.capacity + 31) / 32;
  uint32_t* global_words = in_smem ? nullptr : a.words + 3 * static_cast<int64_t>(bh) * word_pitch + s0 / 32;
  uint32_t* words = in_smem ? smem_words : global_words;
  int* hole_ranks = in_smem ? smem_ranks[0] : reinterpret_cast<int*>(global_words + word_pitch);
  int* mover_ranks = in_smem ? smem_ranks[1] : hole_ranks + word_pitch;
  // the newest slots (key 0xffffffff) are counted, and left out of the range
  uint32_t lowest = 0xffffffffu, highest = 0u;
  int newest = 0;
  constexpr int kLoads = 8;   // slots a thread reads at a time
  for (int x0 = s0 + tid; x0 < s1; x0 += kLoads * ev::kThreads) {
    float wt[kLoads];
    int32_t ps[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int s = x0 + i * ev::kThreads;
      wt[i] = s < s1 ? weight[s] : 0.0f;
      ps[i] = s < s1 && a.recent > 0 ? pos[s] : 0;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int s = x0 + i * ev::kThreads;
      if (s >= s1) break;
      const uint32_t k = ev::key_of(wt[i], a.recent > 0 && ps[i] >= first_new);
      if (in_smem) smem_keys[s - s0] = k;
      if (k == 0xffffffffu) {
        ++newest;
      } else {
        lowest = min(lowest, k);
        highest = max(highest, k);
      }
    }
  }
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  highest = __reduce_max_sync(0xffffffffu, highest);
  if (lane == 0) {
    extremes[0][warp] = lowest;
    extremes[1][warp] = highest;
  }
  int total;
  ev::warp_base(__reduce_add_sync(0xffffffffu, newest), sums, &total);
  newest = total;
  lowest = __reduce_min_sync(0xffffffffu, extremes[0][lane]);
  highest = __reduce_max_sync(0xffffffffu, extremes[1][lane]);
  if (spread > 1) {
    if (tid == 0) {
      shared_words[0] = lowest;
      shared_words[1] = highest;
      shared_words[2] = static_cast<uint32_t>(newest);
    }
    sync();
    for (int i = 0; i < spread; ++i) {
      lowest = min(lowest, word_of(i, 0));
      highest = max(highest, word_of(i, 1));
    }
    before_and_all(2, &newest);
  }

  // the keep-th largest key, and how many slots that hold exactly it stay
  uint32_t limit = 0xffffffffu;
  int need = keep, ties = newest;
  if (newest < keep) {
    need = keep - newest;
    limit = lowest;               // keys from here on, 2^bits of them, are looked at
    int bits = 32 - __clz(highest - lowest);
    for (int round = 0;; ++round) {
      const int shift = max(bits - 11, 0);
      int* bins = hist[round & 1];
      for (int x = tid; x < ev::kBins; x += ev::kThreads) bins[x] = 0;
      __syncthreads();
      for (int s = s0 + tid; s < s1; s += ev::kThreads) {
        const uint32_t k = key(s), d = k - limit;
        if (k != 0xffffffffu && k >= limit && (bits == 32 || d < (1u << bits))) atomicAdd(&bins[d >> shift], 1);
      }
      sync();
      // from the top bin down: thread t looks at bins top - 2t and top - 2t - 1
      const int top = ev::kBins - 1 - 2 * tid;
      int n0 = bins[top], n1 = bins[top - 1];
      if (spread > 1) {
        n0 = n1 = 0;
        const uint32_t at = smem_addr(bins + top - 1);
#pragma unroll 8
        for (int i = 0; i < spread; ++i) {
          const int2 n = ld_cluster_s2(map_to_cta(at, static_cast<uint32_t>(i)));
          n0 += n.y;
          n1 += n.x;
        }
      }
      int v = n0 + n1;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
      }
      const int before = ev::warp_base(__shfl_sync(0xffffffffu, v, 31), sums, &total) + v - n0 - n1;   // above this pair
      if (before < need && before + n0 >= need) {
        chosen[0] = top;
        chosen[1] = need - before;
        chosen[2] = n0;
      } else if (before + n0 < need && before + n0 + n1 >= need) {
        chosen[0] = top - 1;
        chosen[1] = need - before - n0;
        chosen[2] = n1;
      }
      __syncthreads();
      limit += static_cast<uint32_t>(chosen[0]) << shift;
      need = chosen[1];
      ties = chosen[2];
      __syncthreads();
      bits = shift;
      if (shift == 0 || ties == 1) break;
    }
    if (bits > 0) {   // one key is left in the bin: it is the limit (no key is 0)
      if (tid == 0) shared_words[3] = 0u;
      __syncthreads();
      for (int s = s0 + tid; s < s1; s += ev::kThreads) {
        const uint32_t k = key(s);
        if (k != 0xffffffffu && k >= limit && k - limit < (1u << bits)) shared_words[3] = k;
      }
      sync();
      limit = 0u;
      for (int i = 0; i < spread; ++i) limit = max(limit, word_of(i, 3));
    }
  }

  // Kept slots as words of 32 bits, and from here on a thread has a run of
  // words: ranks come from one scan of their bit counts.
  const int num_words = (s1 - s0 + 31) / 32;   // word x: slots from s0 + 32 x
  for (int x = warp; x < num_words; x += ev::kWarps) {
    const int s = s0 + 32 * x + lane;
    const uint32_t k = s < s1 ? key(s) : 0u;
    const uint32_t bits = __ballot_sync(0xffffffffu, s < s1 && k >= limit);
    if (lane == 0) words[x] = bits;
  }
  __syncthreads();
  const int run = (num_words + ev::kThreads - 1) / ev::kThreads;
  const int w0 = min(num_words, tid * run), w1 = min(num_words, w0 + run);
  // exclusive sum over the threads of the block
  auto block_base = [&](int x) {
    int v = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += y;
    }
    return ev::warp_base(__shfl_sync(0xffffffffu, v, 31), sums, &total) + v - x;
  };
  if (ties != need) {   // of the slots with the limit's key the lowest `need` stay
    auto tied = [&](int x) {
      uint32_t bits = 0;
      for (uint32_t left = words[x]; left != 0u; left &= left - 1u) {
        const int i = __ffs(left) - 1;
        if (key(s0 + 32 * x + i) == limit) bits |= 1u << i;
      }
      return bits;
    };
    int mine = 0;
    for (int x = w0; x < w1; ++x) mine += __popc(tied(x));
    int stay_here = need - block_base(mine);   // of this thread's ties
    if (spread > 1) {
      if (tid == 0) shared_words[4] = static_cast<uint32_t>(total);
      sync();
      int all;
      stay_here -= before_and_all(4, &all);
    }
    for (int x = w0; x < w1; ++x) {
      uint32_t drop = tied(x);
      for (; drop != 0u && stay_here > 0; --stay_here) drop &= drop - 1u;
      words[x] &= ~drop;
    }
  }
  // slots of word x before `keep`
  auto before_keep = [&](int x) { return cache::low_bits(keep - s0 - 32 * x); };
  auto holes_of = [&](int x) { return ~words[x] & before_keep(x); };
  auto movers_of = [&](int x) { return words[x] & ~before_keep(x); };
  int holes = 0, movers = 0;
  for (int x = w0; x < w1; ++x) {
    holes += __popc(holes_of(x));
    movers += __popc(movers_of(x));
  }
  int hole_rank = block_base(holes);
  const int block_holes = total;
  int mover_rank = block_base(movers);
  if (spread > 1) {
    if (tid == 0) {
      shared_words[5] = static_cast<uint32_t>(block_holes);
      shared_words[6] = static_cast<uint32_t>(total);
    }
    sync();
    hole_rank += before_and_all(5, &total);
    mover_rank += before_and_all(6, &total);
  }
  // as many movers as holes: `total`
  for (int x = w0; x < w1; ++x) {
    hole_ranks[x] = hole_rank;
    mover_ranks[x] = mover_rank;
    hole_rank += __popc(holes_of(x));
    mover_rank += __popc(movers_of(x));
  }
  __syncthreads();
  int2* moves = kFused ? list : a.moves + static_cast<int64_t>(bh) * a.max_moves;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 2
  for (int x = warp; x < num_words; x += ev::kWarps) {
    const uint32_t hole = holes_of(x), mover = movers_of(x);
    if ((hole >> lane) & 1u) moves[hole_ranks[x] + __popc(hole & below)].y = s0 + 32 * x + lane;
    if ((mover >> lane) & 1u) moves[mover_ranks[x] + __popc(mover & below)].x = s0 + 32 * x + lane;
  }
  if (!kFused && thread == 0) a.counts[bh] = total;
  sync();   // the list is complete, every key has been read, and so has every block's shared memory by the others
  // Weights and positions: a kept slot before `keep` keeps its own (copied
  // where they go elsewhere), a moved one takes them along. A thread's reads go
  // out together, before its first write.
  const bool copy_weight = a.weight_out != a.weight, copy_pos = a.pos_out != nullptr && a.pos_out != a.pos;
  constexpr int kBatch = 4;
  if (copy_weight || copy_pos) {
    const int end = min(s1, keep);
    for (int x0 = s0 + tid; x0 < end; x0 += kBatch * ev::kThreads) {
      float wt[kBatch];
      int32_t ps[kBatch];
      bool on[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = x0 + i * ev::kThreads;
        on[i] = s < end && ((words[(s - s0) / 32] >> (s % 32)) & 1u);
        wt[i] = on[i] && copy_weight ? weight[s] : 0.0f;
        ps[i] = on[i] && copy_pos ? pos[s] : 0;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = x0 + i * ev::kThreads;
        if (on[i] && copy_weight) a.weight_out[base + s] = wt[i];
        if (on[i] && copy_pos) a.pos_out[base + s] = ps[i];
      }
    }
  }
  for (int x0 = thread; x0 < total; x0 += kBatch * threads) {
    int2 m[kBatch];
    float wt[kBatch];
    int32_t ps[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m[i] = x0 + i * threads < total ? moves[x0 + i * threads] : make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      wt[i] = weight[m[i].x];
      ps[i] = pos != nullptr ? pos[m[i].x] : 0;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int x = x0 + i * threads;
      if (x >= total) break;
      a.weight_out[base + m[i].y] = wt[i];
      if (a.pos_out != nullptr) a.pos_out[base + m[i].y] = ps[i];
      if (kFused) places[x] = places_of(a, b, h, m[i]);
    }
  }
  if (kFused) {
    __syncthreads();
    const int per_pass = ev::kThreads / a.c.vec, piece = tid % a.c.vec;
    for (int x = tid / a.c.vec; x < total; x += per_pass) {
      const longlong2 place = places[x];
      if (place.x < 0) continue;
      const uint4 k = a.c.k[place.x + piece], v = a.c.v[place.x + piece];
      a.c.k[place.y + piece] = k;
      a.c.v[place.y + piece] = v;
    }
  }
}

// Moves the listed rows: grid (blocks per list, lists). A warp takes 8 moves
// (16 of dim 64); each of its first lanes works out one move's places (page
// look-ups and divisions once a row, not once a piece) and the warp then moves
// the rows, 16 bytes a lane, eight reads a lane in flight.
__global__ void __launch_bounds__(256, 4) cache_move_kernel(const __grid_constant__ EvictArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int piece = lane % a.c.vec, sub = lane / a.c.vec, rows = 32 / a.c.vec;   // rows a warp moves at a time
  for (int bh = static_cast<int>(blockIdx.y); bh < a.c.batch * a.c.kv_heads; bh += static_cast<int>(gridDim.y)) {
    const int b = bh / a.c.kv_heads, h = bh - b * a.c.kv_heads;
    if (h == 0 && blockIdx.x == 0 && threadIdx.x == 0)   // the only reader of lens in this kernel
      a.lens_out[b] = min(min(max(a.lens[b], 0), a.c.capacity), a.keep);
    const int n = __ldg(a.counts + bh);
    const int thread = static_cast<int>(blockIdx.x * 256 + threadIdx.x), threads = static_cast<int>(gridDim.x) * 256;
    const int2* moves = a.moves + static_cast<int64_t>(bh) * a.max_moves;
    const int batch = 4 * rows;   // moves of a warp at a time
    auto place_of = [&](int x) {
      if (lane >= batch || x >= n) return make_longlong2(-1, -1);
      return places_of(a, b, h, __ldg(moves + x));
    };
    // lane l of the first `batch`: move l % rows of the l / rows-th run of `rows` of this warp
    const int stride = threads / 32 * rows, step = 4 * stride;
    int x0 = thread / 32 * rows;
    const int ahead = lane / rows * stride + lane % rows;
    longlong2 place = place_of(x0 + ahead);
    for (; x0 < n; x0 += step) {
      int64_t to[4];
      uint4 k[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t from = __shfl_sync(0xffffffffu, place.x, i * rows + sub);
        to[i] = __shfl_sync(0xffffffffu, place.y, i * rows + sub);
        if (to[i] >= 0) {
          k[i] = a.c.k[from + piece];
          v[i] = a.c.v[from + piece];
        }
      }
      place = place_of(x0 + step + ahead);   // the next moves' look-ups, while the rows are on their way
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (to[i] >= 0) {
          a.c.k[to[i] + piece] = k[i];
          a.c.v[to[i] + piece] = v[i];
        }
    }
  }
}

}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

namespace {

template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                   Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = cache_launch_attributes(attr, cluster);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_cache_append(const gemm_tn_dev::AppendArgs& a, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(a.c.batch) * a.max_rows * a.c.kv_heads * a.c.vec;
  // lens_out and seen_out may be written here only if no block reads them
  const int write_lens = a.lens_out != a.lens && (a.seen_out == nullptr || a.seen_out != a.seen) ? 1 : 0;
  return launch(gemm_tn_dev::cache_append_kernel, dim3(static_cast<unsigned>((threads + 255) / 256), 1, 1), 256, 0, 1, stream,
                a, write_lens);
}

cudaError_t launch_cache_advance(const gemm_tn_dev::AppendArgs& a, cudaStream_t stream) {
  return launch(gemm_tn_dev::cache_advance_kernel, dim3(static_cast<unsigned>((a.c.batch + 255) / 256), 1, 1), 256, 0, 1, stream, a);
}

int evict_smem_keys(int slots) { return std::min(slots, gemm_tn_dev::ev::kSmemKeys); }

int evict_fused_moves() { return gemm_tn_dev::ev::kFusedMoves; }

template <bool kFused>
static cudaError_t launch_select(const gemm_tn_dev::EvictArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(gemm_tn_dev::cache_select_kernel<kFused>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gemm_tn_dev::ev::kSmemKeys * 4);
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch(gemm_tn_dev::cache_select_kernel<kFused>, dim3(static_cast<unsigned>(a.c.batch * a.c.kv_heads * a.spread), 1, 1),
                gemm_tn_dev::ev::kThreads, static_cast<size_t>(a.smem_keys) * 4, a.spread, stream, a);
}

cudaError_t launch_cache_select(const gemm_tn_dev::EvictArgs& a, cudaStream_t stream) {
  return a.moves == nullptr ? launch_select<true>(a, stream) : launch_select<false>(a, stream);
}

cudaError_t launch_cache_move(const gemm_tn_dev::EvictArgs& a, int num_sms, cudaStream_t stream) {
  const int lists = a.c.batch * a.c.kv_heads;
  const int per_block = 8 * 4 * (32 / a.c.vec);   // moves of a block at a time
  const int most = std::max(1, (a.max_moves + per_block - 1) / per_block);
  const int per_list = std::min(most, std::max(1, (num_sms * 8 + lists - 1) / lists));
  return launch(gemm_tn_dev::cache_move_kernel,
                dim3(static_cast<unsigned>(per_list), static_cast<unsigned>(std::min(lists, 65535)), 1), 256, 0, 1, stream, a);
}

}  // namespace gemm_tn_impl

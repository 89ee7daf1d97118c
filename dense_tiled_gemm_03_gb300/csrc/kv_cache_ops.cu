// kv_cache_ops.cu -- the operators on a paged key/value cache that move rows:
// kv_cache_append writes new tokens' keys and values into their slots,
// kv_cache_evict chooses the slots that stay by accumulated attention weight
// and moves kept rows from behind into the holes (include/kv_cache.h).
//
// Both are bound by the bytes they move. Rows go 16 bytes a thread, a row of
// one head on 8 or 16 neighbouring threads.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "gemm_tn_internal.h"
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

__device__ __forceinline__ void advance(const AppendArgs& a, int b) {
  const int n = new_count(a, b);
  const int seen = a.seen_out != nullptr ? a.seen[b] : 0;
  a.lens_out[b] = min(cached_len(a.c, a.lens, b) + n, a.c.capacity);
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
  const int slot = cached_len(a.c, a.lens, b) + i;
  if (slot >= a.c.capacity) {   // the sequence's pages are full
    cache::report(a.status, cache::kStatusInvalid);
    return;
  }
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
    if (a.pos != nullptr) a.pos[at] = (a.seen != nullptr ? __ldg(a.seen + b) : cached_len(a.c, a.lens, b)) + i;
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
    a.lens_out[b] = min(len + n, a.c.capacity);
  }
}

// ------------------------------------------------------------------ evict

namespace ev {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kSmemKeys = 40 * 1024;   // keys that a block holds in shared memory
constexpr int kFusedMoves = 512;   // most moves of a list that the selecting block makes itself

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

// One block per (sequence, KV head). The `keep` largest keys are found by
// counting: the range between the smallest and the largest key is cut into 2048
// equal bins, then the bin that holds the keep-th largest, until a bin is one
// key (three passes at most, usually two; bins of the keys' own range and not
// of fixed leading bits, which weights share: counting those into a few bins of
// shared memory one after the other took 20 us of 37 for 64 lists of 16384).
// Ties go to the lowest slots. Then the holes before `keep` and the kept slots
// behind it are numbered in ascending order by ballots and paired. Keys are
// held in shared memory where they fit and recomputed from the arrays where
// they do not. kFused: the block moves its rows itself, from a list in shared
// memory, and writes lens_out.
template <bool kFused>
__global__ void __launch_bounds__(ev::kThreads) cache_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ int hist[ev::kBins];
  __shared__ int sums[ev::kWarps];
  __shared__ uint32_t extremes[2][ev::kWarps];
  __shared__ int chosen[2];
  __shared__ int2 list[kFused ? ev::kFusedMoves : 1];
  __shared__ longlong2 places[kFused ? ev::kFusedMoves : 1];
  __shared__ uint32_t kept_bits[ev::kSmemKeys / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int bh = static_cast<int>(blockIdx.x);
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
  if (len <= keep) {
    if (!kFused && tid == 0) a.counts[bh] = 0;
    if (a.weight_out != a.weight)
      for (int s = tid; s < stay; s += ev::kThreads) a.weight_out[base + s] = weight[s];
    if (a.pos_out != nullptr && a.pos_out != a.pos)
      for (int s = tid; s < stay; s += ev::kThreads) a.pos_out[base + s] = pos[s];
    return;
  }
  const int first_new = a.recent > 0 ? a.seen[b] - a.recent : 0;   // positions from here on are the newest
  auto load_key = [&](int s) { return ev::key_of(weight[s], a.recent > 0 && pos[s] >= first_new); };
  const bool in_smem = len <= a.smem_keys;
  auto key = [&](int s) { return in_smem ? smem_keys[s] : load_key(s); };
  // the newest slots (key 0xffffffff) are counted, and left out of the range
  uint32_t lowest = 0xffffffffu, highest = 0u;
  int newest = 0;
#pragma unroll 8
  for (int s = tid; s < len; s += ev::kThreads) {
    const uint32_t k = load_key(s);
    if (in_smem) smem_keys[s] = k;
    if (k == 0xffffffffu) {
      ++newest;
    } else {
      lowest = min(lowest, k);
      highest = max(highest, k);
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

  // the keep-th largest key, and how many slots that hold exactly it stay
  uint32_t limit = 0xffffffffu;
  int need = keep, ties = newest;
  if (newest < keep) {
    need = keep - newest;
    limit = lowest;               // keys from here on, 2^bits of them, are looked at
    int bits = 32 - __clz(highest - lowest);
    while (true) {
      const int shift = max(bits - 11, 0);
      for (int x = tid; x < ev::kBins; x += ev::kThreads) hist[x] = 0;
      __syncthreads();
      for (int s = tid; s < len; s += ev::kThreads) {
        const uint32_t k = key(s), d = k - limit;
        if (k != 0xffffffffu && k >= limit && (bits == 32 || d < (1u << bits))) atomicAdd(&hist[d >> shift], 1);
      }
      __syncthreads();
      // from the top bin down: thread t looks at bins top - 2t and top - 2t - 1
      const int top = ev::kBins - 1 - 2 * tid;
      const int n0 = hist[top], n1 = hist[top - 1];
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
      } else if (before + n0 < need && before + n0 + n1 >= need) {
        chosen[0] = top - 1;
        chosen[1] = need - before - n0;
      }
      __syncthreads();
      limit += static_cast<uint32_t>(chosen[0]) << shift;
      need = chosen[1];
      ties = hist[chosen[0]];
      __syncthreads();
      bits = shift;
      if (shift == 0 || ties == 1) break;
    }
    if (bits > 0) {   // one key is left in the bin: it is the limit
      for (int s = tid; s < len; s += ev::kThreads) {
        const uint32_t k = key(s);
        if (k != 0xffffffffu && k >= limit && k - limit < (1u << bits)) extremes[0][0] = k;
      }
      __syncthreads();
      limit = extremes[0][0];
    }
  }

  // each warp has one contiguous run of slots; runs of 32 in ascending order
  const int per_warp = (len + 32 * ev::kWarps - 1) / (32 * ev::kWarps) * 32;
  const int s0 = min(len, warp * per_warp), s1 = min(len, s0 + per_warp);
  const bool some_ties = ties != need;   // not all slots with the limit's key stay
  int ties_before = 0;
  if (some_ties) {
    int mine = 0;
    for (int s = s0; s < s1; s += 32)
      mine += __popc(__ballot_sync(0xffffffffu, s + lane < s1 && key(s + lane) == limit));
    ties_before = ev::warp_base(mine, sums, &total);
  }
  // whether slot s stays; called by whole warps in ascending order from s0
  auto kept = [&](int s, int& tie_rank) {
    const uint32_t k = s + lane < s1 ? key(s + lane) : 0u;
    const bool in = keep > 0 && s + lane < s1;
    if (!some_ties) return in && k >= limit;
    const bool tie = s + lane < s1 && k == limit;
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    const int rank = tie_rank + __popc(tied & ((1u << lane) - 1u));
    tie_rank += __popc(tied);
    return in && (k > limit || (tie && rank < need));
  };
  // a kept slot before `keep` stays where it is
  auto copy = [&](int s) {
    if (a.weight_out != a.weight) a.weight_out[base + s] = weight[s];
    if (a.pos_out != nullptr && a.pos_out != a.pos) a.pos_out[base + s] = pos[s];
  };
  int holes = 0, movers = 0, tie_rank = ties_before;
  for (int s = s0; s < s1; s += 32) {
    const bool k = kept(s, tie_rank);
    const bool in = s + lane < s1;
    holes += __popc(__ballot_sync(0xffffffffu, in && !k && s + lane < keep));
    movers += __popc(__ballot_sync(0xffffffffu, in && k && s + lane >= keep));
  }
  int hole_rank = ev::warp_base(holes, sums, &total);
  int mover_rank = ev::warp_base(movers, sums, &total);   // as many movers as holes
  if (!kFused && tid == 0) a.counts[bh] = total;
  int2* moves = kFused ? list : a.moves + static_cast<int64_t>(bh) * a.max_moves;
  tie_rank = ties_before;
  for (int s = s0; s < s1; s += 32) {
    const bool k = kept(s, tie_rank);
    const bool in = s + lane < s1;
    const bool hole = in && !k && s + lane < keep, mover = in && k && s + lane >= keep;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    const uint32_t below = (1u << lane) - 1u;
    if (hole) moves[hole_rank + __popc(hb & below)].y = s + lane;
    if (mover) moves[mover_rank + __popc(mb & below)].x = s + lane;
    hole_rank += __popc(hb);
    mover_rank += __popc(mb);
    if (in_smem) {
      const uint32_t bits = __ballot_sync(0xffffffffu, k);
      if (lane == 0) kept_bits[s / 32] = bits;
    } else if (k && s + lane < keep) {
      copy(s + lane);
    }
  }
  __syncthreads();   // the list is complete, and every key has been read
  if (in_smem && (a.weight_out != a.weight || (a.pos_out != nullptr && a.pos_out != a.pos))) {
#pragma unroll 8
    for (int s = tid; s < keep; s += ev::kThreads)
      if ((kept_bits[s / 32] >> (s % 32)) & 1u) copy(s);
  }
#pragma unroll 4
  for (int x = tid; x < total; x += ev::kThreads) {
    const int2 m = moves[x];
    a.weight_out[base + m.y] = weight[m.x];
    if (a.pos_out != nullptr) a.pos_out[base + m.y] = pos[m.x];
    // where the rows lie, worked out once and not by every thread that moves a piece
    const longlong2 place = make_longlong2(slot_at(a.c, b, h, m.x), slot_at(a.c, b, h, m.y));
    if (place.x < 0 || place.y < 0) cache::report(a.status, cache::kStatusInvalid);
    if (kFused) places[x] = place;
    else a.places[static_cast<int64_t>(bh) * a.max_moves + x] = place;
  }
  if (kFused) {
    __syncthreads();
    const int per_pass = ev::kThreads / a.c.vec, piece = tid % a.c.vec;
    for (int x = tid / a.c.vec; x < total; x += per_pass) {
      const longlong2 place = places[x];
      if (place.x < 0 || place.y < 0) continue;
      const uint4 k = a.c.k[place.x + piece], v = a.c.v[place.x + piece];
      a.c.k[place.y + piece] = k;
      a.c.v[place.y + piece] = v;
    }
  }
}

// Moves the listed rows: grid (blocks per list, lists).
__global__ void __launch_bounds__(256) cache_move_kernel(const __grid_constant__ EvictArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int per_block = 256 / a.c.vec;
  const int piece = static_cast<int>(threadIdx.x) % a.c.vec;
  const int sub = static_cast<int>(threadIdx.x) / a.c.vec;
  for (int bh = static_cast<int>(blockIdx.y); bh < a.c.batch * a.c.kv_heads; bh += static_cast<int>(gridDim.y)) {
    const int b = bh / a.c.kv_heads;
    if (bh == b * a.c.kv_heads && blockIdx.x == 0 && threadIdx.x == 0)   // the only reader of lens in this kernel
      a.lens_out[b] = min(min(max(a.lens[b], 0), a.c.capacity), a.keep);
    const int n = __ldg(a.counts + bh);
    const longlong2* places = a.places + static_cast<int64_t>(bh) * a.max_moves;
    // four rows a thread at a time, to have enough reads in flight
    const int step = static_cast<int>(gridDim.x) * per_block;
    for (int x0 = static_cast<int>(blockIdx.x) * per_block + sub; x0 < n; x0 += 4 * step) {
      longlong2 place[4];
      uint4 k[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) place[i] = x0 + i * step < n ? __ldg(places + x0 + i * step) : make_longlong2(-1, -1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (place[i].x >= 0 && place[i].y >= 0) {
          k[i] = a.c.k[place[i].x + piece];
          v[i] = a.c.v[place[i].x + piece];
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (place[i].x >= 0 && place[i].y >= 0) {
          a.c.k[place[i].y + piece] = k[i];
          a.c.v[place[i].y + piece] = v[i];
        }
    }
  }
}

}  // namespace gemm_tn_dev

namespace gemm_tn_impl {

namespace {

template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent_launch_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_cache_append(const gemm_tn_dev::AppendArgs& a, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(a.c.batch) * a.max_rows * a.c.kv_heads * a.c.vec;
  // lens_out and seen_out may be written here only if no block reads them
  const int write_lens = a.lens_out != a.lens && (a.seen_out == nullptr || a.seen_out != a.seen) ? 1 : 0;
  return launch(gemm_tn_dev::cache_append_kernel, dim3(static_cast<unsigned>((threads + 255) / 256), 1, 1), 256, 0, stream,
                a, write_lens);
}

cudaError_t launch_cache_advance(const gemm_tn_dev::AppendArgs& a, cudaStream_t stream) {
  return launch(gemm_tn_dev::cache_advance_kernel, dim3(static_cast<unsigned>((a.c.batch + 255) / 256), 1, 1), 256, 0, stream, a);
}

int evict_smem_keys(int capacity) { return std::min(capacity, gemm_tn_dev::ev::kSmemKeys); }

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
  return launch(gemm_tn_dev::cache_select_kernel<kFused>, dim3(static_cast<unsigned>(a.c.batch * a.c.kv_heads), 1, 1),
                gemm_tn_dev::ev::kThreads, static_cast<size_t>(a.smem_keys) * 4, stream, a);
}

cudaError_t launch_cache_select(const gemm_tn_dev::EvictArgs& a, cudaStream_t stream) {
  return a.moves == nullptr ? launch_select<true>(a, stream) : launch_select<false>(a, stream);
}

cudaError_t launch_cache_move(const gemm_tn_dev::EvictArgs& a, int num_sms, cudaStream_t stream) {
  const int lists = a.c.batch * a.c.kv_heads;
  const int rows_per_block = 256 / a.c.vec;
  const int most = std::max(1, (a.max_moves + 4 * rows_per_block - 1) / (4 * rows_per_block));
  const int per_list = std::min(most, std::max(1, (num_sms * 16 + lists - 1) / lists));
  return launch(gemm_tn_dev::cache_move_kernel,
                dim3(static_cast<unsigned>(per_list), static_cast<unsigned>(std::min(lists, 65535)), 1), 256, 0, stream, a);
}

}  // namespace gemm_tn_impl

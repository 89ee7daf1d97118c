// sm103_cache.cuh -- what the kernels over a paged key/value cache share: the
// bounded waits, and the schedule that cuts a ragged batch's key tiles into
// equal contiguous chunks, one per CTA, from the lengths on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "sm103_cache_ptx.cuh"

namespace gemm_tn_dev {

namespace cache {

constexpr int kTileKeys = 128;     // keys per tile
constexpr int kStatusInvalid = 1;  // == GEMM_TN_ERR_INVALID_VALUE
constexpr int kStatusTimeout = 6;  // == GEMM_TN_ERR_TIMEOUT

// The caller's status word, if there is one: the first error wins.
__device__ __forceinline__ void report(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// The part of a wait that did not end at once.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, int* status, uint64_t timeout_ns,
                                        volatile uint32_t* abort_flag) {
  const uint64_t deadline = globaltimer_ns() + timeout_ns;
  while (true) {
    if (mbar_try_wait<false, false>(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() > deadline) {
      report(status, kStatusTimeout);
      *abort_flag = 1u;
      return false;
    }
  }
}
static __device__ __noinline__ bool wait_on_apart(uint32_t bar, uint32_t parity, int* status, uint64_t timeout_ns,
                                                  volatile uint32_t* abort_flag) {
  return wait_on(bar, parity, status, timeout_ns, abort_flag);
}

// kApart: waits that do not end at once are a function of their own, not code
// in each of some twenty places (the attention of wide row tiles: 4 KB less to
// fetch, and 1024 tokens over 8192 keys 236 -> 229 us; the decode kernel has
// registers to spill for the call and was 1.5% slower).
template <bool kApart>
struct Watch {
  int* status;
  uint64_t timeout_ns;
  volatile uint32_t* abort_flag;

  // Wait for the phase of `bar` with parity `parity`; false on timeout or when
  // another role has given up.
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait<false, false>(bar, parity)) return true;
    if constexpr (kApart) return wait_on_apart(bar, parity, status, timeout_ns, abort_flag);
    else return wait_on(bar, parity, status, timeout_ns, abort_flag);
  }

  // The same for a whole warp, with one outcome.
  __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(bar, parity));
  }

  // The same where nothing is late for a while: asks every half a microsecond, and
  // leaves the issue slots to the warps that share them.
  __device__ __forceinline__ bool patient_wait(uint32_t bar, uint32_t parity) const {
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
    bool ok = true;
    while (ok && !mbar_try_wait<false, false>(bar, parity)) {
      __nanosleep(500);
      if (*abort_flag) {
        ok = false;
      } else if (globaltimer_ns() > deadline) {
        report(status, kStatusTimeout);
        *abort_flag = 1u;
        ok = false;
      }
    }
    return __all_sync(0xffffffffu, ok);
  }

  // Bounded wait while draining after a failure; never raises the flag.
  __device__ __forceinline__ bool drain(uint32_t bar, uint32_t parity) const {
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
    while (!mbar_try_wait<false, false>(bar, parity)) {
      if (globaltimer_ns() > deadline) return false;
    }
    return true;
  }
};

// Which phases of up to 32 barriers copies were issued for, so that a producer
// can wait for them before its CTA exits.
struct Issued {
  uint32_t any = 0, phase = 0;

  __device__ __forceinline__ void note(int i, uint32_t parity) {
    any |= 1u << i;
    phase = (phase & ~(1u << i)) | (parity << i);
  }
  template <class Watch, class Bar>
  __device__ __forceinline__ void drain(const Watch& wd, int count, Bar bar) const {
#pragma unroll 1
    for (int i = 0; i < count; ++i)
      if ((any >> i) & 1u) wd.drain(bar(i), (phase >> i) & 1u);
  }
};

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t out;
  if constexpr (kBf16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    out = *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    out = *reinterpret_cast<uint32_t*>(&v);
  }
  return out;
}

__device__ __forceinline__ int warp_scan(int x, uint32_t lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (static_cast<int>(lane) >= d) x += y;
  }
  return x;
}

// Finds where chunk `chunk` of `chunks` starts, with one length per thread: a
// batch of up to blockDim.x sequences costs one round of loads and one scan.
// Called by the whole block (it synchronises); `sums` is 32 words of shared
// memory. tiles_of(b): key tiles of sequence b in all its items; the host has
// made sure that their sum stays below 2^31. The first `skip` tiles belong to
// no chunk. found(b, tiles, off, left,
// chunk_tiles) is called by the one thread whose sequence holds the chunk's
// first tile: the sequence's tiles, the number of the tile among them, the
// tiles of the chunk and of any chunk; no thread calls it for a chunk past the
// end.
template <class TilesOf, class Found>
__device__ __forceinline__ void find_start(int batch, int chunks, int min_chunk, int skip, int chunk, int* sums,
                                           TilesOf tiles_of, Found found) {
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  const uint32_t lane = lane_id();
  const int warp = tid >> 5, warps = threads >> 5;
  int total = 0;       // of the rounds so far; of all of them from the second pass on
  int before = 0;      // second pass: of the rounds before
  int want = 0, left = 0, chunk_tiles = 0;
  // two passes over rounds of `threads` sequences: the total, then the search
  // (a batch of one round is searched with the first pass's scan)
#pragma unroll 1
  for (int b0 = 0, pass = 0; pass < 2; b0 += threads) {
    if (b0 >= batch) {
      b0 = -threads;
      ++pass;
      continue;
    }
    const int b = b0 + tid;
    const int mine = b < batch ? tiles_of(b) : 0;
    int upto = warp_scan(mine, lane);
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int round = 0;
#pragma unroll 1
    for (int w = 0; w < warps; ++w) {
      const int s = sums[w];
      if (w < warp) upto += s;
      round += s;
    }
    if (pass == 0) total += round;
    if (b0 + threads >= batch && pass == 0) {
      chunk_tiles = max((total - skip + chunks - 1) / chunks, min_chunk);
      const int64_t first = static_cast<int64_t>(chunk_tiles) * chunk + skip;
      if (first >= total) return;
      want = static_cast<int>(first);
      left = min(chunk_tiles, total - want);
      if (b0 == 0) pass = 1;   // one round: it has been scanned
    }
    if (pass == 1) {
      upto += before;
      if (want >= upto - mine && want < upto) found(b, mine, want - (upto - mine), left, chunk_tiles);
      before += round;
      if (before > want) return;
    }
  }
}

// First `n` of 32 bits set (n may be negative or past 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

}  // namespace cache

}  // namespace gemm_tn_dev

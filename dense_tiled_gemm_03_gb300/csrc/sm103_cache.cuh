// sm103_cache.cuh -- what the kernels over a paged key/value cache share: the
// bounded waits, and the schedule that cuts a ragged batch's key tiles into
// equal contiguous chunks, one per CTA, from the lengths on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "sm103_ptx.cuh"

namespace gemm_tn_dev {

namespace cache {

constexpr int kTileKeys = 128;     // keys per tile
constexpr int kStatusInvalid = 1;  // == GEMM_TN_ERR_INVALID_VALUE
constexpr int kStatusTimeout = 6;  // == GEMM_TN_ERR_TIMEOUT

// The caller's status word, if there is one: the first error wins.
__device__ __forceinline__ void report(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

struct Watch {
  int* status;
  uint64_t timeout_ns;
  volatile uint32_t* abort_flag;

  // Wait for the phase of `bar` with parity `parity`; false on timeout or when
  // another role has given up.
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait<false, false>(bar, parity)) return true;
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

  // The same for a whole warp, with one outcome.
  __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(bar, parity));
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

__device__ __forceinline__ int64_t warp_scan(int64_t x, uint32_t lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (static_cast<int>(lane) >= d) x += y;
  }
  return x;
}

// Where chunk `chunk` of `chunks` starts. Called by a whole warp; every lane
// gets the answer. seq_tiles(b): key tiles of sequence b, in all its items.
struct Start {
  int64_t chunk_tiles;   // tiles per chunk
  int64_t total;         // tiles in all
  int b;                 // sequence of the chunk's first tile (the batch size past the end) ...
  int64_t off;           // ... and the tile's number in that sequence
};
template <class SeqTiles>
__device__ __forceinline__ Start find_start(int batch, int chunks, int min_chunk, int chunk, uint32_t lane,
                                            SeqTiles seq_tiles) {
  auto tiles_of = [&](int b) { return b < batch ? seq_tiles(b) : int64_t{0}; };
  const int64_t first = tiles_of(static_cast<int>(lane));   // a batch of up to 32 is read once
  int64_t total = first;
  for (int b0 = 32; b0 < batch; b0 += 32) total += tiles_of(b0 + static_cast<int>(lane));
#pragma unroll
  for (int d = 16; d > 0; d /= 2) total += __shfl_xor_sync(0xffffffffu, total, d);
  Start s;
  s.total = total;
  s.chunk_tiles = max((total + chunks - 1) / chunks, static_cast<int64_t>(min_chunk));
  const int64_t want = s.chunk_tiles * chunk;
  s.b = batch;
  s.off = 0;
  int64_t before = 0;
  for (int b0 = 0; b0 < batch && want < total; b0 += 32) {
    const int64_t mine = b0 == 0 ? first : tiles_of(b0 + static_cast<int>(lane));
    const int64_t upto = before + warp_scan(mine, lane);
    const uint32_t past = __ballot_sync(0xffffffffu, upto > want);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      s.b = b0 + l;
      s.off = want - __shfl_sync(0xffffffffu, upto - mine, l);
      break;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  return s;
}

// First `n` of 32 bits set (n may be negative or past 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

}  // namespace cache

}  // namespace gemm_tn_dev

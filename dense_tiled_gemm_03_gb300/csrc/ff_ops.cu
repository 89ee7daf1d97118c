// ff_ops.cu -- the feed-forward operators that only move and scale: the gated
// projection's elementwise gradient and quantising to e4m3 in blocks of 128.
// Both are bound by memory: each element is read once and written once.
#include <type_traits>

#include "ff_pad.h"
#include "sm103_ff.cuh"

namespace gemm_tn_dev {
namespace ff {

// ------------------------------------------------------------------ gated gradient
// h = act(g) u: dg = dh u act'(g), du = dh act(g), in 32 bits from 16-bit
// values, rounded once to 16. 8192 x 8192 bf16: 97 us with silu, 107 with gelu
// (6.9 and 6.3 TB/s); by single elements, where n is odd, 1000 x 2501 with gelu takes
// 12.5 us and by fours 1000 x 2500 7.0.
constexpr int kGradThreads = 256;

// A piece of kWidth 16-bit elements (8, 4 or 1), as a thread loads it.
template <int kWidth>
struct Piece;
template <>
struct Piece<8> {
  using type = uint4;
  static constexpr int kPer = 2;   // pieces that a thread loads before it computes
};
template <>
struct Piece<4> {
  using type = uint2;
  static constexpr int kPer = 4;
};
template <>
struct Piece<1> {
  using type = uint16_t;
  static constexpr int kPer = 8;
};

// Pieces of 8 or 4 are counted in 32 bits, single elements in 64.
template <bool kBf16, int kAct, int kWidth>
__global__ void __launch_bounds__(kGradThreads) gated_grad_kernel(const GatedGradArgs a) {
  using P = typename Piece<kWidth>::type;
  using Index = typename std::conditional<kWidth == 1, uint64_t, uint32_t>::type;
  constexpr int kPer = Piece<kWidth>::kPer;
  griddep_wait();
  griddep_launch_dependents();
  const uint16_t *grad = static_cast<const uint16_t*>(a.grad), *pre = static_cast<const uint16_t*>(a.pre);
  uint16_t* out = static_cast<uint16_t*>(a.out);
  const Index pieces = static_cast<Index>(a.n / kWidth), total = static_cast<Index>(a.m) * pieces;
  const Index step = static_cast<Index>(gridDim.x) * (kGradThreads * kPer);
  for (Index at = static_cast<Index>(blockIdx.x) * (kGradThreads * kPer) + threadIdx.x; at < total; at += step) {
    P dv[kPer], gv[kPer], uv[kPer];
    uint16_t* to[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const Index x = at + i * kGradThreads;
      if (x >= total) continue;
      const Index row = x / pieces;
      const int64_t r = static_cast<int64_t>(row), j = static_cast<int64_t>(x - row * pieces) * kWidth;
      dv[i] = __ldcs(reinterpret_cast<const P*>(grad + r * a.ldg + j));
      gv[i] = __ldcs(reinterpret_cast<const P*>(pre + r * a.ldp + j));
      uv[i] = __ldcs(reinterpret_cast<const P*>(pre + r * a.ldp + a.n + j));
      to[i] = out + r * a.ldo + j;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (at + i * kGradThreads >= total) continue;
      P dg, du;
      if constexpr (kWidth == 1) {
        const float d = widen16<kBf16>(dv[i]);
        const float2 s = act_slope<kAct>(widen16<kBf16>(gv[i]));
        const uint32_t both = pack16<kBf16>(d * widen16<kBf16>(uv[i]) * s.y, d * s.x);
        dg = static_cast<uint16_t>(both);
        du = static_cast<uint16_t>(both >> 16);
      } else {
        const uint32_t *d = reinterpret_cast<const uint32_t*>(&dv[i]), *g = reinterpret_cast<const uint32_t*>(&gv[i]),
                       *u = reinterpret_cast<const uint32_t*>(&uv[i]);
        uint32_t *og = reinterpret_cast<uint32_t*>(&dg), *ou = reinterpret_cast<uint32_t*>(&du);
#pragma unroll
        for (int w = 0; w < kWidth / 2; ++w) {
          const float d0 = widen16<kBf16>(d[w] & 0xFFFFu), d1 = widen16<kBf16>(d[w] >> 16);
          const float2 s0 = act_slope<kAct>(widen16<kBf16>(g[w] & 0xFFFFu));
          const float2 s1 = act_slope<kAct>(widen16<kBf16>(g[w] >> 16));
          og[w] = pack16<kBf16>(d0 * widen16<kBf16>(u[w] & 0xFFFFu) * s0.y, d1 * widen16<kBf16>(u[w] >> 16) * s1.y);
          ou[w] = pack16<kBf16>(d0 * s0.x, d1 * s1.x);
        }
      }
      *reinterpret_cast<P*>(to[i]) = dg;
      *reinterpret_cast<P*>(to[i] + a.n) = du;
    }
  }
}

// ------------------------------------------------------------------ a product's parts joined
// Four columns a thread, the parts added in order (the same bits every time).
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const gemm_tn_impl::JoinRequest q) {
  griddep_wait();
  griddep_launch_dependents();
  const uint64_t pieces = static_cast<uint64_t>(q.pitch / 4), total = static_cast<uint64_t>(q.m) * pieces;
  for (uint64_t x = blockIdx.x * static_cast<uint64_t>(kJoinThreads) + threadIdx.x; x < total;
       x += static_cast<uint64_t>(gridDim.x) * kJoinThreads) {
    const int64_t row = static_cast<int64_t>(total >> 32 == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(pieces) : x / pieces);
    const int64_t col = static_cast<int64_t>(x - static_cast<uint64_t>(row) * pieces) * 4;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* p = q.parts + row * q.pitch + col;
    for (int s = 0; s < q.splits; ++s) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + s * q.part_stride));
      t = s == 0 ? v : make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
    }
    const float v[4] = {t.x, t.y, t.z, t.w};
    const int64_t at = row * q.ldc + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (col + j >= q.n) continue;
      if (q.out_kind == kOutF32) {
        float* c = static_cast<float*>(q.c) + at + j;
        *c = q.accumulate ? *c + v[j] : v[j];
      } else {
        static_cast<uint16_t*>(q.c)[at + j] =
            static_cast<uint16_t>(q.out_kind == kOutBf16 ? pack16<true>(v[j], 0.0f) : pack16<false>(v[j], 0.0f));
      }
    }
  }
}

// ------------------------------------------------------------------ rows laid out for the TMA
// A copy of 16-bit rows at any even address in rows pad_pitch apart, zeros behind
// the columns. A thread makes kPadPer 16-byte pieces of the copies, counted through
// all rows, each from the aligned pieces of the source that hold it: one or two, or
// none behind the row's last column, where the source may end and nothing is loaded.
struct PadArgs {
  gemm_tn_impl::RepackRequest req[2];   // (rows 0: none)
  uint32_t blocks0;                     // of the first
};
constexpr int kPadThreads = 256, kPadPer = 4;

__global__ void __launch_bounds__(kPadThreads) pad_rows_kernel(const PadArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const bool second = blockIdx.x >= a.blocks0;
  const gemm_tn_impl::RepackRequest& q = second ? a.req[1] : a.req[0];
  const uint32_t pieces = static_cast<uint32_t>(q.ld_dst / 8);
  const int64_t total = q.rows * pieces;
  const int64_t first = static_cast<int64_t>(blockIdx.x - (second ? a.blocks0 : 0u)) * (kPadThreads * kPadPer) + threadIdx.x;
  uint4 lo[kPadPer], hi[kPadPer];
  uint32_t shift[kPadPer];
  int valid[kPadPer];   // elements of the piece inside the row
#pragma unroll
  for (int i = 0; i < kPadPer; ++i) {
    const int64_t at = first + i * kPadThreads;
    valid[i] = 0;
    if (at >= total) continue;
    // (rows and pieces of a row stay below 2^30)
    const int64_t row = total < (int64_t{1} << 32) ? static_cast<int64_t>(static_cast<uint32_t>(at) / pieces) : at / pieces;
    const int64_t col = (at - row * pieces) * 8;
    const uintptr_t line = reinterpret_cast<uintptr_t>(q.src) + static_cast<uintptr_t>(row * q.ld_src) * 2;
    const PadPiece piece = pad_piece(line, q.cols, col);
    valid[i] = piece.valid;
    shift[i] = piece.shift;
    const uint4* from = reinterpret_cast<const uint4*>(piece.at);
    lo[i] = piece.first ? __ldg(from) : make_uint4(0u, 0u, 0u, 0u);
    hi[i] = piece.second ? __ldg(from + 1) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kPadPer; ++i) {
    const int64_t at = first + i * kPadThreads;
    if (at >= total) continue;
    uint32_t w[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
    if (shift[i] & 8u) {
#pragma unroll
      for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
    }
    if (shift[i] & 4u) {
#pragma unroll
      for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
    }
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      out[j] = __funnelshift_r(w[j], w[j + 1], (shift[i] & 2u) * 8u);
      const int left = valid[i] - 2 * j;
      if (left < 2) out[j] = left < 1 ? 0u : out[j] & 0xFFFFu;
    }
    reinterpret_cast<uint4*>(q.dst)[at] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ------------------------------------------------------------------ scales laid out for the product
// 32 x 32 tiles through shared memory, lanes along the source's shorter stride.
struct PackArgs {
  gemm_tn_impl::PackRequest req[2];
  int64_t tiles0;   // of the first request
};

__global__ void __launch_bounds__(256) pack_scales_kernel(const PackArgs a) {
  __shared__ float tile[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const bool second = blockIdx.x >= a.tiles0;
  const gemm_tn_impl::PackRequest& q = second ? a.req[1] : a.req[0];
  const int64_t at = static_cast<int64_t>(blockIdx.x) - (second ? a.tiles0 : 0), across = (q.cols + 31) / 32;
  const int64_t i0 = at / across * 32, j0 = at % across * 32;
  const int lane = static_cast<int>(threadIdx.x) & 31, group = static_cast<int>(threadIdx.x) >> 5;
  const bool along_j = q.s_j <= q.s_i;
  for (int g = group; g < 32; g += 8) {
    const int i = along_j ? g : lane, j = along_j ? lane : g;
    if (i0 + i < q.rows && j0 + j < q.cols) tile[i][j] = q.src[(i0 + i) * q.s_i + (j0 + j) * q.s_j];
  }
  __syncthreads();
  for (int i = group; i < 32; i += 8)
    if (i0 + i < q.rows && j0 + lane < q.cols) q.dst[(i0 + i) * q.pitch + j0 + lane] = tile[i][lane];
}

// ------------------------------------------------------------------ e4m3 in blocks of 128
// A block's scale is the least power of two that brings its largest finite
// magnitude to 448 at most (1 for a block of zeros; no less than 2^-126):
// with t = its exponent, the largest magnitude m 2^e has t = e - 8, or e - 7
// where m > 1.75 = 448 / 256. Dividing by a power of two is exact, so the one
// rounding is that to e4m3 (nearest, ties to even). Infinities and NaN become NaN.
//
// A CTA takes a tile of 128 x 128 elements, each thread holding its part in
// registers: 16 bytes a load, all of them issued before the first is used. A
// block of the scales is a row of the tile, the tile, or (transposed) a column.
// Magnitudes are compared as the integers that their bits are (two 16-bit ones
// at a time), infinities and NaN on top: a block whose largest magnitude is one
// of these is looked through again without them.
//
// 16384 x 8192 bf16: 60.3 us (6.7 TB/s), transposed 64; 11001 x 4096 fp32 by
// tiles, transposed: 39 us (5.8 TB/s; 36 with half of it in L2); 16-bit rows at odd addresses, read element by
// element, take twice that. Each row reduced by itself, as floats (32 shuffles
// a thread instead of 8), it took 129 us.

constexpr int kQuantThreads = 256;

// kSrc: 0 fp16, 1 bf16, 2 fp32.
template <int kSrc>
struct Source {
  static constexpr int kWidth = kSrc == 2 ? 4 : 8;          // elements of a 16-byte load
  static constexpr int kLanes = 128 / kWidth;               // threads along a row
  static constexpr int kRows = 128 / (kQuantThreads / kLanes);   // consecutive rows a thread holds: 8, or 16 (fp32)
  static constexpr uint32_t kLargest = kSrc == 0 ? 0x7BFFu : kSrc == 1 ? 0x7F7Fu : 0x7F7FFFFFu;   // finite magnitude

  // Element j of a load, and its magnitude's bits.
  static __device__ __forceinline__ uint32_t bits(const uint32_t (&w)[4], int j) {
    if constexpr (kSrc == 2) return w[j] & 0x7FFFFFFFu;
    return (w[j >> 1] >> ((j & 1) * 16)) & 0x7FFFu;
  }
  static __device__ __forceinline__ float value(const uint32_t (&w)[4], int j) {
    if constexpr (kSrc == 2) return __uint_as_float(w[j]);
    return widen16<kSrc == 1>((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu);
  }
  static __device__ __forceinline__ float of_bits(uint32_t magnitude) {
    if constexpr (kSrc == 2) return __uint_as_float(magnitude);
    return widen16<kSrc == 1>(magnitude);
  }
  // The larger magnitudes of two words of magnitudes, element by element.
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return kSrc == 2 ? max(a, b) : __vmaxu2(a, b); }
  static __device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & (kSrc == 2 ? 0x7FFFFFFFu : 0x7FFF7FFFu); }
  // The largest of a word's.
  static __device__ __forceinline__ uint32_t largest(uint32_t w) { return kSrc == 2 ? w : max(w >> 16, w & 0xFFFFu); }
  static __device__ __forceinline__ uint32_t largest_finite(uint32_t so_far, const uint32_t (&w)[4]) {
#pragma unroll
    for (int j = 0; j < kWidth; ++j) {
      const uint32_t m = bits(w, j);
      if (m <= kLargest) so_far = max(so_far, m);
    }
    return so_far;
  }
};

// The exponent t of the scale of a block whose largest magnitude is `top`.
__device__ __forceinline__ int scale_exponent(float top) {
  if (top == 0.0f) return 0;
  const uint32_t bits = __float_as_uint(top);
  const int t = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return t < -126 ? -126 : t;   // (t <= 120)
}
__device__ __forceinline__ float power_of_two(int t) { return __uint_as_float(static_cast<uint32_t>(t + 127) << 23); }
// The reciprocal of a power of two from its exponent field, exactly.
__device__ __forceinline__ float inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

__device__ __forceinline__ float nan_unless_finite(float x) {
  return fabsf(x) <= 3.402823466e38f ? x : __uint_as_float(0x7FC00000u);
}
__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d) {
  return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}

// The largest over kLanes lanes of each of kCount values a lane: lane l gets value
// (l * kCount / kLanes)'s. Each step halves the values that a lane holds and
// leaves the halves with the partner that keeps them.
template <int kCount, int kLanes>
__device__ __forceinline__ uint32_t largest_of_lanes(uint32_t (&v)[kCount], int lane) {
  int n = kCount;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < kCount / 2; ++i) {
        if (i >= n) continue;
        const uint32_t mine = upper ? v[i + n] : v[i], theirs = upper ? v[i] : v[i + n];
        v[i] = max(mine, __shfl_xor_sync(0xffffffffu, theirs, o));
      }
    } else {
      v[0] = max(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}

template <int kSrc, bool kTileScale, bool kTransposed>
__global__ void __launch_bounds__(kQuantThreads, kSrc == 2 ? 2 : 4) quantize_kernel(const QuantizeArgs a, const int vec_in,
                                                                                    const int vec_out) {
  using S = Source<kSrc>;
  constexpr int kWidth = S::kWidth, kLanes = S::kLanes, kRows = S::kRows, kWarps = kQuantThreads / 32;
  __shared__ __align__(16) float s_scale[128];
  __shared__ uint32_t s_max[kTransposed && !kTileScale ? kWarps : 1][128];
  __shared__ uint32_t s_top[kWarps];
  __shared__ uint32_t s_odd;   // some magnitude of the tile is infinite or NaN
  __shared__ __align__(16) uint8_t s_tile[kTransposed ? 128 * 128 : 16];

  const uint32_t tiles = static_cast<uint32_t>((a.cols + 127) / 128);
  const uint32_t tile_row = blockIdx.x / tiles, tile_col = blockIdx.x - tile_row * tiles;
  const int64_t row0 = static_cast<int64_t>(tile_row) * 128, col0 = static_cast<int64_t>(tile_col) * 128;
  const int lane = static_cast<int>(threadIdx.x) % kLanes, group = static_cast<int>(threadIdx.x) / kLanes;
  const int warp = static_cast<int>(threadIdx.x) >> 5;
  const int64_t col = col0 + lane * kWidth, first = row0 + group * kRows;
  if (threadIdx.x == 0) s_odd = 0;
  griddep_wait();
  griddep_launch_dependents();

  uint32_t w[kRows][4];
  const uint8_t* from = static_cast<const uint8_t*>(a.x) + (first * a.ldx + col) * (16 / kWidth);
  const int64_t pitch = a.ldx * (16 / kWidth);
  if (vec_in != 0 && col + kWidth <= a.cols && first + kRows <= a.rows) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(from + i * pitch));
      w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i][j] = 0u;
      if (first + i >= a.rows) continue;
      const uint8_t* p = from + i * pitch;
      if (vec_in != 0 && col + kWidth <= a.cols) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
        w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
        continue;
      }
#pragma unroll
      for (int j = 0; j < kWidth; ++j) {
        if (col + j >= a.cols) continue;
        if constexpr (kSrc == 2) {
          w[i][j] = reinterpret_cast<const uint32_t*>(p)[j];
        } else {
          w[i][j >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[j]) << ((j & 1) * 16);
        }
      }
    }
  }

  // ---- the blocks' largest magnitudes and scales
  bool odd = false;   // a block of this thread's holds infinities or NaN
  if constexpr (kTileScale) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) most = S::larger(most, S::magnitudes(w[i][j]));
    auto reduce = [&](uint32_t top) {
      top = __reduce_max_sync(0xffffffffu, top);
      if ((threadIdx.x & 31u) == 0) s_top[warp] = top;
      __syncthreads();
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = max(top, s_top[x]);
      return top;
    };
    uint32_t top = reduce(S::largest(most));
    odd = top > S::kLargest;   // of the whole CTA
    if (odd) {
      top = 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) top = S::largest_finite(top, w[i]);
      __syncthreads();
      top = reduce(top);
    }
    const float s = power_of_two(scale_exponent(S::of_bits(top)));
    if (threadIdx.x == 0)
      a.scale[(kTransposed ? tile_col : tile_row) * a.s_line + (kTransposed ? tile_row : tile_col) * a.s_blk] = s;
    if (threadIdx.x < 128) s_scale[threadIdx.x] = s;
    __syncthreads();
  } else if constexpr (!kTransposed) {
    uint32_t top[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t lo = S::larger(S::magnitudes(w[i][0]), S::magnitudes(w[i][1]));
      const uint32_t hi = S::larger(S::magnitudes(w[i][2]), S::magnitudes(w[i][3]));
      top[i] = S::largest(S::larger(lo, hi));
    }
    uint32_t mine = largest_of_lanes<kRows, kLanes>(top, lane);
    odd = __any_sync(0xffffffffu, mine > S::kLargest);   // of the warp's rows
    if (odd) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) top[i] = S::largest_finite(0u, w[i]);
      mine = largest_of_lanes<kRows, kLanes>(top, lane);
    }
    constexpr int kShare = kLanes / kRows;   // lanes that hold the same row's
    if (lane % kShare == 0) s_scale[group * kRows + lane / kShare] = power_of_two(scale_exponent(S::of_bits(mine)));
    __syncthreads();
    const int64_t line = row0 + threadIdx.x;
    if (threadIdx.x < 128 && line < a.rows) a.scale[line * a.s_line + tile_col * a.s_blk] = s_scale[threadIdx.x];
  } else {
    auto reduce = [&](uint32_t (&most)[4]) {   // the columns' largest over the rows, then over the CTA's threads
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kLanes < 32) most[j] = S::larger(most[j], __shfl_xor_sync(0xffffffffu, most[j], kLanes));
        if ((threadIdx.x & 31u) < static_cast<uint32_t>(kLanes)) s_max[warp][lane * 4 + j] = most[j];
      }
      __syncthreads();
      uint32_t top = 0;
      if (threadIdx.x < 128) {
        // column x of the tile: word x * 4 / kWidth
        const int at = static_cast<int>(threadIdx.x) * 4 / kWidth;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) top = S::larger(top, s_max[x][at]);
        if constexpr (kSrc != 2) top = (top >> ((threadIdx.x & 1u) * 16u)) & 0xFFFFu;
      }
      return top;
    };
    uint32_t most[4] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) most[j] = S::larger(most[j], S::magnitudes(w[i][j]));
    uint32_t top = reduce(most);
    if (top > S::kLargest) s_odd = 1u;
    __syncthreads();
    odd = s_odd != 0;   // of the whole CTA
    if (odd) {
#pragma unroll
      for (int j = 0; j < 4; ++j) most[j] = 0u;
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int j = 0; j < kWidth; ++j) {
          const uint32_t m = S::bits(w[i], j);
          const uint32_t finite = m <= S::kLargest ? m : 0u;
          const int word = kSrc == 2 ? j : j >> 1;
          most[word] = S::larger(most[word], kSrc == 2 ? finite : finite << ((j & 1) * 16));
        }
      top = reduce(most);
    }
    if (threadIdx.x < 128) {
      const float s = power_of_two(scale_exponent(S::of_bits(top)));
      s_scale[threadIdx.x] = s;
      const int64_t line = col0 + threadIdx.x;
      if (line < a.cols) a.scale[line * a.s_line + tile_row * a.s_blk] = s;
    }
    __syncthreads();
  }

  // ---- the quotients
  if constexpr (!kTransposed) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = first + i;
      const float inv = inverse(s_scale[group * kRows + i]);
      float v[kWidth];
#pragma unroll
      for (int j = 0; j < kWidth; ++j) v[j] = S::value(w[i], j) * inv;
      if (odd) {
#pragma unroll
        for (int j = 0; j < kWidth; ++j) v[j] = nan_unless_finite(v[j]);
      }
      uint32_t out[kWidth / 4];
#pragma unroll
      for (int j = 0; j < kWidth / 4; ++j) out[j] = quantize4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      if (row >= a.rows) continue;
      uint8_t* q = a.q + row * a.ldq + col;
      if (vec_out != 0 && col + kWidth <= a.cols) {
        if constexpr (kWidth == 8) {
          *reinterpret_cast<uint2*>(q) = make_uint2(out[0], out[1]);
        } else {
          *reinterpret_cast<uint32_t*>(q) = out[0];
        }
      } else {
#pragma unroll
        for (int j = 0; j < kWidth; ++j)
          if (col + j < a.cols) q[j] = static_cast<uint8_t>(out[j >> 2] >> ((j & 3) * 8));
      }
    }
  } else {
    // the tile by columns, in pieces of 8 rows; a column's piece p lies at
    // p ^ (its lane), so that the lanes of a warp write to all banks
    constexpr int kPieces = kRows / 8;
#pragma unroll
    for (int j = 0; j < kWidth; ++j) {
      const int c = lane * kWidth + j;
      const float inv = inverse(s_scale[c]);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = S::value(w[8 * p + i], j) * inv;
        if (odd) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = nan_unless_finite(v[i]);
        }
        const int piece = (group * kPieces + p) ^ (lane & 15);
        *reinterpret_cast<uint2*>(s_tile + c * 128 + piece * 8) =
            make_uint2(quantize4(v[0], v[1], v[2], v[3]), quantize4(v[4], v[5], v[6], v[7]));
      }
    }
    __syncthreads();
    // 16 threads to a column (a line of q): 8 bytes each
    const int piece = static_cast<int>(threadIdx.x) & 15;
    const int64_t along = row0 + piece * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 16 + (static_cast<int>(threadIdx.x) >> 4);
      const int64_t line = col0 + c;
      if (line >= a.cols || along >= a.rows) continue;
      const uint2 v = *reinterpret_cast<const uint2*>(s_tile + c * 128 + (piece ^ ((c / kWidth) & 15)) * 8);
      uint8_t* q = a.q + line * a.ldq + along;
      if (vec_out != 0 && along + 8 <= a.rows) {
        *reinterpret_cast<uint2*>(q) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (along + j < a.rows) q[j] = static_cast<uint8_t>((j < 4 ? v.x : v.y) >> ((j & 3) * 8));
      }
    }
  }
}

}  // namespace ff
}  // namespace gemm_tn_dev

namespace gemm_tn_impl {
namespace {

using namespace gemm_tn_dev;

template <class Args, class... Rest>
cudaError_t launch(void (*kernel)(Args, Rest...), dim3 grid, int threads, cudaStream_t stream, bool early, const Args& args,
                   Rest... rest) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early && dependent_launch_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args, rest...);
}
// Its set-up may overlap the kernel before it in the stream.
template <class Args, class... Rest>
cudaError_t launch_dependent(void (*kernel)(Args, Rest...), dim3 grid, int threads, cudaStream_t stream, const Args& args,
                             Rest... rest) {
  return launch<Args, Rest...>(kernel, grid, threads, stream, true, args, rest...);
}
// It starts when all before it in the stream has ended. The copies into a
// workspace are launched so: their workspace was freed and allocated anew behind the
// product before. (In rows of 600 calls of A^T B, 16384 x 4095 over 8192 tokens,
// whose copies could start early, the GPU came to a stop; captured rows, where
// the memory's nodes lie between, and rows without copies never did.)
template <class Args>
cudaError_t launch_in_order(void (*kernel)(Args), dim3 grid, int threads, cudaStream_t stream, const Args& args) {
  return launch<Args>(kernel, grid, threads, stream, false, args);
}

template <bool kBf16, int kWidth>
cudaError_t launch_grad(const GatedGradArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int64_t kPerBlock = ff::kGradThreads * ff::Piece<kWidth>::kPer;
  const int64_t blocks = (a.m * (a.n / kWidth) + kPerBlock - 1) / kPerBlock, most = static_cast<int64_t>(num_sms) * 64;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
  auto kernel = a.activation == ff::kSilu   ? ff::gated_grad_kernel<kBf16, ff::kSilu, kWidth>
                : a.activation == ff::kGelu ? ff::gated_grad_kernel<kBf16, ff::kGelu, kWidth>
                                            : ff::gated_grad_kernel<kBf16, ff::kRelu, kWidth>;
  return launch_dependent<GatedGradArgs>(kernel, grid, ff::kGradThreads, stream, a);
}

template <int kSrc>
cudaError_t launch_quant(int block_rows, bool transpose, const QuantizeArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(((a.cols + 127) / 128) * ((a.rows + 127) / 128)));
  const bool in = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % (kSrc == 2 ? 4 : 8) == 0;
  const bool out = reinterpret_cast<uintptr_t>(a.q) % 8 == 0 && a.ldq % 8 == 0;
  auto kernel = block_rows == 1 ? (transpose ? ff::quantize_kernel<kSrc, false, true> : ff::quantize_kernel<kSrc, false, false>)
                                : (transpose ? ff::quantize_kernel<kSrc, true, true> : ff::quantize_kernel<kSrc, true, false>);
  return launch_dependent<QuantizeArgs, int, int>(
      kernel, grid, ff::kQuantThreads, stream, a, in ? 1 : 0, out ? 1 : 0);
}

}  // namespace

cudaError_t launch_gated_grad(bool bf16, const GatedGradArgs& a, int num_sms, cudaStream_t stream) {
  // the widest pieces that n, the pitches and the pointers allow (and 32-bit counts)
  auto allow = [&](int width) {
    auto fits = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % (2 * width) == 0 && ld % width == 0; };
    return a.n % width == 0 && fits(a.grad, a.ldg) && fits(a.pre, a.ldp) && fits(a.out, a.ldo) &&
           a.m * (a.n / width) < (int64_t{1} << 31);
  };
  if (allow(8)) return bf16 ? launch_grad<true, 8>(a, num_sms, stream) : launch_grad<false, 8>(a, num_sms, stream);
  if (allow(4)) return bf16 ? launch_grad<true, 4>(a, num_sms, stream) : launch_grad<false, 4>(a, num_sms, stream);
  return bf16 ? launch_grad<true, 1>(a, num_sms, stream) : launch_grad<false, 1>(a, num_sms, stream);
}

cudaError_t launch_join_parts(const JoinRequest& req, int num_sms, cudaStream_t stream) {
  const int64_t blocks = (req.m * (req.pitch / 4) + ff::kJoinThreads - 1) / ff::kJoinThreads;
  const int64_t most = static_cast<int64_t>(num_sms) * 32;
  return launch_dependent<JoinRequest>(ff::join_parts_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                                       ff::kJoinThreads, stream, req);
}

cudaError_t launch_pad_rows(const RepackRequest (&req)[2], cudaStream_t stream) {
  ff::PadArgs args{{req[0], req[1]}, 0};
  constexpr int64_t kPerBlock = ff::kPadThreads * ff::kPadPer;
  int64_t blocks[2];
  for (int x = 0; x < 2; ++x) blocks[x] = (req[x].rows * (req[x].ld_dst / 8) + kPerBlock - 1) / kPerBlock;
  if (blocks[0] + blocks[1] > INT32_MAX) return cudaErrorInvalidConfiguration;
  args.blocks0 = static_cast<uint32_t>(blocks[0]);
  return launch_in_order<ff::PadArgs>(ff::pad_rows_kernel, dim3(static_cast<unsigned>(blocks[0] + blocks[1])), ff::kPadThreads,
                                      stream, args);
}

cudaError_t launch_pack_scales(const PackRequest (&req)[2], cudaStream_t stream) {
  ff::PackArgs args{{req[0], req[1]}, 0};
  int64_t tiles[2];
  for (int x = 0; x < 2; ++x) tiles[x] = (req[x].rows + 31) / 32 * ((req[x].cols + 31) / 32);
  args.tiles0 = tiles[0];
  return launch_in_order<ff::PackArgs>(ff::pack_scales_kernel, dim3(static_cast<unsigned>(tiles[0] + tiles[1])), 256, stream,
                                       args);
}

cudaError_t launch_quantize(int src_kind, int block_rows, bool transpose, const QuantizeArgs& a, cudaStream_t stream) {
  switch (src_kind) {
    case 0: return launch_quant<0>(block_rows, transpose, a, stream);
    case 1: return launch_quant<1>(block_rows, transpose, a, stream);
    default: return launch_quant<2>(block_rows, transpose, a, stream);
  }
}

}  // namespace gemm_tn_impl

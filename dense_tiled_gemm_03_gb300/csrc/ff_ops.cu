// ff_ops.cu -- the feed-forward operators that only move and scale: the gated
// projection's elementwise gradient and quantising to e4m3 in blocks of 128.
// Both are bound by memory: each element is read once and written once.
#include "sm103_ff.cuh"

namespace gemm_tn_dev {
namespace ff {

// ------------------------------------------------------------------ gated gradient
// h = act(g) u: dg = dh u act'(g), du = dh act(g), in 32 bits from 16-bit
// values, rounded once to 16.
constexpr int kGradThreads = 256;
constexpr int kGradPer = 2;   // 8-element pieces a thread loads before it computes

template <bool kBf16, int kAct>
__device__ __forceinline__ void grad_piece(const uint4& d4, const uint4& g4, const uint4& u4, uint4& dg4, uint4& du4) {
  const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w}, g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
  uint32_t og[4], ou[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float d0 = widen16<kBf16>(d[j] & 0xFFFFu), d1 = widen16<kBf16>(d[j] >> 16);
    const float2 a0 = act_slope<kAct>(widen16<kBf16>(g[j] & 0xFFFFu)), a1 = act_slope<kAct>(widen16<kBf16>(g[j] >> 16));
    og[j] = pack16<kBf16>(d0 * widen16<kBf16>(u[j] & 0xFFFFu) * a0.y, d1 * widen16<kBf16>(u[j] >> 16) * a1.y);
    ou[j] = pack16<kBf16>(d0 * a0.x, d1 * a1.x);
  }
  dg4 = make_uint4(og[0], og[1], og[2], og[3]);
  du4 = make_uint4(ou[0], ou[1], ou[2], ou[3]);
}

// 16-byte pieces are counted in 32 bits (2^32 of them would be 64 GiB an
// operand), single elements in 64.
template <bool kVec>
struct IndexOf {
  using type = uint32_t;
};
template <>
struct IndexOf<false> {
  using type = uint64_t;
};

// kVec: 16-byte pieces (n, the pitches and the pointers allow them); else
// element by element.
template <bool kBf16, int kAct, bool kVec>
__global__ void __launch_bounds__(kGradThreads) gated_grad_kernel(const GatedGradArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const uint16_t *grad = static_cast<const uint16_t*>(a.grad), *pre = static_cast<const uint16_t*>(a.pre);
  uint16_t* out = static_cast<uint16_t*>(a.out);
  constexpr int kWidth = kVec ? 8 : 1;
  using Index = typename IndexOf<kVec>::type;
  const Index pieces = static_cast<Index>(a.n / kWidth), total = static_cast<Index>(a.m) * pieces;
  const Index step = static_cast<Index>(gridDim.x) * (kGradThreads * kGradPer);
  for (Index at = static_cast<Index>(blockIdx.x) * (kGradThreads * kGradPer) + threadIdx.x; at < total; at += step) {
    if constexpr (kVec) {
      uint4 dv[kGradPer], gv[kGradPer], uv[kGradPer];
      uint4* to[kGradPer];
#pragma unroll
      for (int i = 0; i < kGradPer; ++i) {
        const Index x = at + i * kGradThreads;
        if (x >= total) continue;
        const Index row = x / pieces, p = x - row * pieces;
        const int64_t r = static_cast<int64_t>(row);
        dv[i] = __ldcs(reinterpret_cast<const uint4*>(grad + r * a.ldg) + p);
        gv[i] = __ldcs(reinterpret_cast<const uint4*>(pre + r * a.ldp) + p);
        uv[i] = __ldcs(reinterpret_cast<const uint4*>(pre + r * a.ldp + a.n) + p);
        to[i] = reinterpret_cast<uint4*>(out + r * a.ldo) + p;
      }
#pragma unroll
      for (int i = 0; i < kGradPer; ++i) {
        if (at + i * kGradThreads >= total) continue;
        uint4 x, y;
        grad_piece<kBf16, kAct>(dv[i], gv[i], uv[i], x, y);
        to[i][0] = x;
        to[i][pieces] = y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kGradPer; ++i) {
        const Index x = at + i * kGradThreads;
        if (x >= total) continue;
        const int64_t row = static_cast<int64_t>(x / pieces), j = static_cast<int64_t>(x) - row * a.n;
        const float d = widen16<kBf16>(grad[row * a.ldg + j]), u = widen16<kBf16>(pre[row * a.ldp + a.n + j]);
        const float2 s = act_slope<kAct>(widen16<kBf16>(pre[row * a.ldp + j]));
        const uint32_t both = pack16<kBf16>(d * u * s.y, d * s.x);
        out[row * a.ldo + j] = static_cast<uint16_t>(both);
        out[row * a.ldo + a.n + j] = static_cast<uint16_t>(both >> 16);
      }
    }
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

constexpr int kQuantThreads = 256;

__device__ __forceinline__ float finite_magnitude(float x) {
  const float m = fabsf(x);
  return m <= 3.402823466e38f ? m : 0.0f;
}

// The exponent t of the scale of a block whose largest magnitude is `top`.
__device__ __forceinline__ int scale_exponent(float top) {
  if (top == 0.0f) return 0;
  const uint32_t bits = __float_as_uint(top);
  const int t = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return t < -126 ? -126 : t;   // (t <= 120)
}
__device__ __forceinline__ float power_of_two(int t) { return __uint_as_float(static_cast<uint32_t>(t + 127) << 23); }

__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, float inv) {
  auto scaled = [&](float x) { return fabsf(x) <= 3.402823466e38f ? x * inv : __uint_as_float(0x7FC00000u); };
  return cvt_e4m3x2(scaled(a), scaled(b)) | (cvt_e4m3x2(scaled(c), scaled(d)) << 16);
}

// kSrc: 0 fp16, 1 bf16, 2 fp32.
template <int kSrc>
__device__ __forceinline__ float element(const void* x, int64_t at) {
  if constexpr (kSrc == 2) {
    return static_cast<const float*>(x)[at];
  } else {
    return widen16<kSrc == 1>(static_cast<const uint16_t*>(x)[at]);
  }
}

template <int kSrc, bool kTileScale, bool kTransposed>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantizeArgs a, const int vec_in,
                                                                  const int vec_out) {
  constexpr int kWidth = kSrc == 2 ? 4 : 8;          // elements of a 16-byte load
  constexpr int kLanes = 128 / kWidth;               // threads along a row
  constexpr int kRows = 128 / (kQuantThreads / kLanes);   // consecutive rows a thread holds: 8, or 16 (fp32)
  __shared__ float s_scale[128];
  __shared__ float s_max[kQuantThreads / 32][128];
  __shared__ __align__(16) uint8_t s_tile[kTransposed ? 128 * 128 : 16];

  const uint32_t tiles = static_cast<uint32_t>((a.cols + 127) / 128);
  const uint32_t tile_row = blockIdx.x / tiles, tile_col = blockIdx.x - tile_row * tiles;
  const int64_t row0 = static_cast<int64_t>(tile_row) * 128, col0 = static_cast<int64_t>(tile_col) * 128;
  const int lane = static_cast<int>(threadIdx.x) % kLanes, group = static_cast<int>(threadIdx.x) / kLanes;
  const int64_t col = col0 + lane * kWidth;
  const int warp = static_cast<int>(threadIdx.x) >> 5;
  griddep_wait();
  griddep_launch_dependents();

  float v[kRows][kWidth];
  const bool whole = vec_in != 0 && col + kWidth <= a.cols;
  if (whole) {
    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = row0 + group * kRows + i;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < a.rows)
        raw[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) +
                                                       (row * a.ldx + col) * (kSrc == 2 ? 4 : 2)));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < kWidth; ++j) {
        if constexpr (kSrc == 2) {
          v[i][j] = __uint_as_float(w[j]);
        } else {
          v[i][j] = widen16<kSrc == 1>((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = row0 + group * kRows + i;
#pragma unroll
      for (int j = 0; j < kWidth; ++j)
        v[i][j] = row < a.rows && col + j < a.cols ? element<kSrc>(a.x, row * a.ldx + col + j) : 0.0f;
    }
  }

  // scales: s_scale[line of q in this tile] (kTileScale: one for all, in s_scale[0])
  if constexpr (kTileScale) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < kWidth; ++j) top = fmaxf(top, finite_magnitude(v[i][j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31u) == 0) s_max[warp][0] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kQuantThreads / 32; ++w) top = fmaxf(top, s_max[w][0]);
      const float s = power_of_two(scale_exponent(top));
      s_scale[0] = s;
      const int64_t line = kTransposed ? tile_col : tile_row, blk = kTransposed ? tile_row : tile_col;
      a.scale[line * a.s_line + blk * a.s_blk] = s;
    }
    __syncthreads();
  } else if constexpr (!kTransposed) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < kWidth; ++j) top = fmaxf(top, finite_magnitude(v[i][j]));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane == 0) s_scale[group * kRows + i] = power_of_two(scale_exponent(top));
    }
    __syncthreads();
    const int64_t line = row0 + threadIdx.x;
    if (threadIdx.x < 128 && line < a.rows)
      a.scale[line * a.s_line + static_cast<int64_t>(tile_col) * a.s_blk] = s_scale[threadIdx.x];
  } else {
#pragma unroll
    for (int j = 0; j < kWidth; ++j) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) top = fmaxf(top, finite_magnitude(v[i][j]));
      if constexpr (kLanes < 32) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, kLanes));
      if ((threadIdx.x & 31u) < static_cast<uint32_t>(kLanes)) s_max[warp][lane * kWidth + j] = top;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      float top = 0.0f;
      for (int w = 0; w < kQuantThreads / 32; ++w) top = fmaxf(top, s_max[w][threadIdx.x]);
      const float s = power_of_two(scale_exponent(top));
      s_scale[threadIdx.x] = s;
      const int64_t line = col0 + threadIdx.x;
      if (line < a.cols) a.scale[line * a.s_line + static_cast<int64_t>(tile_row) * a.s_blk] = s;
    }
    __syncthreads();
  }
  // the reciprocal of a power of two from its exponent field, exactly
  auto inverse = [](float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); };

  if constexpr (!kTransposed) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = row0 + group * kRows + i;
      const float inv = inverse(s_scale[kTileScale ? 0 : group * kRows + i]);
      uint32_t w[kWidth / 4];
#pragma unroll
      for (int j = 0; j < kWidth / 4; ++j)
        w[j] = quantize4(v[i][4 * j], v[i][4 * j + 1], v[i][4 * j + 2], v[i][4 * j + 3], inv);
      if (row >= a.rows) continue;
      uint8_t* q = a.q + row * a.ldq + col;
      if (vec_out != 0 && col + kWidth <= a.cols) {
        if constexpr (kWidth == 8) {
          *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
        } else {
          *reinterpret_cast<uint32_t*>(q) = w[0];
        }
      } else {
#pragma unroll
        for (int j = 0; j < kWidth; ++j)
          if (col + j < a.cols) q[j] = static_cast<uint8_t>(w[j >> 2] >> ((j & 3) * 8));
      }
    }
  } else {
    // the tile by columns, in pieces of 8 rows; a column's piece p lies at
    // p ^ (its lane), so that the lanes of a warp write to all banks
    constexpr int kPieces = kRows / 8;
#pragma unroll
    for (int j = 0; j < kWidth; ++j) {
      const int c = lane * kWidth + j;
      const float inv = inverse(s_scale[kTileScale ? 0 : c]);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint32_t lo = quantize4(v[8 * p][j], v[8 * p + 1][j], v[8 * p + 2][j], v[8 * p + 3][j], inv);
        const uint32_t hi = quantize4(v[8 * p + 4][j], v[8 * p + 5][j], v[8 * p + 6][j], v[8 * p + 7][j], inv);
        const int piece = (group * kPieces + p) ^ (lane & 15);
        *reinterpret_cast<uint2*>(s_tile + c * 128 + piece * 8) = make_uint2(lo, hi);
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
      const uint2 w = *reinterpret_cast<const uint2*>(s_tile + c * 128 + (piece ^ ((c / kWidth) & 15)) * 8);
      uint8_t* q = a.q + line * a.ldq + along;
      if (vec_out != 0 && along + 8 <= a.rows) {
        *reinterpret_cast<uint2*>(q) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (along + j < a.rows) q[j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> ((j & 3) * 8));
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
cudaError_t launch_dependent(void (*kernel)(Args, Rest...), dim3 grid, int threads, cudaStream_t stream, const Args& args,
                             Rest... rest) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent_launch_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args, rest...);
}

template <bool kBf16, bool kVec>
cudaError_t launch_grad(const GatedGradArgs& a, dim3 grid, cudaStream_t stream) {
  switch (a.activation) {
    case ff::kSilu: return launch_dependent<GatedGradArgs>(ff::gated_grad_kernel<kBf16, ff::kSilu, kVec>, grid, ff::kGradThreads, stream, a);
    case ff::kGelu: return launch_dependent<GatedGradArgs>(ff::gated_grad_kernel<kBf16, ff::kGelu, kVec>, grid, ff::kGradThreads, stream, a);
    default: return launch_dependent<GatedGradArgs>(ff::gated_grad_kernel<kBf16, ff::kRelu, kVec>, grid, ff::kGradThreads, stream, a);
  }
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
  auto wide = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; };
  const bool vec = a.n % 8 == 0 && a.m * (a.n / 8) < (int64_t{1} << 31) && wide(a.grad, a.ldg) && wide(a.pre, a.ldp) && wide(a.out, a.ldo);
  constexpr int64_t kPerBlock = ff::kGradThreads * ff::kGradPer;
  const int64_t units = (a.m * (vec ? a.n / 8 : a.n) + kPerBlock - 1) / kPerBlock;
  const int64_t most = static_cast<int64_t>(num_sms) * 64;
  const dim3 grid(static_cast<unsigned>(units < most ? units : most));
  if (bf16) return vec ? launch_grad<true, true>(a, grid, stream) : launch_grad<true, false>(a, grid, stream);
  return vec ? launch_grad<false, true>(a, grid, stream) : launch_grad<false, false>(a, grid, stream);
}

cudaError_t launch_pack_scales(const PackRequest (&req)[2], cudaStream_t stream) {
  ff::PackArgs args{{req[0], req[1]}, 0};
  int64_t tiles[2];
  for (int x = 0; x < 2; ++x) tiles[x] = (req[x].rows + 31) / 32 * ((req[x].cols + 31) / 32);
  args.tiles0 = tiles[0];
  return launch_dependent<ff::PackArgs>(ff::pack_scales_kernel, dim3(static_cast<unsigned>(tiles[0] + tiles[1])), 256, stream,
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

// sm103_ff.cuh -- what the feed-forward kernels share: bounded waits, the
// activations, the 8-bit tensor-core instruction and the row stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ff_internal.h"
#include "sm103_ptx.cuh"

namespace gemm_tn_dev {
namespace ff {

constexpr int kStatusExpired = 6;   // == GEMM_TN_ERR_TIMEOUT
constexpr int kRelu = 1, kGelu = 2, kSilu = 3;
constexpr int kOutF16 = 0, kOutBf16 = 1, kOutF32 = 2;

// Bounded waits: past the deadline the kernel records the error, tells every
// role of the cluster to stop, and returns.
template <int kClusterSize>
struct Waiter {
  int* status;
  uint64_t timeout_ns;
  volatile uint32_t* abort_flag;
  static constexpr bool kCluster = kClusterSize > 1;

  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait<kCluster>(bar, parity)) return true;
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
    while (true) {
      if (mbar_try_wait<kCluster>(bar, parity)) return true;
      if (*abort_flag) return false;
      if (globaltimer_ns() > deadline) {
        if (status != nullptr) atomicCAS(status, 0, kStatusExpired);
        *abort_flag = 1u;
        if constexpr (kCluster) {
          const uint32_t addr = smem_addr(const_cast<uint32_t*>(abort_flag)), me = cluster_ctarank();
          for (uint32_t r = 0; r < static_cast<uint32_t>(kClusterSize); ++r)
            if (r != me) st_cluster_u32(map_to_cta(addr, r), 1u);
        }
        return false;
      }
    }
  }

  // For what is in flight once another role has given up: never sets the flag.
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
    while (!mbar_try_wait<kCluster>(bar, parity))
      if (globaltimer_ns() > deadline) return;
  }
};

// The last phase issued into each stage of a ring of up to 32 stages.
struct Issued {
  uint32_t issued = 0u, parity = 0u;
  __device__ __forceinline__ void record(int s, uint32_t phase) {
    issued |= 1u << s;
    parity = (parity & ~(1u << s)) | ((phase & 1u) << s);
  }
};

// D[tmem] (+)= A[smem] x B[smem]^T, e4m3 operands, fp32 accumulator; one
// instruction takes 32 elements of K. Its instruction descriptor is that of
// kind::f16 with the formats' fields zero (e4m3).
template <int kCtaGroup>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (kCtaGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
  }
}

// tcgen05.wait::ld as the point where loaded values come to be: an operation on
// them cannot be moved ahead of it.
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
               "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
               "+r"(r[13]), "+r"(r[14]), "+r"(r[15]) :: "memory");
}
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
               "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
               "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
               "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]),
               "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// ------------------------------------------------------------------ activations
// silu: g s with s = 1 / (1 + e^-g); slope s + g s (1 - s).
// gelu: g P with P = erfc(-g / sqrt 2) / 2, the normal distribution's lower
// tail taken directly so that it keeps its relative accuracy far below zero;
// slope P + g e^(-g^2 / 2) / sqrt(2 pi).
// relu: max(g, 0) (NaN stays NaN); slope 1 above zero, else 0.

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
__device__ __forceinline__ float normal_cdf(float g) { return 0.5f * erfcf(-0.70710678118654752f * g); }

template <int kAct>
__device__ __forceinline__ float act(float g) {
  if constexpr (kAct == kSilu) {
    return g * sigmoid(g);
  } else if constexpr (kAct == kGelu) {
    return g * normal_cdf(g);
  } else {
    return g < 0.0f ? 0.0f : g;
  }
}

// The activation and its slope.
template <int kAct>
__device__ __forceinline__ float2 act_slope(float g) {
  if constexpr (kAct == kSilu) {
    const float s = sigmoid(g);
    return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
  } else if constexpr (kAct == kGelu) {
    const float p = normal_cdf(g);
    return make_float2(g * p, fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p));
  } else {
    return make_float2(g < 0.0f ? 0.0f : g, g > 0.0f ? 1.0f : 0.0f);
  }
}

// ------------------------------------------------------------------ 16-bit values

template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kBf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <bool kBf16>
__device__ __forceinline__ float widen16(uint32_t bits) {
  if constexpr (kBf16) {
    return __uint_as_float(bits << 16);
  } else {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
  }
}

// ------------------------------------------------------------------ a warp's 32 x 32 block of C
// Lane l holds row l. The block goes through the warp's staging memory so that
// each store writes whole stretches of rows: 16 bytes a lane where the rows are
// aligned so, else one row's 32 elements an instruction. rows, cols: how many
// of the 32 exist (<= 0: none).

__device__ __forceinline__ void store_block16(uint16_t* c, int64_t ldc, int rows, int cols, const uint32_t (&v)[16],
                                              uint8_t* stage) {
  const uint32_t lane = lane_id();
  const uint32_t s = smem_addr(stage);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    st_shared_v4(s + lane * 64u + ((static_cast<uint32_t>(j) ^ ((lane >> 1) & 3u)) * 16u), v[4 * j], v[4 * j + 1],
                 v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  if (cols >= 32 && ((reinterpret_cast<uintptr_t>(c) | static_cast<uintptr_t>(ldc * 2)) & 15u) == 0) {
    const uint32_t unit = lane & 3u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = static_cast<uint32_t>(i) * 8u + (lane >> 2);
      const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64u + ((unit ^ ((r >> 1) & 3u)) * 16u));
      if (static_cast<int>(r) < rows) *reinterpret_cast<uint4*>(c + static_cast<int64_t>(r) * ldc + unit * 8u) = w;
    }
  } else {
    const bool mine = static_cast<int>(lane) < cols;
    uint16_t* p = c + lane;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      const uint32_t unit = (lane >> 3) ^ ((static_cast<uint32_t>(r) >> 1) & 3u);
      const uint16_t w = *reinterpret_cast<const uint16_t*>(stage + r * 64 + unit * 16u + (lane & 7u) * 2u);
      if (mine && r < rows) *p = w;
      p += ldc;
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void store_block32(float* c, int64_t ldc, int rows, int cols, const float (&v)[32],
                                              bool add, uint8_t* stage) {
  const uint32_t lane = lane_id();
  const uint32_t s = smem_addr(stage);
#pragma unroll
  for (int u = 0; u < 8; ++u)
    st_shared_v4(s + lane * 128u + ((static_cast<uint32_t>(u) ^ (lane & 7u)) * 16u), __float_as_uint(v[4 * u]),
                 __float_as_uint(v[4 * u + 1]), __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
  __syncwarp();
  if (cols >= 32 && ((reinterpret_cast<uintptr_t>(c) | static_cast<uintptr_t>(ldc * 4)) & 15u) == 0) {
    const uint32_t unit = lane & 7u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t r = static_cast<uint32_t>(i) * 4u + (lane >> 3);
      float4 w = *reinterpret_cast<const float4*>(stage + r * 128u + ((unit ^ (r & 7u)) * 16u));
      float4* p = reinterpret_cast<float4*>(c + static_cast<int64_t>(r) * ldc + unit * 4u);
      if (static_cast<int>(r) < rows) {
        if (add) {
          const float4 o = *p;
          w = make_float4(o.x + w.x, o.y + w.y, o.z + w.z, o.w + w.w);
        }
        *p = w;
      }
    }
  } else {
    const bool mine = static_cast<int>(lane) < cols;
    float* p = c + lane;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      const uint32_t unit = (lane >> 2) ^ (static_cast<uint32_t>(r) & 7u);
      const float w = *reinterpret_cast<const float*>(stage + r * 128 + unit * 16u + (lane & 3u) * 4u);
      if (mine && r < rows) *p = add ? *p + w : w;
      p += ldc;
    }
  }
  __syncwarp();
}

// 32 fp32 values a lane as C's element type.
__device__ __forceinline__ void store_block(const FfArgs& a, int row0, int col0, const float (&v)[32], uint8_t* stage) {
  const int64_t at = static_cast<int64_t>(row0) * a.ldc + col0;
  if (a.out_kind == kOutF32) {
    store_block32(static_cast<float*>(a.c) + at, a.ldc, a.m - row0, a.n - col0, v, a.accumulate != 0, stage);
    return;
  }
  uint32_t p[16];
  if (a.out_kind == kOutBf16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) p[j] = pack16<true>(v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) p[j] = pack16<false>(v[2 * j], v[2 * j + 1]);
  }
  store_block16(static_cast<uint16_t*>(a.c) + at, a.ldc, a.m - row0, a.n - col0, p, stage);
}

}  // namespace ff
}  // namespace gemm_tn_dev

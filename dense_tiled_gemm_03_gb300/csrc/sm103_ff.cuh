// sm103_ff.cuh -- what the feed-forward kernels share: bounded waits, the
// activations, the 8-bit tensor-core instruction and the row stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ff_internal.h"
#include "sm103_cache_ptx.cuh"   // elect_one
#include "sm103_ptx.cuh"

namespace gemm_tn_dev {
namespace ff {

constexpr int kStatusExpired = 6;   // == GEMM_TN_ERR_TIMEOUT
constexpr int kRelu = 1, kGelu = 2, kSilu = 3;
constexpr int kOutF16 = 0, kOutBf16 = 1, kOutF32 = 2;

// Bounded waits: past the deadline the kernel records the error, tells every
// role of the cluster to stop, and returns. They acquire at CTA scope: what the
// barriers guard is in shared and tensor memory (an acquire at cluster scope
// also gives up the SM's cached lines, at every block).
template <int kClusterSize>
struct Waiter {
  int* status;
  uint64_t timeout_ns;
  volatile uint32_t* abort_flag;
  static constexpr bool kCluster = kClusterSize > 1;

  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait<false>(bar, parity)) return true;
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
    while (true) {
      if (mbar_try_wait<false>(bar, parity)) return true;
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

  // The same for a whole warp, with one outcome.
  __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(bar, parity));
  }

  // For what is in flight once another role has given up: never sets the flag.
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
    const uint64_t deadline = globaltimer_ns() + timeout_ns;
    while (!mbar_try_wait<false>(bar, parity))
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

// Arrive on a barrier of any CTA of the cluster to hand back tensor memory: what
// it orders is this thread's tcgen05 loads (complete, and fenced before it), no
// data in memory. A release at cluster scope would wait for the warp's loads and
// stores in flight each time: measured at a block of 128 a time, e4m3 4096^3
// took 232 us with it.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}

// ------------------------------------------------------------------ warps that issue as a whole
// Every lane of the producer and MMA warps runs the same code with the same
// operands, and the one lane with leader != 0 (elect_one) issues: the operands
// of tcgen05 and TMA instructions are uniform registers, and where one lane runs
// alone each is moved there for every instruction. An e4m3 block of 128 lasts
// 545 clocks on the tensor core; issued by single threads it took some 700.

// D[tmem] (+)= A[smem] x B[smem]^T: fp16/bf16 (16 elements of K), or e4m3 (32),
// whose instruction descriptor is that of kind::f16 with the formats' fields zero.
template <int kCtaGroup, bool kF8>
__device__ __forceinline__ void mma_warp(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
#define FF_MMA(GROUP, KIND)                                                                                       \
  asm volatile(                                                                                                   \
      "{\n\t.reg .pred p, q;\n\t"                                                                                 \
      "setp.ne.b32 p, %4, 0;\n\t"                                                                                 \
      "setp.ne.b32 q, %5, 0;\n\t"                                                                                 \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}"                              \
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader) : "memory")
  if constexpr (kCtaGroup == 1 && kF8) {
    FF_MMA("1", "f8f6f4");
  } else if constexpr (kCtaGroup == 1) {
    FF_MMA("1", "f16");
  } else if constexpr (kF8) {
    FF_MMA("2", "f8f6f4");
  } else {
    FF_MMA("2", "f16");
  }
#undef FF_MMA
}

// Arrive on `bar` (kCtaGroup 2: at its offset in every CTA of the mask) when
// what the leader issued so far has completed.
template <int kCtaGroup>
__device__ __forceinline__ void commit_warp(uint32_t leader, uint32_t bar, uint16_t mask) {
  if constexpr (kCtaGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        :: "r"(bar), "r"(leader) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        :: "r"(bar), "h"(mask), "r"(leader) : "memory");
  }
}

// 2-D tile load; kCtaGroup 2: the barrier may be the pair's other CTA's.
template <int kCtaGroup>
__device__ __forceinline__ void load_warp(uint32_t leader, const void* tmap, uint32_t dst, uint32_t bar, int32_t x, int32_t y) {
  if constexpr (kCtaGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"(leader) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"(leader) : "memory");
  }
}

// The same with an L2 cache policy.
__device__ __forceinline__ void load_warp_hint(uint32_t leader, const void* tmap, uint32_t dst, uint32_t bar, int32_t x,
                                               int32_t y, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;\n\t}"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "l"(policy), "r"(leader) : "memory");
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

// ------------------------------------------------------------------ asynchronous copies of single values

__device__ __forceinline__ void cp_async_4(void* to_shared, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_addr(to_shared)), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the newest N groups of this thread have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// ------------------------------------------------------------------ activations
// silu: g s with s = 1 / (1 + e^-g), taken below zero as e^g / (1 + e^g) so that
// nothing overflows and it keeps its relative accuracy; slope s + g s (1 - s).
// gelu: g P with P = erfc(-g / sqrt 2) / 2, the normal distribution's lower
// tail taken directly so that it keeps its relative accuracy far below zero;
// slope P + g e^(-g^2 / 2) / sqrt(2 pi). erfc by the Chebyshev fit of Press,
// Teukolsky, Vetterling and Flannery, Numerical Recipes, section 6.2 (erfcc):
// erfc(z) = t e^(-z^2 + p(t)), t = 1 / (1 + z / 2), z >= 0, to 1.2e-7 of the
// value; e^(-z^2) is the slope's too. (With CUDA's erfcf and expf the gradient of
// 8192 x 8192 took 148 us instead of 107.)
// relu: max(g, 0) (NaN stays NaN); slope 1 above zero, else 0.
//
// s and P are off by at most 2^-20 of their value, and where e^-|g| (silu) or
// e^(-g^2 / 2) (gelu) is below 2^-126 by its steps of 2^-149. The product's silu
// takes e^-|g| without the correction: |g| 2^-23 of the value, no more than what
// g's own rounding as an fp32 sum makes of it (fp16, 1111 tokens, 2048 to 2 x 5003, replayed:
// 32.0 us, with the correction 33.8; with 1 / (1 + e^-g), which is zero below -87, 31.6).

// 2^x by the multi-function unit, results below the normal numbers among them.
__device__ __forceinline__ float exp2_any(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^-(a + a_low), 0 <= a <= 128 (where it is zero) and a_low within a's last place:
// the square of 2^x, x half of -a in base 2, times what the roundings of a's product
// and of log2(e) leave out, which an exponent of -100 would make 2^-17 of the result.
__device__ __forceinline__ float exp_minus(float a, float a_low) {
  constexpr float kC = -0.72134752044448170f, kLow = -9.6298150e-9f;   // -log2(e) / 2
  const float x = kC * a, x_low = fmaf(kLow, a, fmaf(kC, a, -x));
  const float h = ex2_approx(x);
  return h * fmaf(h, fmaf(x_low, 2.0f * 0.69314718055994531f, -a_low), h);
}
__device__ __forceinline__ float sigmoid_from(float g, float e) {   // e = e^-|g|
  return __fdividef(g < 0.0f ? e : 1.0f, 1.0f + e);
}
// P(g), and e^(-g^2 / 2) in `e`.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  const float z = fminf(fabsf(g), 16.0f), half = 0.5f * z, a = half * z;
  e = exp_minus(a, fmaf(half, z, -a));
  const float t = __fdividef(1.0f, fmaf(0.35355339059327376f, fabsf(g), 1.0f));   // z / 2 = |g| / (2 sqrt 2)
  float p = fmaf(t, 0.17087277f, -0.82215223f);
  p = fmaf(t, p, 1.48851587f);
  p = fmaf(t, p, -1.13520398f);
  p = fmaf(t, p, 0.27886807f);
  p = fmaf(t, p, -0.18628806f);
  p = fmaf(t, p, 0.09678418f);
  p = fmaf(t, p, 0.37409196f);
  p = fmaf(t, p, 1.00002368f);
  p = fmaf(t, p, -1.26551223f);
  const float lower = 0.5f * t * e * ex2_approx(p * 1.44269504088896341f);   // P(-|g|)
  return g < 0.0f ? lower : 1.0f - lower;
}

// The activation of an fp32 sum.
template <int kAct>
__device__ __forceinline__ float act(float g) {
  if constexpr (kAct == kSilu) {
    return g * sigmoid_from(g, exp2_any(-1.44269504088896341f * fabsf(g)));
  } else if constexpr (kAct == kGelu) {
    float e;
    return g * normal_cdf(g, e);
  } else {
    return g < 0.0f ? 0.0f : g;
  }
}

// The activation and its slope, of a 16-bit value.
template <int kAct>
__device__ __forceinline__ float2 act_slope(float g) {
  if constexpr (kAct == kSilu) {
    const float s = sigmoid_from(g, exp_minus(fminf(fabsf(g), 128.0f), 0.0f));
    return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
  } else if constexpr (kAct == kGelu) {
    float e;
    const float p = normal_cdf(g, e);
    return make_float2(g * p, fmaf(g * 0.39894228040143268f, e, p));
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

// ------------------------------------------------------------------ a warp's rows of C
// 64 bytes of each of 32 rows: lane l holds row l's, 16 words. They go through
// the warp's 2 KiB of staging so that each store writes whole stretches of rows:
// 16 bytes a lane where the rows are aligned so, else one element a lane along
// the rows. rows, cols: how many of the 32 rows and 64 / kSize columns exist
// (<= 0: none). add (4-byte elements): to what is there.
constexpr uint32_t kStagingBytes = 2048;

template <int kSize>
__device__ __forceinline__ void store_rows(void* to, int64_t ldc, int rows, int cols, const uint32_t (&v)[16], bool add,
                                           uint8_t* stage) {
  constexpr int kCols = 64 / kSize;
  const uint32_t lane = lane_id();
  const uint32_t s = smem_addr(stage);
  // 16-byte unit u of row r lies at u ^ ((r >> 1) & 3): all banks in every access
#pragma unroll
  for (uint32_t u = 0; u < 4; ++u)
    st_shared_v4(s + lane * 64u + ((u ^ ((lane >> 1) & 3u)) * 16u), v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
  __syncwarp();
  uint8_t* c = static_cast<uint8_t*>(to);
  const int64_t pitch = ldc * kSize;
  if (cols >= kCols && ((reinterpret_cast<uintptr_t>(c) | static_cast<uintptr_t>(pitch)) & 15u) == 0) {
    const uint32_t unit = lane & 3u;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t r = i * 8u + (lane >> 2);
      uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64u + ((unit ^ ((r >> 1) & 3u)) * 16u));
      if (static_cast<int>(r) >= rows) continue;
      uint4* p = reinterpret_cast<uint4*>(c + r * pitch) + unit;
      if (kSize == 4 && add) {
        const uint4 o = *p;
        w.x = __float_as_uint(__uint_as_float(o.x) + __uint_as_float(w.x));
        w.y = __float_as_uint(__uint_as_float(o.y) + __uint_as_float(w.y));
        w.z = __float_as_uint(__uint_as_float(o.z) + __uint_as_float(w.z));
        w.w = __float_as_uint(__uint_as_float(o.w) + __uint_as_float(w.w));
      }
      *p = w;
    }
  } else {
    constexpr uint32_t kPer = 16 / kSize;      // elements of a unit
    constexpr int kStep = 32 / kCols;          // rows an access covers: 1, or 2 (fp32)
    const uint32_t col = lane % kCols, sub = lane / kCols;
    const bool mine = static_cast<int>(col) < cols;
    uint8_t* p = c + static_cast<int64_t>(sub) * pitch + col * kSize;
#pragma unroll 8
    for (int i = 0; i < 32; i += kStep) {
      const uint32_t r = static_cast<uint32_t>(i) + sub;
      const uint8_t* from = stage + r * 64u + (((col / kPer) ^ ((r >> 1) & 3u)) * 16u) + (col % kPer) * kSize;
      if (mine && static_cast<int>(r) < rows) {
        if constexpr (kSize == 2) {
          *reinterpret_cast<uint16_t*>(p) = *reinterpret_cast<const uint16_t*>(from);
        } else {
          const float w = *reinterpret_cast<const float*>(from);
          float* q = reinterpret_cast<float*>(p);
          *q = add ? *q + w : w;
        }
      }
      p += kStep * pitch;
    }
  }
  __syncwarp();
}

// 32 fp32 values a lane, from column col0 of row row0 + lane, as C's element type.
__device__ __forceinline__ void store_block(const FfArgs& a, int row0, int col0, const float (&v)[32], uint8_t* stage,
                                            int64_t offset = 0) {
  const int64_t at = static_cast<int64_t>(row0) * a.ldc + col0 + offset;
  uint32_t w[16];
  if (a.out_kind == kOutF32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[16 * h + j]);
      store_rows<4>(static_cast<float*>(a.c) + at + 16 * h, a.ldc, a.m - row0, a.n - col0 - 16 * h, w, a.accumulate != 0,
                    stage);
    }
    return;
  }
  if (a.out_kind == kOutBf16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack16<true>(v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack16<false>(v[2 * j], v[2 * j + 1]);
  }
  store_rows<2>(static_cast<uint16_t*>(a.c) + at, a.ldc, a.m - row0, a.n - col0, w, false, stage);
}

}  // namespace ff
}  // namespace gemm_tn_dev

// sm103_ff_skinny.cu -- the feed-forward products for few rows of A (decoded
// tokens): the gated projection and the e4m3 product, bound by reading B once.
//
// The roles swap: 128 rows of B are the MMA's M side and A's rows (zero-filled
// past m) its N side, so that a CTA streams B through its ring and an
// accumulator lane holds one column of C. For the gated projection the 128 rows
// are 64 of the gate and the same 64 of the other projection. K is cut over a
// cluster of S CTAs, whose fp32 partials are added in CTA order through
// distributed shared memory.
//
// A CTA takes half of an SM's shared memory, so that one's last loads and its
// join overlap another's stream; S is the least that gives the device two CTAs
// an SM (ff_api.cu).
#include <atomic>

#include "sm103_ff.cuh"

namespace gemm_tn_dev {
namespace ff {
namespace skinny {

constexpr int kThreads = 192;   // warp 0 loads, warp 1 multiplies, warps 2 to 5 are the epilogue
constexpr uint32_t kStageB = 128 * 128;
constexpr uint32_t kRingBudget = 100 * 1024;

// kN: rows of A (MMA N); kGatedForm: gated 16-bit, else e4m3 with block scales.
template <int kN_, int kSplits_, bool kGatedForm_, bool kBf16_>
struct Cfg {
  static constexpr int kN = kN_, kSplits = kSplits_;
  static constexpr bool kGatedForm = kGatedForm_, kBf16 = kBf16_, kScaled = !kGatedForm_;
  static constexpr int kBlockK = kScaled ? 128 : 64;
  static constexpr uint32_t kStageA = kN * 128;
  static constexpr int kStages = static_cast<int>(kRingBudget / (kStageB + kStageA));
  static constexpr int kBuffers = kScaled ? 2 : 1;
  static constexpr uint32_t kTmemCols = kBuffers * kN < 32 ? 32 : kBuffers * kN;
  static constexpr int kPartStride = kN + 4;   // floats between the partial's rows (columns of C)
  static constexpr uint32_t kOffB = 0;
  static constexpr uint32_t kOffA = kOffB + kStages * kStageB;
  static constexpr uint32_t kRingEnd = kOffA + kStages * kStageA;
  static constexpr uint32_t kOffScale = kRingEnd;   // e4m3: [4 warps][2][kN] scales of A's rows
  static constexpr uint32_t kOffBar = kOffScale + (kScaled ? 4 * 2 * kN * 4 : 0);
  static constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 1;
  static constexpr uint32_t kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
  static constexpr uint32_t kSmemBytes = kOffAbort + 4 + 1024;
  static constexpr uint32_t kIdesc = mma_idesc_f16(!kScaled && kBf16, 128, kN);
  static constexpr int kOutN = kGatedForm ? 64 : 128;   // columns of C
  static_assert(kN == 16 || kN == 32 || kN == 64 || kN == 128, "rows of A");
  static_assert(kStageA % 1024 == 0, "swizzle atoms stay 1024-aligned");
  static_assert(128 * kPartStride * 4 <= kRingEnd, "the partial fits in the idle ring");
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs to an SM");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 2) ff_skinny_kernel(const __grid_constant__ FfArgs args) {
  constexpr int S = C::kSplits;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t base = smem_addr(smem);
  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
  const int tn = static_cast<int>(blockIdx.x) / S;
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * args.num_k_blocks / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * args.num_k_blocks / S);

  auto a_tile = [&](int s) { return base + C::kOffA + s * C::kStageA; };
  auto b_tile = [&](int s) { return base + C::kOffB + s * kStageB; };
  auto full_bar = [&](int s) { return base + C::kOffBar + 8u * s; };
  auto empty_bar = [&](int s) { return base + C::kOffBar + 8u * (C::kStages + s); };
  auto sum_full = [&](int b) { return base + C::kOffBar + 8u * (2 * C::kStages + b); };
  auto sum_empty = [&](int b) { return base + C::kOffBar + 8u * (2 * C::kStages + C::kBuffers + b); };
  const uint32_t drain_bar = base + C::kOffBar + 8u * (2 * C::kStages + 2 * C::kBuffers);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < C::kBuffers; ++b) {
      mbar_init(sum_full(b), 1);
      mbar_init(sum_empty(b), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_descriptor(&args.tmap_a);
    tma_prefetch_descriptor(&args.tmap_b);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  // the peers' memory is touched in the join alone: their start is waited for there
  if constexpr (S > 1) cluster_arrive_relaxed();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  const Waiter<1> wd{args.status, args.timeout_ns, abort_flag};

  if (warp == 0) {
    // -------------------------------------------------------------- TMA producer (the whole warp, one lane issues)
    const uint32_t elected = elect_one();
    const uint64_t once = l2_policy_evict_first();
    int stage = 0;
    uint32_t phase = 0;
    Issued issued;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!wd.warp_wait(empty_bar(stage), phase ^ 1u)) break;
      const uint32_t bar = full_bar(stage);
      if (elected != 0) mbar_arrive_expect_tx(bar, kStageB + C::kStageA);
      __syncwarp();
      if (kb - kb0 != args.drop_load_kb) {
        const int k0 = kb * C::kBlockK;
        if constexpr (C::kGatedForm) {
          load_warp_hint(elected, &args.tmap_b, b_tile(stage), bar, k0, tn * 64, once);
          load_warp_hint(elected, &args.tmap_b, b_tile(stage) + kStageB / 2, bar, k0, tn * 64 + args.n, once);
        } else {
          load_warp_hint(elected, &args.tmap_b, b_tile(stage), bar, k0, tn * 128, once);
        }
        load_warp<1>(elected, &args.tmap_a, a_tile(stage), bar, k0, 0);
      }
      issued.record(stage, phase);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    for (int s = 0; s < C::kStages; ++s)
      if ((issued.issued >> s) & 1u) wd.drain(full_bar(s), (issued.parity >> s) & 1u);
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer: D[j][i] += B[j] A[i]
    const uint32_t elected = elect_one();
    int stage = 0, buf = 0;
    uint32_t phase = 0, buf_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (C::kScaled && !wd.warp_wait(sum_empty(buf), buf_phase ^ 1u)) break;
      if (!wd.warp_wait(full_bar(stage), phase)) break;
      tc_fence_after_sync();
      const uint32_t d = tmem_base + static_cast<uint32_t>(buf * C::kN);
      const uint64_t a_desc = sw128_kmajor_desc(a_tile(stage)), b_desc = sw128_kmajor_desc(b_tile(stage));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_warp<1, C::kScaled>(elected, d, b_desc + 2u * kk, a_desc + 2u * kk, C::kIdesc,
                                kk > 0 || (!C::kScaled && kb > kb0) ? 1u : 0u);
      commit_warp<1>(elected, empty_bar(stage), 0);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
      if (C::kScaled || kb == kb1 - 1) {
        commit_warp<1>(elected, sum_full(buf), 0);
        if (++buf == C::kBuffers) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
    }
    commit_warp<1>(elected, drain_bar, 0);
    wd.drain(drain_bar, 0);
  } else {
    // -------------------------------------------------------------- a lane's sums -> own shared memory
    const uint32_t quarter = warp & 3u;
    const uint32_t row = quarter * 32u + lane;   // of the 128 rows of B
    const uint32_t t_row = tmem_base + ((quarter * 32u) << 16);
    const uint32_t part = base + row * C::kPartStride * 4u;
    bool ok = true;
    if constexpr (C::kScaled) {
      const int col = tn * 128 + static_cast<int>(row);   // of C
      const float* sb = args.b_scale + static_cast<int64_t>(min(col, args.n - 1) / (args.b_block_rows)) * args.bs_row;
      float* vec = reinterpret_cast<float*>(smem + C::kOffScale) + quarter * (2 * C::kN);
      constexpr int kPer = (C::kN + 31) / 32;
      // the scales of a block are loaded a block ahead
      float a_next[kPer], b_next = 0.0f;
      auto load = [&](int kb) {
        b_next = __ldg(sb + kb * args.bs_blk);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          a_next[i] = __ldg(args.a_scale + static_cast<int64_t>(min(i * 32 + static_cast<int>(lane), args.m - 1)) *
                                               args.as_row + kb * args.as_blk);
      };
      uint64_t sum[C::kN / 2];
#pragma unroll
      for (int j = 0; j < C::kN / 2; ++j) sum[j] = 0;
      if (kb0 < kb1) load(kb0);
      int buf = 0;
      uint32_t buf_phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        float* now = vec + (kb & 1) * C::kN;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (C::kN >= 32 || lane < static_cast<uint32_t>(C::kN)) now[i * 32 + lane] = a_next[i];
        __syncwarp();
        const uint64_t b2 = f32x2_pack(b_next, b_next);
        if (kb + 1 < kb1) load(kb + 1);
        if (!__all_sync(0xffffffffu, wd.wait(sum_full(buf), buf_phase))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < C::kN / 16; ++c) {
          uint32_t v[16];
          tmem_load_32x16(t_row + static_cast<uint32_t>(buf * C::kN + c * 16), v);
          tmem_loaded(v);
          if (c == C::kN / 16 - 1) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(sum_empty(buf));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint64_t a2 = *reinterpret_cast<const uint64_t*>(now + c * 16 + 2 * j);
            const uint64_t p = f32x2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            sum[c * 8 + j] = f32x2_fma(f32x2_mul(p, a2), b2, sum[c * 8 + j]);
          }
        }
        if (++buf == C::kBuffers) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      // the ring is idle once the last block has been multiplied
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ok) {
#pragma unroll
        for (int j = 0; j < C::kN / 4; ++j) {
          float f0, f1, f2, f3;
          f32x2_unpack(sum[2 * j], f0, f1);
          f32x2_unpack(sum[2 * j + 1], f2, f3);
          st_shared_v4(part + 16u * j, __float_as_uint(f0), __float_as_uint(f1), __float_as_uint(f2),
                       __float_as_uint(f3));
        }
      }
    } else if (kb0 < kb1) {
      ok = __all_sync(0xffffffffu, wd.wait(sum_full(0), 0));
      if (ok) {
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < C::kN / 16; ++c) {
          uint32_t v[16];
          tmem_load_32x16(t_row + static_cast<uint32_t>(c * 16), v);
          tmem_loaded(v);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_v4(part + 64u * c + 16u * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
    }
  }
  __syncwarp();

  // ---------------------------------------------------------------- the cluster's partials, added in CTA order
  tc_fence_before_sync();
  if constexpr (S > 1) {
    cluster_wait();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  {
    constexpr int kCols = C::kOutN / S;   // columns of C that this CTA finishes
    const int c0 = static_cast<int>(rank) * kCols;
    auto total = [&](int r, int i) {
      const uint32_t off = base + static_cast<uint32_t>(r * C::kPartStride + i) * 4u;
      float v[S];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if constexpr (S > 1) {
          v[s] = ld_cluster_f32(map_to_cta(off, static_cast<uint32_t>(s)));
        } else {
          v[s] = *reinterpret_cast<const float*>(smem + (off - base));
        }
      }
      float t = v[0];
#pragma unroll
      for (int s = 1; s < S; ++s) t += v[s];
      return t;
    };
    const int rows = min(args.m, C::kN);
    for (int x = threadIdx.x; x < kCols * rows; x += kThreads) {   // consecutive threads: consecutive columns of C
      const int r = c0 + x % kCols, i = x / kCols;
      const int col = tn * C::kOutN + r;
      if (col >= args.n) continue;
      const int64_t at = static_cast<int64_t>(i) * args.ldc + col;
      if constexpr (C::kGatedForm) {
        const float g = total(r, i), u = total(r + 64, i);
        const float h = (args.activation == kSilu ? act<kSilu>(g) : args.activation == kGelu ? act<kGelu>(g)
                                                                                             : act<kRelu>(g)) * u;
        static_cast<uint16_t*>(args.c)[at] = static_cast<uint16_t>(pack16<C::kBf16>(h, 0.0f));
        if (args.pre != nullptr) {
          uint16_t* pre = static_cast<uint16_t*>(args.pre) + static_cast<int64_t>(i) * args.ldp + col;
          pre[0] = static_cast<uint16_t>(pack16<C::kBf16>(g, 0.0f));
          pre[args.n] = static_cast<uint16_t>(pack16<C::kBf16>(u, 0.0f));
        }
      } else {
        const float v = total(r, i);
        if (args.out_kind == kOutF32) {
          float* c = static_cast<float*>(args.c) + at;
          *c = args.accumulate ? *c + v : v;
        } else {
          static_cast<uint16_t*>(args.c)[at] = static_cast<uint16_t>(
              args.out_kind == kOutBf16 ? pack16<true>(v, 0.0f) : pack16<false>(v, 0.0f));
        }
      }
    }
  }
  if constexpr (S > 1) cluster_sync_all();   // peers may still be reading this CTA's partial
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem_base, C::kTmemCols);
  }
}

}  // namespace skinny
}  // namespace ff
}  // namespace gemm_tn_dev

namespace gemm_tn_impl {
namespace {

using namespace gemm_tn_dev::ff::skinny;

template <class C>
cudaError_t launch_one(const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(ff_skinny_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmemBytes));
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (C::kSplits > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = C::kSplits;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (dependent_launch_enabled()) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, ff_skinny_kernel<C>, args);
}

template <int kN, bool kGatedForm, bool kBf16>
cudaError_t launch_splits(int splits, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  switch (splits) {
    case 1: return launch_one<Cfg<kN, 1, kGatedForm, kBf16>>(args, grid, stream);
    case 2: return launch_one<Cfg<kN, 2, kGatedForm, kBf16>>(args, grid, stream);
    case 4: return launch_one<Cfg<kN, 4, kGatedForm, kBf16>>(args, grid, stream);
    case 8: return launch_one<Cfg<kN, 8, kGatedForm, kBf16>>(args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <bool kGatedForm, bool kBf16>
cudaError_t launch_rows(int rows, int splits, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  switch (rows) {
    case 16: return launch_splits<16, kGatedForm, kBf16>(splits, args, grid, stream);
    case 32: return launch_splits<32, kGatedForm, kBf16>(splits, args, grid, stream);
    case 64: return launch_splits<64, kGatedForm, kBf16>(splits, args, grid, stream);
    case 128: return launch_splits<128, kGatedForm, kBf16>(splits, args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_ff_skinny(int kind, bool bf16, int rows, int splits, const gemm_tn_dev::FfArgs& args, int grid,
                             cudaStream_t stream) {
  if (kind != kFfGated) return launch_rows<false, false>(rows, splits, args, grid, stream);
  return bf16 ? launch_rows<true, true>(rows, splits, args, grid, stream)
              : launch_rows<true, false>(rows, splits, args, grid, stream);
}

}  // namespace gemm_tn_impl

// sm103_ff_skinny.cu -- the feed-forward products for few rows of A (decoded
// tokens): the gated projection and the e4m3 product, bound by reading B once.
//
// The roles swap: 128 rows of B are the MMA's M side and A's rows (zero-filled
// past m; 128 at most to a tile) its N side, so that a CTA streams B through its ring and an
// accumulator lane holds one column of C. For the gated projection the 128 rows
// are 64 of the gate and the same 64 of the other projection. K is cut over a
// cluster of S CTAs, whose fp32 partials are added in CTA order through
// distributed shared memory.
//
// S is the most for which all clusters run at once (ff_api.cu), a CTA to an SM:
// what a CTA streams is bound by its loads in flight, so it takes all of the SM's
// shared memory. With more tiles than SMs two CTAs share one, and the last
// loads and the join of one overlap the other's stream.
//
// Bound by memory: bf16, one token, 4096 to 2 x 16384: 40.3 us, 6.7 TB/s (whole
// tiles 73); e4m3, 8 tokens, 8192 to 16384: 23.4 us, 5.7 TB/s, of which about 3 are
// the start and the end. Small ones by latency: fp16, 24 tokens, 1000 to 2 x 2049: 5.4 us.
#include <atomic>

#include "sm103_ff.cuh"

namespace gemm_tn_dev {
namespace ff {
namespace skinny {

constexpr int kThreads = 192;   // warp 0 loads, warp 1 multiplies, warps 2 to 5 are the epilogue
constexpr uint32_t kStageB = 128 * 128;

// kN: rows of A (MMA N); kGatedForm: gated 16-bit, else e4m3 with block scales;
// kPerSm: CTAs that share an SM.
template <int kN_, int kSplits_, int kPerSm_, bool kGatedForm_, bool kBf16_>
struct Cfg {
  static constexpr int kPerSm = kPerSm_;
  static constexpr uint32_t kRingBudget = kPerSm == 2 ? 100 * 1024 : 200 * 1024;
  static constexpr int kN = kN_, kSplits = kSplits_;
  static constexpr bool kGatedForm = kGatedForm_, kBf16 = kBf16_, kScaled = !kGatedForm_;
  static constexpr int kBlockK = kScaled ? 128 : 64;
  static constexpr uint32_t kStageA = kN * 128;
  static constexpr int kStages = static_cast<int>(kRingBudget / (kStageB + kStageA));
  static constexpr int kBuffers = kScaled ? 4 / kPerSm : 1;   // (of 512 columns to an SM)
  static constexpr uint32_t kTmemCols = kBuffers * kN < 32 ? 32 : kBuffers * kN;
  static constexpr int kPartStride = kN + 4;   // floats between the partial's rows (columns of C)
  static constexpr uint32_t kOffB = 0;
  static constexpr uint32_t kOffA = kOffB + kStages * kStageB;
  static constexpr uint32_t kRingEnd = kOffA + kStages * kStageA;
  // e4m3: each epilogue warp's ring of scales, of kAhead blocks: A's rows', then its own rows of B
  static constexpr int kAhead = 8;
  static constexpr int kScaleFloats = kN + 32;
  static constexpr uint32_t kOffScale = kRingEnd;
  static constexpr uint32_t kOffBar = kOffScale + (kScaled ? 4 * kAhead * kScaleFloats * 4 : 0);
  static constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 1;
  static constexpr uint32_t kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr uint32_t kOffAbort = kOffTmemSlot + 4;
  static constexpr uint32_t kSmemBytes = kOffAbort + 4 + 1024;
  static constexpr uint32_t kIdesc = mma_idesc_f16(!kScaled && kBf16, 128, kN);
  static constexpr int kOutN = kGatedForm ? 64 : 128;   // columns of C
  static_assert(kN == 16 || kN == 32 || kN == 64 || kN == 128, "rows of A");
  static_assert(kStageA % 1024 == 0, "swizzle atoms stay 1024-aligned");
  static_assert(128 * kPartStride * 4 <= kRingEnd, "the partial fits in the idle ring");
  static_assert(kStages <= 32, "issued phases fit a 32-bit mask");
  static_assert(kPerSm * (kSmemBytes + 1024) <= 228 * 1024, "kPerSm CTAs to an SM");
};

template <class C>
__global__ void __launch_bounds__(kThreads, C::kPerSm) ff_skinny_kernel(const __grid_constant__ FfArgs args) {
  constexpr int S = C::kSplits;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t base = smem_addr(smem);
  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
  const int tile = static_cast<int>(blockIdx.x) / S, tm = tile / args.num_n_tiles, tn = tile - tm * args.num_n_tiles;
  const int row0 = tm * C::kN;   // of A and C
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
  if (args.alone == 0) griddep_launch_dependents();
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
        load_warp<1>(elected, &args.tmap_a, a_tile(stage), bar, k0, row0);
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
      const float* sb = args.b_scale + static_cast<int64_t>(min(col, args.n - 1) / args.b_block_rows) * args.bs_row;
      float* ring = reinterpret_cast<float*>(smem + C::kOffScale) + quarter * (C::kAhead * C::kScaleFloats);
      // the scales' copies run kAhead - 1 blocks ahead: a block lasts less than a load
      auto fetch = [&](int kb) {
        if (kb < kb1) {
          float* to = ring + (kb & (C::kAhead - 1)) * C::kScaleFloats;
#pragma unroll
          for (int i = 0; i < C::kN; i += 32)
            if (C::kN >= 32 || lane < static_cast<uint32_t>(C::kN))
              cp_async_4(to + i + lane, args.a_scale + static_cast<int64_t>(min(row0 + i + static_cast<int>(lane), args.m - 1)) *
                                                           args.as_row + kb * args.as_blk);
          cp_async_4(to + C::kN + lane, sb + kb * args.bs_blk);
        }
        cp_async_commit();
      };
      uint64_t sum[C::kN / 2];
#pragma unroll
      for (int j = 0; j < C::kN / 2; ++j) sum[j] = 0;
      for (int i = 0; i < C::kAhead - 1; ++i) fetch(kb0 + i);
      int buf = 0;
      uint32_t buf_phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        __syncwarp();   // the slot's last readers are done with it
        fetch(kb + C::kAhead - 1);
        cp_async_wait<C::kAhead - 1>();
        __syncwarp();
        const float* now = ring + (kb & (C::kAhead - 1)) * C::kScaleFloats;
        const uint64_t b2 = f32x2_pack(now[C::kN + lane], now[C::kN + lane]);
        if (!wd.warp_wait(sum_full(buf), buf_phase)) {
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
          for (int j = 0; j < 8; j += 2) {
            const ulonglong2 a2 = *reinterpret_cast<const ulonglong2*>(now + c * 16 + 2 * j);
            const uint64_t p0 = f32x2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            const uint64_t p1 = f32x2_pack(__uint_as_float(v[2 * j + 2]), __uint_as_float(v[2 * j + 3]));
            // (the scales' product first, as in whole tiles: a large one and a small one may meet)
            sum[c * 8 + j] = f32x2_fma(p0, f32x2_mul(a2.x, b2), sum[c * 8 + j]);
            sum[c * 8 + j + 1] = f32x2_fma(p1, f32x2_mul(a2.y, b2), sum[c * 8 + j + 1]);
          }
        }
        if (++buf == C::kBuffers) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      cp_async_wait<0>();
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
    auto total = [&](int r, int i) {      // of row r of the partials, rows i to i + 3 of A
      const uint32_t off = static_cast<uint32_t>(r * C::kPartStride + i) * 4u;
      float4 v[S];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if constexpr (S > 1) {
          v[s] = ld_cluster_f4(map_to_cta(base + off, static_cast<uint32_t>(s)));
        } else {
          v[s] = *reinterpret_cast<const float4*>(smem + off);
        }
      }
#pragma unroll
      for (int s = 1; s < S; ++s) {
        v[0].x += v[s].x;
        v[0].y += v[s].y;
        v[0].z += v[s].z;
        v[0].w += v[s].w;
      }
      return v[0];
    };
    const int rows = min(args.m - row0, C::kN);
    // consecutive threads: consecutive columns of C, four rows each
    for (int x = threadIdx.x; x < kCols * ((rows + 3) / 4); x += kThreads) {
      const int r = c0 + x % kCols, i0 = x / kCols * 4;
      const int col = tn * C::kOutN + r;
      if (col >= args.n) continue;
      const float4 t = total(r, i0);
      const float v[4] = {t.x, t.y, t.z, t.w};
      if constexpr (C::kGatedForm) {
        const float4 t2 = total(r + 64, i0);
        const float u[4] = {t2.x, t2.y, t2.z, t2.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i0 + j >= rows) continue;
          const float g = v[j];
          const float h = (args.activation == kSilu ? act<kSilu>(g) : args.activation == kGelu ? act<kGelu>(g)
                                                                                               : act<kRelu>(g)) * u[j];
          static_cast<uint16_t*>(args.c)[static_cast<int64_t>(row0 + i0 + j) * args.ldc + col] =
              static_cast<uint16_t>(pack16<C::kBf16>(h, 0.0f));
          if (args.pre != nullptr) {
            uint16_t* pre = static_cast<uint16_t*>(args.pre) + static_cast<int64_t>(row0 + i0 + j) * args.ldp + col;
            const uint32_t both = pack16<C::kBf16>(g, u[j]);
            pre[0] = static_cast<uint16_t>(both);
            pre[args.n] = static_cast<uint16_t>(both >> 16);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i0 + j >= rows) continue;
          const int64_t at = static_cast<int64_t>(row0 + i0 + j) * args.ldc + col;
          if (args.out_kind == kOutF32) {
            float* c = static_cast<float*>(args.c) + at;
            *c = args.accumulate ? *c + v[j] : v[j];
          } else {
            static_cast<uint16_t*>(args.c)[at] = static_cast<uint16_t>(
                args.out_kind == kOutBf16 ? pack16<true>(v[j], 0.0f) : pack16<false>(v[j], 0.0f));
          }
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
cudaError_t fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int grid, cudaStream_t stream) {
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
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  if (C::kSplits > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = C::kSplits;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  return cudaSuccess;
}

template <class C>
cudaError_t launch_one(const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  const cudaError_t e = fill<C>(cfg, attr, grid, stream);
  if (e != cudaSuccess) return e;
  if (dependent_launch_enabled()) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, ff_skinny_kernel<C>, args);
}

template <int kSplits>
int resident(int sms) {
  using C = Cfg<16, kSplits, 1, true, true>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  int clusters = 0;
  if (fill<C>(cfg, attr, sms - sms % kSplits, nullptr) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&clusters, ff_skinny_kernel<C>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return clusters;
}

// What ff_api.cu asks for (ff_skinny_has).
template <int kN, bool kGatedForm, bool kBf16>
cudaError_t launch_splits(int splits, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  if constexpr (kN <= 32) {
    if (splits == 0) return launch_one<Cfg<kN, 1, 2, kGatedForm, kBf16>>(args, grid, stream);
    if (splits == 1) return launch_one<Cfg<kN, 1, 1, kGatedForm, kBf16>>(args, grid, stream);
  }
  if constexpr (kN <= 64 || kGatedForm) {
    if (splits == 2) return launch_one<Cfg<kN, 2, 1, kGatedForm, kBf16>>(args, grid, stream);
  }
  if (splits == 4) return launch_one<Cfg<kN, 4, 1, kGatedForm, kBf16>>(args, grid, stream);
  if (splits == 8) return launch_one<Cfg<kN, 8, 1, kGatedForm, kBf16>>(args, grid, stream);
  return cudaErrorInvalidValue;
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

int ff_resident_clusters(int splits, int sms) {
  return splits == 2 ? resident<2>(sms) : splits == 4 ? resident<4>(sms) : splits == 8 ? resident<8>(sms) : sms;
}

cudaError_t launch_ff_skinny(int kind, bool bf16, int rows, int splits, const gemm_tn_dev::FfArgs& args, int grid,
                             cudaStream_t stream) {
  if (kind != kFfGated) return launch_rows<false, false>(rows, splits, args, grid, stream);
  return bf16 ? launch_rows<true, true>(rows, splits, args, grid, stream)
              : launch_rows<true, false>(rows, splits, args, grid, stream);
}

}  // namespace gemm_tn_impl

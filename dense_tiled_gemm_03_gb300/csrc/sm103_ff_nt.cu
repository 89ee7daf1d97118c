// sm103_ff_nt.cu -- C = A^T B (sm103_ff_gemm.cuh), a weight's gradient.
//
// bf16, 16384 x 4096 over 8192 tokens: 564 us in a short graph (1950 TFLOP/s),
// 638 at the power limit; the tensor pipe is active 91% of the kernel. What bounds
// a small one (5000 x 1024 over 1000 tokens: 20 us) is the round of tiles begun for
// the last few, and the start and end of the kernel.
#include "sm103_ff_gemm.cuh"

namespace gemm_tn_impl {

using namespace gemm_tn_dev::ff;

template <bool kBf16>
cudaError_t launch_nt(int tile, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  switch (tile) {
    case kFfPair256: return FfLauncher<Tile<kNt, 2, 256, 6, kBf16>>::launch(args, grid, stream);
    case kFfPair128: return FfLauncher<Tile<kNt, 2, 128, 8, kBf16>>::launch(args, grid, stream);
    case kFfSingle128: return FfLauncher<Tile<kNt, 1, 128, 6, kBf16>>::launch(args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_ff_nt(int tile, bool bf16, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  return bf16 ? launch_nt<true>(tile, args, grid, stream) : launch_nt<false>(tile, args, grid, stream);
}

}  // namespace gemm_tn_impl

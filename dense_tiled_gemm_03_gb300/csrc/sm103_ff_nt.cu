// sm103_ff_nt.cu -- instantiations.
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

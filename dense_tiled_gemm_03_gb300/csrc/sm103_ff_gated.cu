// sm103_ff_gated.cu -- the gated projection in whole tiles (sm103_ff_gemm.cuh).
//
// bf16, 8192 tokens, 4096 to 2 x 16384: 1108 to 1133 us a call in a short replayed graph
// with both projections written too (1941 to 1985 TFLOP/s), 1300 in a long row of calls,
// where the board's power limit holds the SM clock at 1.6 GHz; the tensor pipe is
// active 96% of the kernel. fp16, 1111 tokens, 2048 to 2 x 5003: 32 us with the
// operands in L2 and 37 from memory, 200 tiles in three rounds of 76 pairs.
#include "sm103_ff_gemm.cuh"

namespace gemm_tn_impl {

using namespace gemm_tn_dev::ff;

template <bool kBf16>
cudaError_t launch_gated(int tile, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  switch (tile) {
    case kFfPair256: return FfLauncher<Tile<kGated, 2, 256, 6, kBf16>>::launch(args, grid, stream);
    case kFfPair128: return FfLauncher<Tile<kGated, 2, 128, 8, kBf16>>::launch(args, grid, stream);
    case kFfSingle128: return FfLauncher<Tile<kGated, 1, 128, 6, kBf16>>::launch(args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_ff_gated(int tile, bool bf16, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  return bf16 ? launch_gated<true>(tile, args, grid, stream) : launch_gated<false>(tile, args, grid, stream);
}

}  // namespace gemm_tn_impl

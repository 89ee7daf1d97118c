// sm103_ff_e4m3.cu -- the e4m3 product in whole tiles (sm103_ff_gemm.cuh).
//
// 8192^3 to bf16, a scale for 128 x 128 of B: 374 us (2940 TFLOP/s; 417 in a long
// row of calls). The tensor core alone, nothing added up, takes 325: what is left
// of the 16384 FLOP a clock is the hand-over of every block of 128 through a
// barrier each way (870 clocks, of which two buffers in halves hide most). With a
// scale for every row of B 547 us: the epilogue's two multiply-adds and a shared
// load for each pair of elements, 297 instructions of a warp for a block against
// 190, take longer than the product.
#include "sm103_ff_gemm.cuh"

namespace gemm_tn_impl {

using namespace gemm_tn_dev::ff;

template <int kForm>
using E4m3Pair256 = Tile<kForm, 2, 256, 6, false>;

template <int kForm>
cudaError_t launch_e4m3(int tile, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  switch (tile) {
    case kFfPair256: return FfLauncher<E4m3Pair256<kForm>>::launch(args, grid, stream);
    case kFfPair128: return FfLauncher<Tile<kForm, 2, 128, 8, false>>::launch(args, grid, stream);
    case kFfSingle128: return FfLauncher<Tile<kForm, 1, 128, 6, false>>::launch(args, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_ff_e4m3(int tile, bool b_rows, const gemm_tn_dev::FfArgs& args, int grid, cudaStream_t stream) {
  return b_rows ? launch_e4m3<kE4m3Rows>(tile, args, grid, stream) : launch_e4m3<kE4m3>(tile, args, grid, stream);
}

int ff_resident_pairs(int sms) { return FfLauncher<E4m3Pair256<kE4m3>>::resident(sms); }

}  // namespace gemm_tn_impl

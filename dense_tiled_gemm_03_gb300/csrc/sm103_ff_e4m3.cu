// sm103_ff_e4m3.cu -- instantiations.
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

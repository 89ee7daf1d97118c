// ff_pad.h -- the layout of a copy of 16-bit rows (pad_rows_kernel), and which of
// the source's memory each part of it reads; plain C++ for the host and the device.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FF_PAD_CALL __host__ __device__ __forceinline__
#else
#define FF_PAD_CALL inline
#endif

namespace gemm_tn_dev {
namespace ff {

// Elements between rows of the copy: whole 128-byte lines, since a box's row is one;
// up to half a line whole 16-byte pieces, which take less memory and time (A^T B with A
// 262144 x 20: 116 us, in lines 123; x 36 123 in lines, 128 in pieces).
FF_PAD_CALL int64_t pad_pitch(int64_t cols) { return cols <= 32 ? (cols + 7) / 8 * 8 : (cols + 63) / 64 * 64; }

// A 16-byte piece of the copy: 8 elements of a row, or those of them that the row
// has, from the one or two aligned 16-byte pieces of the source that hold them. Behind
// the row's last column, where the source may end, there are none to load.
struct PadPiece {
  int valid;        // elements inside the row: 8, fewer at its end, none (<= 0) behind it
  uint32_t shift;   // bytes from `at` to the first of them
  uintptr_t at;     // the first aligned piece
  bool first, second;   // whether it, and the one behind it, hold any of them
};

// The piece at column `col` of a row of `cols` elements that begins at address `row`.
FF_PAD_CALL PadPiece pad_piece(uintptr_t row, int64_t cols, int64_t col) {
  const int64_t left = cols - col;
  const int valid = static_cast<int>(left < 8 ? left : 8);
  const uintptr_t from = row + static_cast<uintptr_t>(col) * 2, at = from & ~static_cast<uintptr_t>(15);
  const uintptr_t end = from + static_cast<uintptr_t>(static_cast<int64_t>(valid)) * 2;
  return {valid, static_cast<uint32_t>(from - at), at, valid > 0, valid > 0 && at + 16 < end};
}

}  // namespace ff
}  // namespace gemm_tn_dev

#undef FF_PAD_CALL

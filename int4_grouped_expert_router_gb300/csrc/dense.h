// Products with 16-bit weights (dense.cu).
//
// Layout of an uploaded weight: tiles of 128 rows x 64 columns, 16 KB each and contiguous, rows and columns behind the last
// being 0; a block of 128 rows is its column tiles one after another. In a tile the rows are 128 bytes apart and the 16-byte
// chunks of row r lie at chunk ^ (r % 8): the 128-byte swizzle of the tensor core's operands, so that a tile is one bulk copy.
#pragma once

#include "coli_internal.h"

namespace coli {

constexpr int kDenseRows = 128, kDenseCols = 64;
constexpr uint32_t kDenseTile = kDenseRows * kDenseCols * 2;  // bytes

inline size_t dense_bytes(int O, int I) {
  return (size_t)((O + kDenseRows - 1) / kDenseRows) * (size_t)((I + kDenseCols - 1) / kDenseCols) * kDenseTile;
}

struct DenseArgs {
  const uint8_t* w;
  int O, I;
  const void* x;
  long long x_stride;
  int S;
  const float* bias;
  int act;
  const void* mul;
  const void* resid;
  void* y;
  long long mul_stride, resid_stride, y_stride;
  int* err;
};

// Workspace of a call that lays its activations out first: `parts` planes (up to 3) of S rows, each padded to 16 bytes.
inline size_t dense_x_bytes(long long S, int I, int parts) { return (size_t)S * ((size_t)(I + 7) / 8 * 16) * parts; }

// rows [row0, row0 + rows) of W [. x I], row-major at `src`, into the layout; row0 a multiple of kDenseRows.
cudaError_t launch_dense_pack(cudaStream_t stream, const uint16_t* src, int rows, int row0, int I, uint8_t* w);
// w_map: the weight's tiles as rows of 64, in boxes of a tile.
int launch_dense(coli_ctx* ctx, const DenseArgs& a, const CUtensorMap& w_map, int x_dtype, int y_dtype);

}  // namespace coli

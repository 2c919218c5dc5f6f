// Internal interface between the C-ABI front end (kda_block_api.cpp, plain
// C++) and the HIP translation unit of the norms at a block's end
// (kda_block_norm.hip): the heads' norm with the output gate, and the
// residual sum with the norm before the next block.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda_layer.h"

namespace kda {

constexpr int kBlockNormMaxDim = 8192;  // channels that one norm runs over

// Rows of D channels, H of them a token.
struct BlockNormArgs {
  const void *x, *z;  // z: the gate, or what x is added to
  int64_t ld_x, ld_z; // between tokens
  const float *w, *channels;
  int64_t rows;
  int H, D;
  int act;            // gate: 0 sigmoid, 1 SiLU
  float scale, eps;
};

// How a row is spread: `vec` consecutive channels a lane and load, `lanes`
// lanes a row (256: the workgroup), `loads` of them a lane.  Vectors of 16
// bytes where they tile the row, else single channels.  The fewest lanes with
// one load of them, but two loads rather than more than a wave; four loads a
// lane of a wave leave the backward pass one wave a SIMD (54.6 us for 8192 rows
// of 2048 channels in bf16, against 43.5 for one load of the workgroup).
struct RowShape {
  int vec, lanes, loads;
};
constexpr RowShape block_norm_shape(int D, int elem) {
  const int vec = D % (16 / elem) == 0 ? 16 / elem : 1, n = (D + vec - 1) / vec;
  if (n <= 16) return RowShape{vec, 16, 1};
  if (n <= 32) return RowShape{vec, 32, 1};
  if (n <= 64) return RowShape{vec, 64, 1};
  if (n <= 128) return RowShape{vec, 64, 2};
  if (n <= 256) return RowShape{vec, 256, 1};
  if (n <= 512) return RowShape{vec, 256, 2};
  if (n <= 1024) return RowShape{vec, 256, 4};
  if (n <= 2048) return RowShape{vec, 256, 8};
  return RowShape{vec, 256, 32};
}

constexpr int kBlockNormThreads = 256;
// Workgroups of the backward pass at most; each leaves a row of partial sums
// for every parameter (8192 rows of 2048 channels in bf16 43.7 us, with 256 of
// them 46.4, with 1024 50.7).
constexpr int kBlockNormParts = 512;

inline bool block_norm_fits(int64_t rows, int D, int elem) {
  const int64_t each = kBlockNormThreads / block_norm_shape(D, elem).lanes;
  return rows <= INT32_MAX && grid_fits(ceil_div(rows, each), kBlockNormThreads);
}
inline int64_t block_norm_parts(int64_t rows, int D, int elem) {
  const int64_t n = ceil_div(rows, kBlockNormThreads / block_norm_shape(D, elem).lanes);
  return n < kBlockNormParts ? n : kBlockNormParts;
}

int launch_gated_norm_forward(int is_bf16, const BlockNormArgs& a, void* y, void* stream);
int launch_gated_norm_backward(int is_bf16, const BlockNormArgs& a, const void* dy, void* dx, void* dz, float* dw,
                               float* part, void* stream);
int launch_residual_norm_forward(int is_bf16, const BlockNormArgs& a, void* y, void* total, void* stream);
// a.z: the total that the forward pass left
int launch_residual_norm_backward(int is_bf16, const BlockNormArgs& a, const void* dy, const void* dtotal, void* dx,
                                  void* dres, float* dw, float* dchannels, float* part, void* stream);

}  // namespace kda

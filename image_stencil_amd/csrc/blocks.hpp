// blocks.hpp -- plans and kernel launchers of the operators around attention
// (sum and norm between blocks, dense layers) behind the C ABI.
#pragma once

#include "imgstencil.h"

namespace is {

// Pointers of a block_norm call; null where absent. Sizes and strides in the descriptor.
struct NormPointers {
  const void *x, *y, *gate, *scale, *shift;
  const float *post_weight, *weight, *bias;
  void *x_out, *out;
};
// Threads of a launch (host only; the launcher's rule).
double block_norm_threads(const block_norm_desc &d);
hipError_t launch_block_norm(const block_norm_desc &d, const NormPointers &p, hipStream_t s);

struct DensePlan {
  dense_desc asked;       // as the caller gave it
  dense_desc d;           // rows flattened where the strides allow it
  const char *name;
  bool few;               // few rows: weights streamed past the rows' sums
  int tile;               // which tile (many rows), or 16-row groups (few rows)
  int tile_rows, tile_features;
  int splits, split_in;   // parts of the inner sum, and their length
  int block, lds;
  int64_t row_tiles, feature_tiles;   // of one entry
};

constexpr double kMaxLaunchThreads = 4294967295.0;

// Fills everything after d; false when the grid would be too large.
bool configure_dense(DensePlan &p);
size_t dense_workspace(const DensePlan &p);
hipError_t launch_dense(const DensePlan &p, const void *x, const void *w, const float *bias, const void *residual,
                        void *out, void *ws, hipStream_t s);

}  // namespace is

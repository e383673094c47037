// attention.hpp -- plans and kernel launchers of the attention operators
// (rotary positions, the norm of queries and keys with the rotation, cross
// attention) behind the C ABI.
#pragma once

#include <math.h>

#include "imgstencil.h"

namespace is {

// A rotary plan: the descriptor and each frequency of an axis in turns per
// position (f / 2 pi, 64 bits), so that an angle is reduced to one turn by
// dropping whole turns before it is rounded to 32 bits.
struct RotaryPlan {
  rotary_desc d;
  int per_axis;                          // Pa = rot / 2 / axes
  double freq[IS_MAX_HEAD_DIM / 2];      // radians per position
  double turns[IS_MAX_HEAD_DIM / 2];     // turns per position, less whole ones, of every pair (axis after axis)
};

// One tensor of a rotary launch.
struct RotaryPart {
  const void *x;
  void *y;
  const float *weight;        // d fp32 or null (ones); used with a norm only
  const int32_t *positions;   // null: no rotation (rot = 0)
  int64_t pos_batch_stride;
  is_tokens xt, yt;
};

// norm: 0 (none), IS_NORM_RMS or IS_NORM_LAYER. parts with no element are skipped.
hipError_t launch_rotary(const RotaryPlan &p, is_dtype dtype, int norm, float eps, const RotaryPart *parts,
                         int nparts, hipStream_t s);
// Elements a lane of the rotary kernel moves per access: 16 bytes, 8 or one
// element (host only; the launcher's rule).
int rotary_vector_width(const RotaryPlan &p, is_dtype dtype);
// Blocks of kRotaryBlock threads that one part takes (host only; the launcher's rule).
constexpr int kRotaryBlock = 256;
int64_t rotary_blocks(const RotaryPlan &p, int vec, const is_tokens &t);

struct AttentionPlan {
  cross_attention_desc d;
  float scale;            // resolved: never 0
  const char *name;
  int group;              // query heads per key head
  int rows;               // lq * group: rows that share a key head's keys
  int dp;                 // d padded to the kernel's head size
  int tile_rows;          // rows per workgroup
  int row_tiles;
  int splits;             // workgroups the keys of one row tile are split over
  int split_keys;         // keys per split, a multiple of a wave's key tile
  int run;                // row tiles a workgroup goes through
  int block, lds;
  int64_t units;          // n * hkv * row_tiles
  int64_t workgroups;     // of one split: n * hkv * runs of row tiles
};

// A launch counts its threads in 32 bits.
constexpr double kMaxThreads = 4294967295.0;

// What the kernel multiplies scores by: |scale| in units of a power of two.
inline float score_factor(float scale) { return (float)(fabs((double)scale) * 1.4426950408889634); }

// Fills everything after d and scale; false when the grid would be too large.
bool configure_attention(AttentionPlan &p);
size_t attention_workspace(const AttentionPlan &p);
hipError_t launch_attention(const AttentionPlan &p, const void *q, const void *k, const void *v,
                            const uint8_t *mask, const int32_t *lengths, void *out, float *lse, void *ws,
                            hipStream_t s);

}  // namespace is

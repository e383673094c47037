// held.hpp -- states held in 8 bits: their layout, plans and kernel launchers.
//
// The states of one entry, head and block of 32 tokens are a record of 64 dp bytes
// (dp: d padded to a multiple of 32), records in the order [entry][head][block]:
//   K: [dp / 16][32 tokens][16]              16 elements of a token
//   V: [dp / 32][half][32 elements][16]      16 tokens of an element: the half's tokens
//      8 a + 4 half + (0..3), a = 0..3, in this order
// which is what the 64 lanes of a wave hold of a 32-row operand of
// v_mfma_f32_32x32x16 for two steps, 16 consecutive bytes each, so that a record is
// read in whole 1 KB pieces (the order of K's inner index is free, and V's is the order
// in which the score accumulators hold the keys). Behind all records: the scales
// of k and v of each, two floats.
#pragma once

#include <type_traits>

#include "attention.hpp"
#include "imgstencil.h"

namespace is {

inline int held_padded(int d) { return (d + 31) / 32 * 32; }
inline int64_t held_blocks(int len) { return ((int64_t)len + IS_HELD_BLOCK - 1) / IS_HELD_BLOCK; }
inline int64_t held_records(const held_states_desc &d) { return (int64_t)d.n * d.heads * held_blocks(d.len); }
inline int64_t held_scales_at(const held_states_desc &d) { return held_records(d) * 64 * held_padded(d.d); }
inline size_t held_bytes(const held_states_desc &d) { return (size_t)(held_scales_at(d) + held_records(d) * 8); }

// Calls f(std::integral_constant<int, DP>) for a padded head size.
template <typename F>
hipError_t for_padded(int dp, F &&f) {
  switch (dp) {
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 96: return f(std::integral_constant<int, 96>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 160: return f(std::integral_constant<int, 160>{});
    case 192: return f(std::integral_constant<int, 192>{});
    case 224: return f(std::integral_constant<int, 224>{});
    default: return f(std::integral_constant<int, 256>{});
  }
}

// One side (keys or values) of a store or load: the caller's tensor.
struct HeldSide {
  const void *p;
  int64_t batch, token, head;
};

hipError_t launch_held_store(const held_states_desc &d, const HeldSide &k, const HeldSide &v, int len, int at,
                             const uint8_t *mask, int64_t mask_stride, const int32_t *lengths, void *held,
                             hipStream_t s);
hipError_t launch_held_load(const held_states_desc &d, const void *held, int at, int len, const HeldSide &k,
                            const HeldSide &v, bool read_next, hipStream_t s);

struct HeldPlan {
  held_attention_desc d;
  float scale;            // resolved: never 0
  const char *name;
  int group, rows;        // query heads per key head; rows that share a key head's keys
  bool direct;            // the held bytes are read by the attention itself
  int row_tiles, splits, split_blocks;   // direct: tiles of 32 rows; parts of the keys, in blocks
  int block, lds;
  int64_t workgroups;     // of one split
  AttentionPlan loaded;   // otherwise: cross attention to the loaded states
};

bool configure_held(HeldPlan &p);
size_t held_workspace(const HeldPlan &p);
hipError_t launch_held_attention(const HeldPlan &p, const void *q, const void *held, const uint8_t *mask,
                                 const int32_t *lengths, void *out, float *lse, void *ws, hipStream_t s);

}  // namespace is

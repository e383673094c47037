// join.hpp -- joins the parts of attention rows whose keys were split over
// workgroups.
#pragma once

#include <float.h>
#include <math.h>

#include "common.hpp"

namespace is {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

// part: O / l of every part, [entry and key head][split][row tile][tile row][d];
// part_lse: log2 of the sum of exponentials, in the same order.
struct JoinArgs {
  const float *part, *part_lse;
  void *out;
  float *lse;
  int64_t os[3];
  int lq, hq, hkv, d, group, rows, row_tiles, tile_rows, splits;
  int log_sg;              // threads (log2) that join the splits of 8 elements
  int64_t items;           // 8 elements each
};

// Joins the splits of a row. 2^log_sg neighbouring threads take 8 elements,
// each the splits of its own, and exchange sums: with few rows, the latency of
// reading one split after another would be all the time.
template <typename T>
__global__ __launch_bounds__(256) void is_k11_attention_join(const JoinArgs a) {
  typedef T T8 __attribute__((ext_vector_type(8)));
  const int64_t thread = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int sg = threadIdx.x & ((1 << a.log_sg) - 1);
  const int64_t it = thread >> a.log_sg;
  if (it >= a.items) return;   // whole groups leave
  const int chunks = a.d / 8, e = (int)(it % chunks) * 8;
  const int64_t row = it / chunks;
  const int r = (int)(row % a.rows), bh = (int)(row / a.rows);
  const int rt = r / a.tile_rows, tr = r % a.tile_rows;
  const int64_t step = (int64_t)a.row_tiles * a.tile_rows;
  const int64_t at = ((int64_t)bh * a.splits * a.row_tiles + rt) * a.tile_rows + tr;
  float top = -FLT_MAX, sum = 0.f, f[8] = {};
  for (int i = sg; i < a.splits; i += 1 << a.log_sg) {
    const float x = a.part_lse[at + i * step];
    const floatx4 *p = reinterpret_cast<const floatx4 *>(a.part + (at + i * step) * a.d + e);
    const floatx4 lo = p[0], hi = p[1];
    const float next = fmaxf(top, x), old = __builtin_amdgcn_exp2f(top - next), w = __builtin_amdgcn_exp2f(x - next);
    top = next;
    sum = sum * old + w;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[u] = f[u] * old + w * lo[u];
      f[4 + u] = f[4 + u] * old + w * hi[u];
    }
  }
  float most = top;
  for (int i = 0; i < a.log_sg; ++i) most = fmaxf(most, __shfl_xor(most, 1 << i));
  const float scale = __builtin_amdgcn_exp2f(top - most);
  sum *= scale;
#pragma unroll
  for (int u = 0; u < 8; ++u) f[u] *= scale;
  for (int i = 0; i < a.log_sg; ++i) {
    sum += __shfl_xor(sum, 1 << i);
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] += __shfl_xor(f[u], 1 << i);
  }
  if (sg != 0) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T8 w;
#pragma unroll
  for (int u = 0; u < 8; ++u) w[u] = (T)(f[u] * inv);
  const int b = bh / a.hkv, i = r / a.group, h = bh % a.hkv * a.group + r % a.group;
  *reinterpret_cast<T8 *>(static_cast<T *>(a.out) + b * a.os[0] + i * a.os[1] + h * a.os[2] + e) = w;
  if (a.lse && e == 0)
    a.lse[((int64_t)b * a.hq + h) * a.lq + i] =
        sum == 0.f ? -INFINITY : (most + __log2f(sum)) * 0.69314718055994531f;
}

// Threads (log2) that join the splits of 8 elements.
int join_group(int splits) {
  int l = 0;
  while (l < 5 && (1 << l) < splits) ++l;
  return l;
}

template <typename T>
hipError_t launch_join(const JoinArgs &j, hipStream_t s) {
  return launch_kernel(is_k11_attention_join<T>, dim3((unsigned)(((j.items << j.log_sg) + 255) / 256)), dim3(256), 0, s,
                       j);
}

}  // namespace
}  // namespace is

// k11_attention.hip -- cross attention, the plain kernel: one workgroup per
// query row walks the visible keys in tiles of 256 with a running maximum and
// sum of the softmax.
#include <math.h>

#include "attention.hpp"
#include "common.hpp"

namespace is {
namespace {

constexpr int kKeys = 256;

struct Args {
  const void *q, *k, *v;
  const uint8_t *mask;
  const int32_t *lengths;
  void *out;
  float *lse;
  cross_attention_desc d;
  float scale;
};

__device__ __forceinline__ float block_max(float v, float *tmp) {
  for (int i = 32; i; i >>= 1) v = fmaxf(v, __shfl_xor(v, i));
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x / 64] = v;
  __syncthreads();
  v = fmaxf(fmaxf(tmp[0], tmp[1]), fmaxf(tmp[2], tmp[3]));
  __syncthreads();
  return v;
}

template <typename T>
__global__ __launch_bounds__(kKeys) void is_k11_attention_plain(const Args a) {
  __shared__ float q[IS_MAX_HEAD_DIM], p[kKeys], tmp[4];
  const cross_attention_desc &d = a.d;
  const int64_t row = blockIdx.x;
  const int i = (int)(row % d.lq), h = (int)(row / d.lq % d.hq), b = (int)(row / d.lq / d.hq);
  const int hk = h / (d.hq / d.hkv), t = threadIdx.x;
  const T *qp = static_cast<const T *>(a.q) + b * d.q_stride[0] + i * d.q_stride[1] + h * d.q_stride[2];
  const T *kp = static_cast<const T *>(a.k) + b * d.k_stride[0] + hk * d.k_stride[2];
  const T *vp = static_cast<const T *>(a.v) + b * d.v_stride[0] + hk * d.v_stride[2];
  T *op = static_cast<T *>(a.out) + b * d.out_stride[0] + i * d.out_stride[1] + h * d.out_stride[2];
  if (t < d.d) q[t] = (float)qp[t];
  __syncthreads();
  int len = d.lk;
  if (a.lengths) len = min(len, max(0, a.lengths[b]));
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int j0 = 0; j0 < len; j0 += kKeys) {
    const int j = j0 + t;
    const bool see = j < len && (!a.mask || a.mask[b * d.mask_batch_stride + j]);
    float s = -INFINITY;
    if (see) {
      s = 0.f;
      for (int c = 0; c < d.d; ++c) s += q[c] * (float)kp[j * d.k_stride[1] + c];
      s *= a.scale;
    }
    const float top = fmaxf(m, block_max(s, tmp));
    const float base = top == -INFINITY ? 0.f : top;
    const float shrink = expf(m - base);
    p[t] = see ? expf(s - base) : -1.f;   // -1: not visible
    __syncthreads();
    l *= shrink;
    o *= shrink;
    for (int c = 0; c < kKeys; ++c) {
      if (p[c] < 0.f) continue;
      l += p[c];
      if (t < d.d) o += p[c] * (float)vp[(int64_t)(j0 + c) * d.v_stride[1] + t];
    }
    m = top;
    __syncthreads();
  }
  if (t < d.d) op[t] = (T)(l == 0.f ? 0.f : o / l);
  if (t == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

bool configure_attention(AttentionPlan &p) {
  const cross_attention_desc &d = p.d;
  p.name = "is_k11_attention_plain";
  p.group = d.hq / d.hkv;
  p.rows = d.lq * p.group;
  p.dp = d.d;
  p.tile_rows = 1;
  p.row_tiles = p.rows;
  p.splits = 1;
  p.split_keys = d.lk;
  p.block = kKeys;
  p.lds = 0;
  p.units = (int64_t)d.n * d.hkv * p.row_tiles;
  return p.units <= 2147483647;
}

size_t attention_workspace(const AttentionPlan &) { return 0; }

hipError_t launch_attention(const AttentionPlan &p, const void *q, const void *k, const void *v,
                            const uint8_t *mask, const int32_t *lengths, void *out, float *lse, void *,
                            hipStream_t s) {
  const Args a = {q, k, v, mask, lengths, out, lse, p.d, p.scale};
  if (p.d.dtype == IS_F16)
    return launch_kernel(is_k11_attention_plain<_Float16>, dim3((unsigned)p.units), dim3(kKeys), 0, s, a);
  return launch_kernel(is_k11_attention_plain<__bf16>, dim3((unsigned)p.units), dim3(kKeys), 0, s, a);
}

}  // namespace is

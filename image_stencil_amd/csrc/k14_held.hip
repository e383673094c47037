// k14_held.hip -- keys and values into 8 bits and back.
//
// A workgroup takes one block of 32 tokens of one entry and head, keys then values:
// each thread has 8 neighbouring elements of a token, so that reads and writes
// of the caller's tensor are whole rows of a head. The scale is the power of two
// that brings the largest finite magnitude to 448 or under, taken from its exponent
// and fraction bits, so that quotients are exact and rounding is that of the
// conversion to e4m3 alone. The record is put together in LDS and leaves in whole
// lines.
#include <math.h>

#include "common.hpp"
#include "held.hpp"

namespace is {
namespace {

constexpr int kThreads = 256;
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));

struct Args {
  HeldSide side[2];        // keys, values
  char *held;
  int64_t scales_at;       // bytes
  const uint8_t *mask;
  const int32_t *lengths;
  int64_t mask_stride;
  int heads, d, len, at;   // len, at: tokens of the call
  int blocks, capacity_blocks;   // blocks that the call touches; of an entry and head
};

// Byte of (token, element) in the key and the value part of a record.
__device__ __forceinline__ int key_byte(int token, int e) { return (e >> 4) * 512 + token * 16 + (e & 15); }
__device__ __forceinline__ int value_byte(int token, int e) {
  const int half = (token >> 2) & 1, order = (token >> 3) * 4 + (token & 3);
  return (e >> 5) * 1024 + half * 512 + (e & 31) * 16 + order;
}

template <typename T>
__device__ __forceinline__ constexpr int top_exponent() { return sizeof(T) == 2 && __is_same(T, _Float16) ? 8 : 120; }

// Largest magnitude of the workgroup.
__device__ __forceinline__ float block_max(float v, float *shared) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) v = fmaxf(v, __shfl_xor(v, m));
  if ((threadIdx.x & (kWave - 1)) == 0) shared[threadIdx.x / kWave] = v;
  __syncthreads();
  return fmaxf(fmaxf(shared[0], shared[1]), fmaxf(shared[2], shared[3]));
}

// DP: d padded. A thread holds NV vectors of 8 elements.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void is_k14_held_store(const Args a) {
  typedef T uvec __attribute__((ext_vector_type(8), aligned(sizeof(T))));   // at any element
  constexpr int CH = DP / 8, NV = (32 * CH + kThreads - 1) / kThreads;
  __shared__ __attribute__((aligned(16))) char record[32 * DP];
  __shared__ float shared[2][4];
  lds_poison(record, sizeof(record));
  const int per = a.blocks, blk = blockIdx.x % per, bh = blockIdx.x / per, b = bh / a.heads, h = bh % a.heads;
  int len = a.len;
  if (a.lengths) len = min(len, max(0, a.lengths[b]));
  const int64_t rec = (int64_t)bh * a.capacity_blocks + a.at / 32 + blk;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const HeldSide &t = a.side[side];
    const T *p = static_cast<const T *>(t.p) + b * t.batch + h * t.head;
    float f[NV][8];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int item = threadIdx.x + i * kThreads, token = item / CH, e = item % CH * 8, at = blk * 32 + token;
      bool in = item < 32 * CH && e < a.d && at < len;
      if (in && a.mask) in = a.mask[b * a.mask_stride + at] != 0;
      uvec x = {};
      if (in) x = *reinterpret_cast<const uvec *>(p + at * t.token + e);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[i][j] = (float)x[j];
        const float m = fabsf(f[i][j]);
        if (m < INFINITY) most = fmaxf(most, m);
      }
    }
    most = block_max(most, shared[side]);
    // most = 1.f 2^(E - 127) = (1.f / 2) 2^(E - 126), and 448 = (1.75 / 2) 2^9.
    const unsigned bits = __float_as_uint(most);
    int e2 = (int)(bits >> 23) - ((bits & 0x7fffffu) <= 0x600000u ? 135 : 134);
    e2 = max(e2, -120);
    const float scale = __uint_as_float((unsigned)(e2 + 127) << 23), inv = __uint_as_float((unsigned)(127 - e2) << 23);
    const float cap = e2 == top_exponent<T>() ? 240.f : 448.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int item = threadIdx.x + i * kThreads, token = item / CH, e = item % CH * 8;
      if (item >= 32 * CH) continue;
      float z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = f[i][j] * inv;
        z[j] = fabsf(f[i][j]) < INFINITY ? fminf(fmaxf(q, -cap), cap) : NAN;
      }
      int lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(z[4], z[5], 0, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(z[6], z[7], hi, true);
      if (side == 0) {
        *reinterpret_cast<uintx2 *>(record + key_byte(token, e)) = uintx2{(unsigned)lo, (unsigned)hi};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) record[value_byte(token, e + j)] = (char)((j < 4 ? lo : hi) >> (8 * (j & 3)));
      }
    }
    __syncthreads();
    char *to = a.held + rec * 64 * DP + side * 32 * DP;
    for (int i = threadIdx.x; i < 2 * DP; i += kThreads)
      *reinterpret_cast<uintx4 *>(to + i * 16) = *reinterpret_cast<const uintx4 *>(record + i * 16);
    if (threadIdx.x == 0) *reinterpret_cast<float *>(a.held + a.scales_at + (rec * 2 + side) * 4) = scale;
    __syncthreads();
  }
}

template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void is_k14_held_load(const Args a) {
  typedef T uvec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  typedef float F2 __attribute__((ext_vector_type(2)));
  constexpr int CH = DP / 8;
  __shared__ __attribute__((aligned(16))) char record[64 * DP];
  lds_poison(record, sizeof(record));
  const int per = a.blocks, blk = a.at / 32 + blockIdx.x % per, bh = blockIdx.x / per, b = bh / a.heads, h = bh % a.heads;
  const int64_t rec = (int64_t)bh * a.capacity_blocks + blk;
  const char *from = a.held + rec * 64 * DP;
  for (int i = threadIdx.x; i < 4 * DP; i += kThreads)
    *reinterpret_cast<uintx4 *>(record + i * 16) = *reinterpret_cast<const uintx4 *>(from + i * 16);
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const HeldSide &t = a.side[side];
    const float scale = *reinterpret_cast<const float *>(a.held + a.scales_at + (rec * 2 + side) * 4);
    T *p = static_cast<T *>(const_cast<void *>(t.p)) + b * t.batch + h * t.head;
    for (int item = threadIdx.x; item < 32 * CH; item += kThreads) {
      const int token = item / CH, e = item % CH * 8, at = blk * 32 + token - a.at;
      if (e >= a.d || at < 0 || at >= a.len) continue;
      uintx2 w;
      if (side == 0) {
        w = *reinterpret_cast<const uintx2 *>(record + key_byte(token, e));
      } else {
        w = uintx2{0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j / 4] |= (unsigned)(unsigned char)record[32 * DP + value_byte(token, e + j)] << (8 * (j & 3));
      }
      uvec y;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const F2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
        y[4 * j] = (T)(lo[0] * scale);
        y[4 * j + 1] = (T)(lo[1] * scale);
        y[4 * j + 2] = (T)(hi[0] * scale);
        y[4 * j + 3] = (T)(hi[1] * scale);
      }
      *reinterpret_cast<uvec *>(p + at * t.token + e) = y;
    }
  }
}

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

Args arguments_of(const held_states_desc &d, const HeldSide &k, const HeldSide &v, int len, int at, const void *held) {
  Args a = {};
  a.side[0] = k;
  a.side[1] = v;
  a.held = static_cast<char *>(const_cast<void *>(held));
  a.scales_at = held_scales_at(d);
  a.heads = d.heads;
  a.d = d.d;
  a.len = len;
  a.at = at;
  a.blocks = (int)(held_blocks(at + len) - at / IS_HELD_BLOCK);
  a.capacity_blocks = (int)held_blocks(d.len);
  return a;
}

}  // namespace

hipError_t launch_held_store(const held_states_desc &d, const HeldSide &k, const HeldSide &v, int len, int at,
                             const uint8_t *mask, int64_t mask_stride, const int32_t *lengths, void *held,
                             hipStream_t s) {
  Args a = arguments_of(d, k, v, len, at, held);
  a.mask = mask;
  a.mask_stride = mask_stride;
  a.lengths = lengths;
  const dim3 grid((unsigned)((int64_t)d.n * d.heads * a.blocks));
  return for_padded(held_padded(d.d), [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    return d.dtype == IS_F16 ? launch_kernel(is_k14_held_store<_Float16, DP>, grid, dim3(kThreads), 0, s, a)
                             : launch_kernel(is_k14_held_store<__bf16, DP>, grid, dim3(kThreads), 0, s, a);
  });
}

hipError_t launch_held_load(const held_states_desc &d, const void *held, int at, int len, const HeldSide &k,
                            const HeldSide &v, hipStream_t s) {
  const Args a = arguments_of(d, k, v, len, at, held);
  const dim3 grid((unsigned)((int64_t)d.n * d.heads * a.blocks));
  return for_padded(held_padded(d.d), [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    return d.dtype == IS_F16 ? launch_kernel(is_k14_held_load<_Float16, DP>, grid, dim3(kThreads), 0, s, a)
                             : launch_kernel(is_k14_held_load<__bf16, DP>, grid, dim3(kThreads), 0, s, a);
  });
}

}  // namespace is

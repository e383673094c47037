// k14_held.hip -- keys and values into 8 bits and back.
//
// A workgroup takes one block of 32 tokens of one entry and head: two waves its keys, two
// its values, all loads first. A key thread has 8 neighbouring elements of a token at a
// time, a value thread those of four tokens, which are neighbours in the record, so that
// both touch the caller's tensor in whole rows of a head and put words, not bytes,
// together. The scale is the power of two that brings the largest finite magnitude to
// 448 or under, taken from its exponent and fraction bits, so that quotients are exact and
// rounding is that of the conversion to e4m3 alone. The record is put together in LDS
// (16-byte slots permuted, so that lanes a row apart meet different banks) and
// leaves in whole lines.
//
// Bound: one read of the states and one write of half their bytes, and back. 4 entries of
// 16384 tokens, 4 heads of 128, bf16: put 44.8 us, got 37.3, 81 together, the rate of a large
// copy (80). What is read or written once passes the caches by: 52 and 48.6 us without
// that. (Single bytes to LDS in place of words of four tokens: put 57.)
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

// Slots of 16 bytes of a record while it is put together: token t of a key piece p, element
// e of a value half lie in another place of their 8.
__device__ __forceinline__ int key_slot(int piece, int token) { return piece * 32 + (token ^ (piece & 7)); }
__device__ __forceinline__ int value_slot(int half, int e) {
  return (e >> 5) * 64 + half * 32 + ((e & 31) ^ ((e >> 3) & 7));
}

// The largest finite magnitude.
template <typename V>
__device__ __forceinline__ float most_of(const V &x, float most) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = fabsf((float)x[j]);
    if (m < INFINITY) most = fmaxf(most, m);
  }
  return most;
}

// 8 numbers times inv as e4m3, at most cap: one that is none becomes NaN.
template <typename V>
__device__ __forceinline__ uintx2 e4m3(const V &x, float inv, float cap) {
  float z[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = (float)x[j];
    z[j] = fabsf(f) < INFINITY ? fminf(fmaxf(f * inv, -cap), cap) : NAN;
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(z[4], z[5], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(z[6], z[7], hi, true);
  return uintx2{(unsigned)lo, (unsigned)hi};
}

// DP: d padded.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void is_k14_held_store(const Args a) {
  typedef T uvec __attribute__((ext_vector_type(8), aligned(sizeof(T))));   // at any element
  constexpr int CH = DP / 8, HALF = kThreads / 2;
  constexpr int NK = 32 * CH / HALF;                         // vectors of a key thread
  constexpr int NG = (8 * CH + HALF - 1) / HALF;             // token fours of a value thread
  constexpr int NV = NK > 4 * NG ? NK : 4 * NG;
  __shared__ __attribute__((aligned(16))) uintx4 record[4 * DP];
  __shared__ float shared[4];
  lds_poison(record, sizeof(record));
  // Neighbouring workgroups: the heads of the same tokens, which lie together in memory.
  const int h = blockIdx.x % a.heads, rest = blockIdx.x / a.heads, blk = rest % a.blocks, b = rest / a.blocks;
  const int bh = b * a.heads + h;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), side = wave >> 1, thread = threadIdx.x & (HALF - 1);
  int len = a.len;
  if (a.lengths) len = min(len, max(0, a.lengths[b]));
  const int64_t rec = (int64_t)bh * a.capacity_blocks + a.at / 32 + blk;
  const HeldSide &t = a.side[side];
  const T *p = static_cast<const T *>(t.p) + b * t.batch + h * t.head;
  auto vector = [&](int token, int e) -> uvec {
    const int at = blk * 32 + token;
    bool in = e < a.d && at < len;
    if (in && a.mask) in = a.mask[b * a.mask_stride + at] != 0;
    return in ? __builtin_nontemporal_load(reinterpret_cast<const uvec *>(p + at * t.token + e)) : uvec{};
  };
  // Key vector i: token item / CH. Value four i: tokens 8 a + 4 half + (0..3) of group 2 a + half.
  uvec x[NV];
  float most = 0.f;
  if (side == 0) {
#pragma unroll
    for (int i = 0; i < NK; ++i) x[i] = vector((thread + i * HALF) / CH, (thread + i * HALF) % CH * 8);
#pragma unroll
    for (int i = 0; i < NK; ++i) most = most_of(x[i], most);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * NG; ++i) {
      const int item = thread + i / 4 * HALF;
      x[i] = item < 8 * CH ? vector(item / CH * 4 + i % 4, item % CH * 8) : uvec{};
    }
#pragma unroll
    for (int i = 0; i < 4 * NG; ++i) most = most_of(x[i], most);
  }
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) most = fmaxf(most, __shfl_xor(most, m));
  if ((threadIdx.x & (kWave - 1)) == 0) shared[wave] = most;
  __syncthreads();
  most = fmaxf(shared[2 * side], shared[2 * side + 1]);
  // most = 1.f 2^(E - 127) = (1.f / 2) 2^(E - 126), and 448 = (1.75 / 2) 2^9.
  const unsigned bits = __float_as_uint(most);
  int e2 = (int)(bits >> 23) - ((bits & 0x7fffffu) <= 0x600000u ? 135 : 134);
  e2 = max(e2, -120);
  const float scale = __uint_as_float((unsigned)(e2 + 127) << 23), inv = __uint_as_float((unsigned)(127 - e2) << 23);
  const float cap = e2 == top_exponent<T>() ? 240.f : 448.f;
  if (side == 0) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int item = thread + i * HALF, token = item / CH, e = item % CH * 8;
      reinterpret_cast<uintx2 *>(record + key_slot(e >> 4, token))[e >> 3 & 1] = e4m3(x[i], inv, cap);
    }
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int item = thread + g * HALF, group = item / CH, e = item % CH * 8;
      if (item >= 8 * CH) continue;
      uintx2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = e4m3(x[4 * g + i], inv, cap);
#pragma unroll
      for (int j = 0; j < 8; ++j) {      // byte j % 4 of the four tokens' words
        const unsigned pick = (j & 3) | (4 + (j & 3)) << 8;
        const unsigned lo = __builtin_amdgcn_perm(w[1][j / 4], w[0][j / 4], pick);
        const unsigned hi = __builtin_amdgcn_perm(w[3][j / 4], w[2][j / 4], pick);
        reinterpret_cast<unsigned *>(record + 2 * DP + value_slot(group & 1, e + j))[group >> 1] =
            __builtin_amdgcn_perm(hi, lo, 0x05040100u);
      }
    }
  }
  __syncthreads();
  uintx4 *to = reinterpret_cast<uintx4 *>(a.held + rec * 64 * DP);
  for (int i = threadIdx.x; i < 4 * DP; i += kThreads) {
    const int v = i - 2 * DP;
    to[i] = record[i < 2 * DP ? key_slot(i / 32, i % 32) : 2 * DP + value_slot(v / 32 & 1, v / 64 * 32 + v % 32)];
  }
  if (thread == 0) *reinterpret_cast<float *>(a.held + a.scales_at + (rec * 2 + side) * 4) = scale;
}

// READ_NEXT: by the next kernel, so that the caches are to keep it.
template <typename T, int DP, bool READ_NEXT>
__global__ __launch_bounds__(kThreads) void is_k14_held_load(const Args a) {
  typedef T uvec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  typedef float F2 __attribute__((ext_vector_type(2)));
  constexpr int CH = DP / 8;
  __shared__ __attribute__((aligned(16))) char record[64 * DP];
  lds_poison(record, sizeof(record));
  const int h = blockIdx.x % a.heads, rest = blockIdx.x / a.heads, blk = a.at / 32 + rest % a.blocks, b = rest / a.blocks;
  const int bh = b * a.heads + h;
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
      uvec *to = reinterpret_cast<uvec *>(p + at * t.token + e);
      if constexpr (READ_NEXT) *to = y;
      else __builtin_nontemporal_store(y, to);
    }
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
                            const HeldSide &v, bool read_next, hipStream_t s) {
  const Args a = arguments_of(d, k, v, len, at, held);
  const dim3 grid((unsigned)((int64_t)d.n * d.heads * a.blocks));
  return for_padded(held_padded(d.d), [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kThreads), 0, s, a); };
    if (d.dtype == IS_F16) return read_next ? go(is_k14_held_load<_Float16, DP, true>) : go(is_k14_held_load<_Float16, DP, false>);
    return read_next ? go(is_k14_held_load<__bf16, DP, true>) : go(is_k14_held_load<__bf16, DP, false>);
  });
}

}  // namespace is

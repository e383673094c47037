// k15_held_attention.hip -- cross attention to states held in 8 bits.
//
//   out = softmax(scale q k^T) v,  k and v = e4m3 numbers times a power of two for
//   each block of 32 keys.
//
// Up to some thousand rows (is_k15_held_attention): each wave walks blocks of its own for
// the same 32 rows; with few, the read of the held bytes is all the work. A record holds the operands as the
// lanes need them, so they go from memory to registers in pieces of 1 KB, are
// converted there (two numbers and their scale an instruction, exactly) and multiplied;
// LDS only joins the waves at the end. Products, running maximum and the
// order of keys are those of the cross attention kernel:
//   S^T (keys x rows) = K Q^T,   O^T (d x rows) = V^T P^T.
// Probabilities are rounded to the data type for the second product, whose instruction takes
// no wider operand; their sum l is of the unrounded ones, in fp32, like every other sum. That
// puts up to half a step of the type of sum p |v| / l on top of the result's own rounding (on
// random inputs, relative to 64 bits: bf16 0.0023 and fp16 0.00029, p in fp32 0.0017 and 0.00021).
// More rows: every call loads the states into the workspace, as 16-bit numbers, and the
// cross attention kernel runs on them.
//
// What bounds it, measured on MI355Xs: one token for each of 4 entries over 32771 keys, 16
// query and 2 key heads of 128, bf16: 17.4 us with the joining launch (16-bit states: 30.9),
// the read 14.4 us of it, 4.7 TB/s; 1024 rows over 4 x 4096 keys, 2 heads of 128: 30.6 us;
// loaded first, 3600 tokens over 3600, 2 x 8 heads of 64, fp16: 80, of which the load is 5.
#include <float.h>
#include <math.h>

#include "common.hpp"
#include "held.hpp"
#include "join.hpp"

namespace is {
namespace {

constexpr int kWaves = 4;
constexpr float kLazy = 8.f;   // log2 of how far a row's maximum may outgrow the one used

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfx8 __attribute__((ext_vector_type(8)));

struct Args {
  const void *q;
  const char *held;
  int64_t scales_at;
  const uint8_t *mask;
  const int32_t *lengths;
  void *out;
  float *lse, *part, *part_lse;
  int64_t qs[3], os[3], mask_bs;
  int lq, lk, hq, hkv, d, group, rows, row_tiles, splits, split_blocks, blocks;
  float c;                // |scale| log2(e)
  unsigned flip;          // sign bits of a negative scale
};

__device__ __forceinline__ floatx16 mma(halfx8 a, halfx8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mma(bfx8 a, bfx8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 8 held numbers (two words) times their block's scale.
template <typename T>
__device__ __forceinline__ T __attribute__((ext_vector_type(8))) unheld(unsigned lo, unsigned hi, float scale) {
  typedef T T8 __attribute__((ext_vector_type(8)));
  typedef T T2 __attribute__((ext_vector_type(2)));
  T2 r[4];
  if constexpr (__is_same(T, _Float16)) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true);
  } else {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  }
  T8 y;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = r[i / 2][i % 2];
  return y;
}

// The value of the lane 32 away, joined by max or sum.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int DP>
struct Geo {
  static constexpr int PIECES = DP / 32;            // 1 KB pieces of K (as many of V)
  static constexpr int JOIN_PITCH = DP + 4;         // floats
  static constexpr int BYTES = kWaves * 32 * (JOIN_PITCH + 2) * 4;
  static constexpr int WAVES = DP <= 128 ? 2 : 1;   // a SIMD
};

template <typename T, int DP, bool MASK>
__global__ __launch_bounds__(kWaves * 64, Geo<DP>::WAVES) void is_k15_held_attention(const Args a) {
  using G = Geo<DP>;
  typedef T T8 __attribute__((ext_vector_type(8)));
  constexpr int NP = G::PIECES;
  __shared__ __attribute__((aligned(16))) char lds[G::BYTES];
  lds_poison(lds, sizeof(lds));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n32 = lane & 31, half = lane >> 5;
  // Workgroup -> (entry and key head, split, row tile): a group's row tiles share an XCD.
  const int place = xcd_remap(blockIdx.x, gridDim.x);
  const int rt = place % a.row_tiles, g = place / a.row_tiles;
  const int split = g % a.splits, bh = g / a.splits, b = bh / a.hkv, hk = bh % a.hkv;

  int len = a.lk;
  if (a.lengths) len = min(len, max(0, a.lengths[b]));
  const int first = split * a.split_blocks;
  const int blocks = max(0, min((len + 31) / 32 - first, a.split_blocks));
  const int nt = (blocks - wave + kWaves - 1) / kWaves;      // blocks of this wave
  const int64_t rec0 = (int64_t)bh * a.blocks + first + wave;
  const char *at = a.held + rec0 * (64 * DP) + lane * 16;
  const float *scales = reinterpret_cast<const float *>(a.held + a.scales_at) + rec0 * 2;
  const uint8_t *mask = MASK ? a.mask + b * a.mask_bs + (first + wave) * 32 : nullptr;

  // ---- Queries: row n32's elements 32 c + 16 half + 8 s + (0..7) are step 2 c + s.
  const int r = rt * 32 + n32;
  const bool live = r < a.rows;
  const int i = live ? r / a.group : 0, h = live ? hk * a.group + r - i * a.group : 0;
  const T *q = static_cast<const T *>(a.q) + b * a.qs[0] + i * a.qs[1] + h * a.qs[2];
  T8 qf[2 * NP];
#pragma unroll
  for (int u = 0; u < 2 * NP; ++u) {
    const int e = (u >> 1) * 32 + half * 16 + (u & 1) * 8;
    uintx4 w = {0, 0, 0, 0};
    if (live && e < a.d) w = *reinterpret_cast<const uintx4 *>(q + e);
    w ^= a.flip;
    qf[u] = __builtin_bit_cast(T8, w);
  }

  uintx4 kr[2][NP], vr[2][NP];
  float ks[2], vs[2];
  uint8_t seen[2] = {1, 1};
  auto fetch = [&](int j, int to) {
    if (j >= nt) return;
    const char *p = at + (int64_t)j * kWaves * 64 * DP;
#pragma unroll
    for (int c = 0; c < NP; ++c) kr[to][c] = *reinterpret_cast<const uintx4 *>(p + c * 1024);
#pragma unroll
    for (int c = 0; c < NP; ++c) vr[to][c] = *reinterpret_cast<const uintx4 *>(p + 32 * DP + c * 1024);
    ks[to] = scales[(int64_t)j * kWaves * 2];
    vs[to] = scales[(int64_t)j * kWaves * 2 + 1];
    if constexpr (MASK) {
      const int key = (first + wave + j * kWaves) * 32 + n32;
      seen[to] = key < a.lk ? mask[j * kWaves * 32 + n32] : 0;
    }
  };
  floatx16 o[NP];
#pragma unroll
  for (int c = 0; c < NP; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[c][e] = 0.f;
  float m = -FLT_MAX, l = 0.f;

  auto step = [&](int j, int from) {
    const int left = len - (first + wave + j * kWaves) * 32;      // keys of this block, at least 1
    unsigned word = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
    if constexpr (MASK) word &= (unsigned)__ballot(seen[from] != 0);
    word = __builtin_amdgcn_readfirstlane(word);
    if (word == 0) return;
    floatx16 s;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
    for (int c = 0; c < NP; ++c) {
      s = mma(unheld<T>(kr[from][c][0], kr[from][c][1], ks[from]), qf[2 * c], s);
      s = mma(unheld<T>(kr[from][c][2], kr[from][c][3], ks[from]), qf[2 * c + 1], s);
    }
    // Accumulator e: key 8 (e / 4) + 4 half + e % 4.
    if (word != 0xffffffffu) {
      const unsigned mine = word >> (4 * half);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = mine >> (8 * (e >> 2) + (e & 3)) & 1 ? s[e] : -INFINITY;
      unsigned bytes[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) bytes[u] = (((mine >> (8 * u) & 15u) * 0x00204081u) & 0x01010101u) * 0xffu;
#pragma unroll
      for (int c = 0; c < NP; ++c)
#pragma unroll
        for (int u = 0; u < 4; ++u) vr[from][c][u] &= bytes[u];
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
    top = max_halves(top) * a.c;
    // The maximum in use moves when a row outgrows it.
    if (__any(top > m + kLazy)) {
      const float next = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int c = 0; c < NP; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[c][e] *= f;
    }
    T8 p[2];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x = __builtin_amdgcn_exp2f(s[e] * a.c - m);
      l += x;
      p[e / 8][e % 8] = (T)x;
    }
#pragma unroll
    for (int c = 0; c < NP; ++c) {
      o[c] = mma(unheld<T>(vr[from][c][0], vr[from][c][1], vs[from]), p[0], o[c]);
      o[c] = mma(unheld<T>(vr[from][c][2], vr[from][c][3], vs[from]), p[1], o[c]);
    }
  };
  fetch(0, 0);
  fetch(1, 1);
  for (int j = 0; j < nt; j += 2) {
    step(j, 0);
    fetch(j + 2, 0);
    if (j + 1 < nt) step(j + 1, 1);
    fetch(j + 3, 1);
  }

  // ---- Join the waves: out = sum_w 2^(M_w - M) O_w / sum_w 2^(M_w - M) l_w.
  l = sum_halves(l);
  float *jo = reinterpret_cast<float *>(lds), *jm = jo + kWaves * 32 * G::JOIN_PITCH, *jl = jm + kWaves * 32;
#pragma unroll
  for (int c = 0; c < NP; ++c)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<floatx4 *>(jo + (wave * 32 + n32) * G::JOIN_PITCH + 32 * c + 8 * u + 4 * half) =
          floatx4{o[c][4 * u], o[c][4 * u + 1], o[c][4 * u + 2], o[c][4 * u + 3]};
  if (half == 0) {
    jm[wave * 32 + n32] = m;
    jl[wave * 32 + n32] = l;
  }
  __syncthreads();
  const int chunks = a.d / 8;
  for (int it = threadIdx.x; it < 32 * chunks; it += kWaves * 64) {
    const int tr = it / chunks, e = it % chunks * 8, row = rt * 32 + tr;
    if (row >= a.rows) break;   // rows only grow with it
    float top = jm[tr], sum = 0.f, f[8] = {};
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, jm[w * 32 + tr]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float x = __builtin_amdgcn_exp2f(jm[w * 32 + tr] - top);
      sum += x * jl[w * 32 + tr];
#pragma unroll
      for (int y = 0; y < 8; ++y) f[y] += x * jo[(w * 32 + tr) * G::JOIN_PITCH + e + y];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);
#pragma unroll
    for (int y = 0; y < 8; ++y) f[y] *= inv;
    if (a.splits > 1) {
      const int64_t to = ((int64_t)g * a.row_tiles + rt) * 32 + tr;
      floatx4 *p = reinterpret_cast<floatx4 *>(a.part + to * a.d + e);
      p[0] = floatx4{f[0], f[1], f[2], f[3]};
      p[1] = floatx4{f[4], f[5], f[6], f[7]};
      if (e == 0) a.part_lse[to] = lse2;
    } else {
      const int qi = row / a.group, qh = hk * a.group + row - qi * a.group;
      T8 w;
#pragma unroll
      for (int y = 0; y < 8; ++y) w[y] = (T)f[y];
      *reinterpret_cast<T8 *>(static_cast<T *>(a.out) + b * a.os[0] + qi * a.os[1] + qh * a.os[2] + e) = w;
      if (a.lse && e == 0) a.lse[((int64_t)b * a.hq + qh) * a.lq + qi] = lse2 * 0.69314718055994531f;
    }
  }
}

template <typename T>
hipError_t launch_t(const HeldPlan &p, const Args &a, hipStream_t s) {
  const dim3 grid((unsigned)(p.workgroups * p.splits));
  const hipError_t e = for_padded(held_padded(a.d), [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    return a.mask ? launch_kernel(is_k15_held_attention<T, DP, true>, grid, dim3(kWaves * 64), 0, s, a)
                  : launch_kernel(is_k15_held_attention<T, DP, false>, grid, dim3(kWaves * 64), 0, s, a);
  });
  if (e != hipSuccess || p.splits == 1) return e;
  const JoinArgs j = {a.part, a.part_lse, a.out, a.lse, {a.os[0], a.os[1], a.os[2]}, a.lq, a.hq, a.hkv, a.d, a.group,
                      a.rows, a.row_tiles, 32, p.splits, join_group(p.splits),
                      (int64_t)p.d.held.n * a.hkv * a.rows * (a.d / 8)};
  return launch_join<T>(j, s);
}

// Bytes of the loaded keys (as many of values), a multiple of 16.
size_t loaded_bytes(const HeldPlan &p) {
  const held_states_desc &h = p.d.held;
  return (size_t)h.n * h.len * h.heads * h.d * 2;
}

}  // namespace

bool configure_held(HeldPlan &p) {
  const held_attention_desc &d = p.d;
  const held_states_desc &h = d.held;
  p.group = d.hq / h.heads;
  p.rows = d.lq * p.group;
  p.row_tiles = (p.rows + 31) / 32;
  const int64_t blocks = held_blocks(h.len), units = (int64_t)h.n * h.heads * p.row_tiles;
  // The held bytes directly up to 1024 row tiles (heads over 128: 512); beyond, the products
  // take so long that loading the states first for the faster kernel pays. Direct and loaded: 2 entries x 8 heads of 64 over 3600 keys, 3600 rows (1808
  // workgroups) 81.8 and 79.8 us, 1024 rows (512) 25.5 and 40.2; 4 x 2 heads of 128 over 4096
  // keys, 4096 rows (1024) 80.8 and 80.2, 8192 rows 160 and 136; 2 heads of 256 over 2000 keys,
  // 8192 rows (512) 58 and 64, 14400 rows 109 and 81.
  // (A token of more than 2^23 elements is beyond that kernel's strides.)
  const int64_t token = (int64_t)h.heads * h.d;
  p.direct = units <= (held_padded(h.d) <= 128 ? 1024 : 512) || token > (int64_t)1 << 23;
  p.splits = 1;
  p.split_blocks = (int)(blocks < 1 ? 1 : blocks);
  p.workgroups = units;
  p.block = kWaves * 64;
  p.name = "is_k15_held_attention";
  (void)for_padded(held_padded(h.d), [&](auto dp) {
    p.lds = Geo<decltype(dp)::value>::BYTES;
    return hipSuccess;
  });
  if (p.direct) {
    // A workgroup a CU, and at least two blocks a wave. (One token for each of 4 entries
    // over 32771 keys, 2 heads of 128: 32 parts 18.5 us with the join, 61 parts 19.0, 114
    // parts 22.2; 1000 keys, 4 heads of 128: 8 parts 7.7, none 8.2.) Several row tiles and
    // heads to 128, where the products are the work: two a CU if that leaves a wave 16 blocks
    // (1024 rows over 16384 keys, 8 heads of 64: 56 us, one a CU 81; but 512 rows over 3600
    // keys, 16 heads: 19.7 and 17.1).
    auto parts = [&](int64_t groups, int64_t each) {
      const int64_t n = units > 0 ? groups / units : 1, most = blocks / (each * kWaves);
      return n < most ? n : most;
    };
    int64_t splits = parts(256, 2);
    if (p.row_tiles > 1 && held_padded(h.d) <= 128 && parts(512, 16) > splits) splits = parts(512, 16);
    if (splits > 1) {
      p.split_blocks = (int)((blocks + splits - 1) / splits);
      p.splits = (int)((blocks + p.split_blocks - 1) / p.split_blocks);
    }
    const double join = (double)((int64_t)h.n * h.heads * p.rows * (h.d / 8) << join_group(p.splits)) + 255.0;
    return (double)p.workgroups * p.splits * p.block <= kMaxThreads && join <= kMaxThreads;
  }
  AttentionPlan &c = p.loaded;
  c.d = {h.n, d.lq, h.len, d.hq, h.heads, h.d, h.dtype, d.scale, {}, {}, {}, {}, d.mask_batch_stride};
  const int64_t batch = token * h.len;
  for (int i = 0; i < 3; ++i) {
    c.d.q_stride[i] = d.q_stride[i];
    c.d.out_stride[i] = d.out_stride[i];
    c.d.k_stride[i] = c.d.v_stride[i] = i == 0 ? batch : i == 1 ? token : h.d;
  }
  c.scale = p.scale;
  p.name = "is_k14_held_load, is_k11_attention";
  return configure_attention(c);
}

size_t held_workspace(const HeldPlan &p) {
  if (!p.direct) return 2 * loaded_bytes(p) + attention_workspace(p.loaded);
  return p.splits == 1 ? 0 : (size_t)p.workgroups * p.splits * 32 * (p.d.held.d + 1) * 4;
}

hipError_t launch_held_attention(const HeldPlan &p, const void *q, const void *held, const uint8_t *mask,
                                 const int32_t *lengths, void *out, float *lse, void *ws, hipStream_t s) {
  const held_attention_desc &d = p.d;
  const held_states_desc &h = d.held;
  if (!p.direct) {
    char *k = static_cast<char *>(ws), *v = k + loaded_bytes(p), *more = v + loaded_bytes(p);
    const int64_t token = (int64_t)h.heads * h.d, batch = token * h.len;
    if (h.n > 0 && h.len > 0) {
      const hipError_t e = launch_held_load(h, held, 0, h.len, {k, batch, token, h.d}, {v, batch, token, h.d}, true, s);
      if (e != hipSuccess) return e;
    }
    return launch_attention(p.loaded, q, k, v, mask, lengths, out, lse, more, s);
  }
  Args a;
  a.q = q;
  a.held = static_cast<const char *>(held);
  a.scales_at = held_scales_at(h);
  a.mask = mask;
  a.lengths = lengths;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float *>(ws);
  a.part_lse = a.part ? a.part + (size_t)p.workgroups * p.splits * 32 * h.d : nullptr;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = d.q_stride[i];
    a.os[i] = d.out_stride[i];
  }
  a.mask_bs = d.mask_batch_stride;
  a.lq = d.lq;
  a.lk = h.len;
  a.hq = d.hq;
  a.hkv = h.heads;
  a.d = h.d;
  a.group = p.group;
  a.rows = p.rows;
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.split_blocks = p.split_blocks;
  a.blocks = (int)held_blocks(h.len);
  a.c = score_factor(p.scale);
  a.flip = p.scale < 0.f ? 0x80008000u : 0u;
  return h.dtype == IS_F16 ? launch_t<_Float16>(p, a, s) : launch_t<__bf16>(p, a, s);
}

}  // namespace is

// k13_dense.hip -- dense layers on tokens:  out = residual + act(x w^T + bias).
//
// Weights are the first operand of the matrix instructions and tokens the second,
// so that a lane's results are consecutive features of one token.
//
// Many rows (is_k13_dense): a workgroup of WF x WT waves computes 32 FB WF
// features x 32 TB WT tokens with v_mfma_f32_32x32x16. Steps of 64 inputs of both
// operands lie in LDS in two buffers, brought by DMA without passing registers: a
// 128-byte row in 8 chunks of 16 bytes, chunk c of row r in slot c ^ ((r >> 1) & 7),
// so that 16 lanes reading one chunk of 16 rows meet 16 different bank groups. The
// last quarter of a step runs after the barrier that frees its buffer: its products
// cover the first operand reads of the next step, whose data the barrier has
// waited for, and the loads of the step after go out there. Results pass LDS as
// fp32 once, a wave's own part, so that residual and output are touched in whole
// rows of the wave's features.
//
// Few rows (is_k13_dense_few): the weights are read once, straight into registers,
// 16 features x 32 inputs an instruction (v_mfma_f32_16x16x32); the waves of a
// workgroup take the inner sum in turn and join in LDS.
#include <math.h>

#include "blocks.hpp"
#include "common.hpp"
#include "dma.hpp"

namespace is {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bfx8 __attribute__((ext_vector_type(8)));

struct Args {
  const void *x, *w, *residual;
  const float *bias;
  void *out;
  float *part;             // splits > 1: sums of the parts, [split][entry][row][feature]
  int64_t xb, xr, rb, rr, ob, orow, wr;
  int entries, len, in, features, act;
  int splits, split_in;
  int row_tiles, feature_tiles;
};

__device__ __forceinline__ floatx16 mma32(halfx8 a, halfx8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mma32(bfx8 a, bfx8 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mma16(halfx8 a, halfx8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mma16(bfx8 a, bfx8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}

// GELU is x Phi(x) = max(x, 0) - |x| Phi(-|x|), with Phi(-z) = exp(-z^2 / 2) R(z) and R a
// polynomial in t = 1 / (1 + 0.31 z), fitted to erfcx(z / sqrt 2) / 2 on 0 <= z <= 14:
// within 4.7e-6 of it everywhere, a hundredth of fp16's half step, so that small
// results at far negative x keep their digits. Where an exponential overflows, the
// factor beside it is zero: x is kept finite for that product.
__device__ __forceinline__ float activate(float x, int act) {
  if (act == IS_ACT_RELU) return x < 0.f ? 0.f : x;     // NaN stays
  if (act == IS_ACT_GELU) {
    const float z = fminf(fabsf(x), 14.f), t = __builtin_amdgcn_rcpf(1.f + 0.31f * z);
    float r = -0.07392936f;
    r = r * t + 0.18045098f;
    r = r * t + 0.01574401f;
    r = r * t + 0.13343013f;
    r = r * t + 0.1204412f;
    r = r * t + 0.12386071f;
    const float tail = z * t * r * __builtin_amdgcn_exp2f(-0.72134752f * z * z);
    return (x < 0.f ? 0.f : x) - tail;
  }
  if (act == IS_ACT_GELU_TANH) {
    const float u = 1.5957691216f * (x + 0.044715f * x * x * x);    // 2 sqrt(2 / pi)
    return fmaxf(x, -3.4e38f) * sigmoid(u);
  }
  if (act == IS_ACT_SILU) return fmaxf(x, -3.4e38f) * sigmoid(x);
  return x;
}

// The end of 8 features f .. f + 7 of a row: z the sums. Rows may lie at any element.
template <typename T>
__device__ __forceinline__ void finish8(const Args &a, const float (&z)[8], const float (&bias)[8], const T *residual,
                                        T *out, int f) {
  typedef T uvec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  typedef T vec __attribute__((ext_vector_type(8)));
  const bool whole = f + 8 <= a.features;
  vec r = {};
  if (residual) {
    if (whole) {
      r = *reinterpret_cast<const uvec *>(residual + f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (f + j < a.features) r[j] = residual[f + j];
    }
  }
  vec o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (T)((float)r[j] + activate(z[j] + bias[j], a.act));
  if (whole) {
    *reinterpret_cast<uvec *>(out + f) = o;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (f + j < a.features) out[f + j] = o[j];
  }
}

template <int FB, int TB, int WF, int WT>
struct Tile {
  static constexpr int NW = WF * WT, TF = 32 * FB * WF, TT = 32 * TB * WT;
  static constexpr int ROW = 128;                          // bytes of a row of a step
  static constexpr int NI_W = TF / 8 / NW, NI_X = TT / 8 / NW;   // 1 KB loads of a wave and step
  static constexpr int W_BYTES = TF * ROW, STAGE = (TF + TT) * ROW, BYTES = 2 * STAGE;
  static constexpr int OUT = 32 * 32 * FB * 4;             // a wave's results of 32 tokens, fp32
  static_assert(NI_W * 8 * NW == TF && NI_X * 8 * NW == TT, "whole loads");
  static_assert(NW * OUT <= BYTES, "results pass the buffers");
};

template <typename T, int FB, int TB, int WF, int WT>
__global__ __launch_bounds__(WF *WT * 64, WF *WT == 8 ? 2 : 2) void is_k13_dense(const Args a) {
  using G = Tile<FB, TB, WF, WT>;
  typedef T T8 __attribute__((ext_vector_type(8)));
  __shared__ __attribute__((aligned(1024))) char lds[G::BYTES];
  lds_poison(lds, sizeof(lds));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n32 = lane & 31, half = lane >> 5, wf = wave % WF, wt = wave / WF;

  // Workgroup -> (part of the sum, entry, row tile, feature tile): an XCD's
  // workgroups take neighbouring tiles, features first within 8 row tiles.
  int place = xcd_remap(blockIdx.x, gridDim.x);
  const int tiles = a.row_tiles * a.feature_tiles;
  const int group = place / tiles;
  place -= group * tiles;
  const int entry = group / a.splits, split = group - entry * a.splits;
  const int span = 8 * a.feature_tiles, first = place / span * 8, high = min(8, a.row_tiles - first);
  const int in_span = place - first * a.feature_tiles;
  const int rt = first + in_span % high, ft = in_span / high;

  const int in0 = split * a.split_in, in1 = min(a.in, in0 + a.split_in);
  const int steps = (in1 - in0 + 63) / 64;
  const T *x = static_cast<const T *>(a.x) + entry * a.xb + (int64_t)rt * G::TT * a.xr + in0;
  const T *w = static_cast<const T *>(a.w) + (int64_t)ft * G::TF * a.wr + in0;

  // Loads of this wave: operation i brings rows 8 (wave NI + i) .. + 7.
  unsigned wo[G::NI_W], xo[G::NI_X];
  const int r8 = lane >> 3;
  int wc[G::NI_W], xc[G::NI_X];
#pragma unroll
  for (int i = 0; i < G::NI_W; ++i) {
    const int r = (wave * G::NI_W + i) * 8 + r8;
    wc[i] = (lane & 7) ^ ((r >> 1) & 7);
    wo[i] = ft * G::TF + r < a.features ? (unsigned)(r * (int)a.wr * 2 + wc[i] * 16) : kOutside;
  }
#pragma unroll
  for (int i = 0; i < G::NI_X; ++i) {
    const int r = (wave * G::NI_X + i) * 8 + r8;
    xc[i] = (lane & 7) ^ ((r >> 1) & 7);
    xo[i] = rt * G::TT + r < a.len ? (unsigned)(r * (int)a.xr * 2 + xc[i] * 16) : kOutside;
  }
  const unsigned lds_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
  auto issue = [&](int t) {
    if (t >= steps) return;
    const int left = (in1 - in0 - t * 64) / 8;        // chunks of a row that exist
    const uint64_t wat = (uint64_t)(uintptr_t)w + (uint64_t)t * G::ROW, xat = (uint64_t)(uintptr_t)x + (uint64_t)t * G::ROW;
    const unsigned at = lds_at + (unsigned)((t & 1) * G::STAGE);
    if (left >= 8) {
      load_lds16<G::NI_W>(buffer_at(wat, 0x80000000u), at + wave * G::NI_W * 1024, wo);
      load_lds16<G::NI_X>(buffer_at(xat, 0x80000000u), at + G::W_BYTES + wave * G::NI_X * 1024, xo);
    } else {
      unsigned o[G::NI_W], p[G::NI_X];
#pragma unroll
      for (int i = 0; i < G::NI_W; ++i) o[i] = wc[i] < left ? wo[i] : kOutside;
#pragma unroll
      for (int i = 0; i < G::NI_X; ++i) p[i] = xc[i] < left ? xo[i] : kOutside;
      load_lds16<G::NI_W>(buffer_at(wat, 0x80000000u), at + wave * G::NI_W * 1024, o);
      load_lds16<G::NI_X>(buffer_at(xat, 0x80000000u), at + G::W_BYTES + wave * G::NI_X * 1024, p);
    }
  };

  const int turn = (n32 >> 1) & 7;
  const char *wl = lds + (wf * 32 * FB + n32) * G::ROW, *xl = lds + G::W_BYTES + (wt * 32 * TB + n32) * G::ROW;
  T8 fw[2][FB], fx[2][TB];
  floatx16 acc[FB][TB];
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  auto read = [&](int t, int kk, int to) {
    const int at = (t & 1) * G::STAGE + (((2 * kk + half) ^ turn) << 4);
#pragma unroll
    for (int i = 0; i < FB; ++i) fw[to][i] = *reinterpret_cast<const T8 *>(wl + at + i * 32 * G::ROW);
#pragma unroll
    for (int j = 0; j < TB; ++j) fx[to][j] = *reinterpret_cast<const T8 *>(xl + at + j * 32 * G::ROW);
  };
  auto products = [&](int from) {
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j) acc[i][j] = mma32(fw[from][i], fx[from][j], acc[i][j]);
  };

  issue(0);
  issue(1);
  if (steps > 1) loads_left<G::NI_W + G::NI_X>();
  else loads_left<0>();
  lds_barrier();
  read(0, 0, 0);
  for (int t = 0; t < steps; ++t) {
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) {
      read(t, kk + 1, (kk + 1) & 1);
      products(kk & 1);
    }
    loads_left<0>();       // the next step has arrived (this wave's part)
    lds_barrier();         // and everyone's; this step's operands are all in registers
    issue(t + 2);
    if (t + 1 < steps) read(t + 1, 0, 0);
    products(1);
  }
  lds_barrier();

  // Results: lane = token n32 of block j, features 32 i + 8 u + 4 half + (0..3).
  constexpr int CHUNKS = 8 * FB;                  // 16-byte chunks of a token's row
  char *mine = lds + wave * G::OUT;
  auto slot = [](int c, int token) { return (c ^ (CHUNKS >= 16 ? token & 15 : (token >> 1) & 7)) << 4; };
  constexpr int LPR = 4 * FB, RPI = 64 / LPR;     // lanes of a row, rows an instruction
  const int col = lane % LPR, f = ft * G::TF + wf * 32 * FB + col * 8;
  float bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = a.bias && f + e < a.features ? a.bias[f + e] : 0.f;
#pragma unroll
  for (int j = 0; j < TB; ++j) {
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<floatx4 *>(mine + n32 * CHUNKS * 16 + slot(8 * i + 2 * u + half, n32)) =
            floatx4{acc[i][j][4 * u], acc[i][j][4 * u + 1], acc[i][j][4 * u + 2], acc[i][j][4 * u + 3]};
    __asm__ volatile("" ::: "memory");
    const int row0 = rt * G::TT + (wt * TB + j) * 32;
#pragma unroll 2
    for (int s = 0; s < 32 / RPI; ++s) {
      const int token = s * RPI + lane / LPR, row = row0 + token;
      float z[8];
      *reinterpret_cast<floatx4 *>(z) = *reinterpret_cast<const floatx4 *>(mine + token * CHUNKS * 16 + slot(2 * col, token));
      *reinterpret_cast<floatx4 *>(z + 4) =
          *reinterpret_cast<const floatx4 *>(mine + token * CHUNKS * 16 + slot(2 * col + 1, token));
      if (row >= a.len || f >= a.features) continue;
      if (a.splits > 1) {
        float *p = a.part + (((int64_t)split * a.entries + entry) * a.len + row) * a.features + f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (f + e < a.features) p[e] = z[e];
      } else {
        const T *res = a.residual ? static_cast<const T *>(a.residual) + entry * a.rb + row * a.rr : nullptr;
        finish8<T>(a, z, bias, res, static_cast<T *>(a.out) + entry * a.ob + row * a.orow, f);
      }
    }
    __asm__ volatile("" ::: "memory");
  }
}

// Adds the parts of 8 features of a row.
template <typename T>
__global__ __launch_bounds__(256) void is_k13_dense_join(const Args a, int64_t items) {
  const int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  const int groups = (a.features + 7) / 8, f = (int)(it % groups) * 8;
  const int64_t r = it / groups, entry = r / a.len, row = r - entry * a.len;
  const int64_t step = (int64_t)a.entries * a.len * a.features;
  const float *p = a.part + r * a.features + f;
  float z[8] = {}, bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = a.bias && f + e < a.features ? a.bias[f + e] : 0.f;
  for (int s = 0; s < a.splits; ++s) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (f + e < a.features) z[e] += p[s * step + e];
  }
  const T *res = a.residual ? static_cast<const T *>(a.residual) + entry * a.rb + row * a.rr : nullptr;
  finish8<T>(a, z, bias, res, static_cast<T *>(a.out) + entry * a.ob + row * a.orow, f);
}

// Few rows: FB blocks of 16 features x TB blocks of 16 rows, NW waves that take
// chunks of 32 inputs in turn, U of them in flight each.
template <typename T, int FB, int TB, int NW, int U>
__global__ __launch_bounds__(NW * 64) void is_k13_dense_few(const Args a) {
  typedef T T8 __attribute__((ext_vector_type(8)));
  constexpr int JOIN = FB * TB * 64 * 16;      // bytes of a wave's sums
  __shared__ __attribute__((aligned(16))) char lds[NW * JOIN];
  lds_poison(lds, sizeof(lds));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, quarter = lane >> 4;
  const int ft = blockIdx.x % a.feature_tiles, rest = blockIdx.x / a.feature_tiles;
  const int rt = rest % a.row_tiles, entry = rest / a.row_tiles;
  const int f0 = ft * 16 * FB, r0 = rt * 16 * TB;
  const T *w = static_cast<const T *>(a.w) + (int64_t)f0 * a.wr;
  const T *x = static_cast<const T *>(a.x) + entry * a.xb + (int64_t)r0 * a.xr;

  floatx4 acc[FB][TB];
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int chunks = (a.in + 31) / 32;
  // Rows that do not exist are read from the last one that does, and their sums
  // dropped; inputs past the end are zeros in both operands.
  int64_t wo[FB], xo[TB];
#pragma unroll
  for (int i = 0; i < FB; ++i) wo[i] = (int64_t)min(i * 16 + n16, a.features - 1 - f0) * a.wr + quarter * 8;
#pragma unroll
  for (int j = 0; j < TB; ++j) xo[j] = (int64_t)min(j * 16 + n16, a.len - 1 - r0) * a.xr + quarter * 8;
  for (int c0 = wave * U; c0 < chunks; c0 += NW * U) {
    T8 fw[U][FB], fx[U][TB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = (c0 + u) * 32 + quarter * 8 < a.in;
#pragma unroll
      for (int i = 0; i < FB; ++i)
        fw[u][i] = in ? *reinterpret_cast<const T8 *>(w + wo[i] + (c0 + u) * 32) : T8{};
#pragma unroll
      for (int j = 0; j < TB; ++j)
        fx[u][j] = in ? *reinterpret_cast<const T8 *>(x + xo[j] + (c0 + u) * 32) : T8{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = mma16(fw[u][i], fx[u][j], acc[i][j]);
  }

  // Join: lane = row n16 of block j, features 16 i + 4 quarter + (0..3).
  floatx4 *sums = reinterpret_cast<floatx4 *>(lds);
#pragma unroll
  for (int i = 0; i < FB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) sums[((wave * FB + i) * TB + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int it = threadIdx.x; it < FB * TB * 64; it += NW * 64) {
    floatx4 z = sums[it];
#pragma unroll
    for (int v = 1; v < NW; ++v) z += sums[v * FB * TB * 64 + it];
    const int l = it & 63, ij = it >> 6, i = ij / TB, j = ij % TB;
    const int row = r0 + j * 16 + (l & 15), f = f0 + i * 16 + (l >> 4) * 4;
    if (row >= a.len) continue;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + entry * a.rb + row * a.rr : nullptr;
    T *out = static_cast<T *>(a.out) + entry * a.ob + row * a.orow;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f + e < a.features)
        out[f + e] = (T)((res ? (float)res[f + e] : 0.f) + activate(z[e] + (a.bias ? a.bias[f + e] : 0.f), a.act));
  }
}

struct TileShape {
  int features, rows, waves, lds;
};
template <int FB, int TB, int WF, int WT>
constexpr TileShape shape() {
  using G = Tile<FB, TB, WF, WT>;
  return {G::TF, G::TT, G::NW, G::BYTES};
}
constexpr TileShape kTiles[] = {shape<4, 2, 2, 4>(), shape<2, 2, 2, 2>(), shape<1, 1, 2, 2>()};

constexpr int kFewWaves = 8, kFewAhead = 4;

template <typename T>
hipError_t launch_t(const DensePlan &p, const Args &a, hipStream_t s) {
  const unsigned blocks = (unsigned)((int64_t)a.entries * p.row_tiles * p.feature_tiles * p.splits);
  if (p.few) {
    if (p.tile == 1) return launch_kernel(is_k13_dense_few<T, 1, 1, kFewWaves, kFewAhead>, dim3(blocks), dim3(p.block), 0, s, a);
    return launch_kernel(is_k13_dense_few<T, 2, 2, kFewWaves, kFewAhead>, dim3(blocks), dim3(p.block), 0, s, a);
  }
  hipError_t e;
  switch (p.tile) {
    case 0: e = launch_kernel(is_k13_dense<T, 4, 2, 2, 4>, dim3(blocks), dim3(p.block), 0, s, a); break;
    case 1: e = launch_kernel(is_k13_dense<T, 2, 2, 2, 2>, dim3(blocks), dim3(p.block), 0, s, a); break;
    default: e = launch_kernel(is_k13_dense<T, 1, 1, 2, 2>, dim3(blocks), dim3(p.block), 0, s, a); break;
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t items = (int64_t)a.entries * a.len * ((a.features + 7) / 8);
  return launch_kernel(is_k13_dense_join<T>, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a, items);
}

}  // namespace

bool configure_dense(DensePlan &p) {
  dense_desc &d = p.d;
  // Entries whose rows follow each other at one distance are one.
  auto flat = [&](const int64_t *s) { return d.n <= 1 || d.len == 1 || s[0] == (int64_t)d.len * s[1]; };
  if (flat(d.x_stride) && flat(d.residual_stride) && flat(d.out_stride) && d.n > 0 && d.len > 0 &&
      (double)d.n * d.len < 2147483000.0) {
    if (d.len == 1)
      for (int64_t *s : {d.x_stride, d.residual_stride, d.out_stride}) s[1] = s[0];
    d.len *= d.n;
    d.n = 1;
  }
  p.splits = 1;
  p.split_in = (d.in + 63) / 64 * 64;
  p.few = d.len <= 32;
  if (p.few) {
    p.tile = d.len <= 16 ? 1 : 2;
    p.tile_rows = p.tile_features = 16 * p.tile;
    p.block = 64 * kFewWaves;
    p.lds = kFewWaves * p.tile * p.tile * 1024;
    p.name = "is_k13_dense_few";
  } else {
    auto tiles = [&](int i) {
      return (double)d.n * ceil((double)d.len / kTiles[i].rows) * ceil((double)d.features / kTiles[i].features);
    };
    p.tile = tiles(0) >= 200 ? 0 : tiles(1) >= 256 ? 1 : 2;
    p.tile_rows = kTiles[p.tile].rows;
    p.tile_features = kTiles[p.tile].features;
    p.block = 64 * kTiles[p.tile].waves;
    p.lds = kTiles[p.tile].lds;
    p.name = "is_k13_dense";
  }
  p.row_tiles = (d.len + p.tile_rows - 1) / p.tile_rows;
  p.feature_tiles = (d.features + p.tile_features - 1) / p.tile_features;
  return (double)d.n * p.row_tiles * p.feature_tiles * p.splits * p.block <= kMaxLaunchThreads;
}

size_t dense_workspace(const DensePlan &p) {
  return p.splits == 1 ? 0 : (size_t)p.splits * p.d.n * p.d.len * p.d.features * 4;
}

hipError_t launch_dense(const DensePlan &p, const void *x, const void *w, const float *bias, const void *residual,
                        void *out, void *ws, hipStream_t s) {
  const dense_desc &d = p.d;
  Args a;
  a.x = x;
  a.w = w;
  a.residual = residual;
  a.bias = bias;
  a.out = out;
  a.part = static_cast<float *>(ws);
  a.xb = d.x_stride[0];
  a.xr = d.x_stride[1];
  a.rb = d.residual_stride[0];
  a.rr = d.residual_stride[1];
  a.ob = d.out_stride[0];
  a.orow = d.out_stride[1];
  a.wr = d.w_stride;
  a.entries = d.n;
  a.len = d.len;
  a.in = d.in;
  a.features = d.features;
  a.act = d.activation;
  a.splits = p.splits;
  a.split_in = p.split_in;
  a.row_tiles = (int)p.row_tiles;
  a.feature_tiles = (int)p.feature_tiles;
  return d.dtype == IS_F16 ? launch_t<_Float16>(p, a, s) : launch_t<__bf16>(p, a, s);
}

}  // namespace is

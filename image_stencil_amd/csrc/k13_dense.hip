// k13_dense.hip -- dense layers on tokens:  out = residual + act(x w^T + bias).
//
// Weights are the first operand of the matrix instructions and tokens the second,
// so that a lane's results are consecutive features of one token.
//
// Many rows (is_k13_dense): a workgroup of WF x WT waves computes tiles of 32 FB WF
// features x 32 TB WT tokens with v_mfma_f32_32x32x16, one after another. A step is 64
// inputs of both operands, brought to LDS by DMA without passing registers: a
// 128-byte row in 8 chunks of 16 bytes, chunk c of row r in slot c ^ ((r >> 1) & 7),
// so that 16 lanes reading one chunk of 16 rows meet 16 different bank groups. The
// weights' and the tokens' halves of the steps go round five LDS slots, which keeps loads
// one and a half steps ahead, also from one tile to the next. The last quarter of a step
// runs after the barrier that frees its slots: its products cover the first operand reads
// of the next step. Results pass the one free slot as fp32, a wave's own part, so that
// residual and output are touched by 4 lanes a token. Their stores have the first step of
// the next tile to complete in: the wait at its end leaves only that step's own loads open.
//
// Few rows (is_k13_dense_few): the weights are read once, straight into registers,
// 16 features x 32 inputs an instruction (v_mfma_f32_16x16x32); the waves of a
// workgroup take the inner sum in turn and join in LDS.
//
// What bounds it, measured on several MI355Xs (bf16, inputs changing from call to call):
// 65536 rows, 4096 to 1024, with residual: 448 to 468 us, 1.17 to 1.23 PFLOP/s, matrix cores
// 67% busy; 8192 cubed 804 to 841, 1.31 to 1.37 PFLOP/s, 77% busy at 1.4 to 1.7 GHz, which
// the power limit sets (a library product without residual: 376 and 688). Two 3600-token
// frames, 512 to 2048: 21.6 to 22.9 us without an activation, ReLU 0.3 more, SiLU 3.3,
// tanh-GELU 3.8, GELU 5.6 to 6.1 (an end that knows of no residual and shorter activations:
// 23.5, 24.1, 26.4, 27.3, 30.5 before, 22.9, 23.2, 26.2, 26.7, 29.0 after); 8 steps are 12.4 of
// it, the write of a whole tile per CU much of the rest. 16 rows, 8192 to 8192: 33, 4.1 TB/s
// (one row 28 to 30; a library product of 16 rows 29 to 30): the 16 rows of x, read again by
// each workgroup, are as many requests as half the weights.
// Steps that were taken back: touching the lines of later steps (a dword of each, 892 to
// 1050); both quarters of an accumulator's half step one after the other (841 to 874); weights
// of few rows past the caches (33.6 to 35.9: an instruction takes half of each line).
#include <math.h>

#include "blocks.hpp"
#include "common.hpp"
#include "divide.hpp"
#include "dma.hpp"
#include "internal.hpp"

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
  float *part;             // splits > 1: sums of the parts, [split][entry][row][part_row]
  int64_t xb, xr, rb, rr, ob, orow, wr;
  int entries, len, in, features, act;
  int splits, split_in, part_row;      // part_row: features, rounded up to 8
  int row_tiles, feature_tiles, units;    // units: tiles of all entries and parts
  Divisor by_tiles, by_splits, by_span, by_last;   // tiles of an entry, of 8 row tiles; row tiles mod 8
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

// x / (1 + 2^u). Where the exponential overflows, the quotient is zero: x is kept finite
// for the product.
__device__ __forceinline__ float over(float x, float u) {
  return fmaxf(x, -3.4e38f) * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u));
}

// GELU is x Phi(x) = max(x, 0) - |x| Phi(-|x|), with Phi(-z) = exp(-z^2 / 2) R(z) and R a
// polynomial in t = 1 / (1 + 0.31 z), fitted to erfcx(z / sqrt 2) / 2 on 0 <= z <= 14:
// within 4.7e-6 of it everywhere, a hundredth of fp16's half step, so that small
// results at far negative x keep their digits. NaN stays NaN in all. (Every instruction
// counts: for the 65536 results of a CU's tile one takes 0.4 us.)
template <int ACT>
__device__ __forceinline__ float activated(float x) {
  if constexpr (ACT == IS_ACT_RELU) return __builtin_elementwise_maximum(x, 0.f);
  if constexpr (ACT == IS_ACT_GELU) {
    const float z = __builtin_elementwise_minimum(fabsf(x), 14.f), t = __builtin_amdgcn_rcpf(1.f + 0.31f * z);
    float r = -0.07392936f;
    r = r * t + 0.18045098f;
    r = r * t + 0.01574401f;
    r = r * t + 0.13343013f;
    r = r * t + 0.1204412f;
    r = r * t + 0.12386071f;
    return fmaxf(x, 0.f) - z * (t * r * __builtin_amdgcn_exp2f(-0.72134752f * z * z));
  }
  if constexpr (ACT == IS_ACT_GELU_TANH) {      // x / (1 + exp(-2 sqrt(2 / pi) (x + 0.044715 x^3)))
    return over(x, x * (-0.10294324f * (x * x) - 2.3022082f));
  }
  if constexpr (ACT == IS_ACT_SILU) return over(x, -1.4426950408889634f * x);
  return x;
}
// Calls f(std::integral_constant<int, activation>{}).
template <typename F>
__device__ __forceinline__ void for_activation(int act, F &&f) {
  switch (act) {
    case IS_ACT_RELU: return f(std::integral_constant<int, IS_ACT_RELU>{});
    case IS_ACT_GELU: return f(std::integral_constant<int, IS_ACT_GELU>{});
    case IS_ACT_GELU_TANH: return f(std::integral_constant<int, IS_ACT_GELU_TANH>{});
    case IS_ACT_SILU: return f(std::integral_constant<int, IS_ACT_SILU>{});
    default: return f(std::integral_constant<int, IS_ACT_NONE>{});
  }
}
__device__ __forceinline__ float activate(float x, int act) {
  for_activation(act, [&](auto kind) { x = activated<decltype(kind)::value>(x); });
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
  static constexpr int NI = TF / 8 / NW;                   // 1 KB loads of a wave, step and operand
  static constexpr int SLOT = TF * ROW, SLOTS = 5;
  // Results on their way out lie where the wave's own loads go: 32 features of 32 or 16
  // tokens at a time, fp32.
  static constexpr int OUT_TOKENS = NI * 1024 / 128;
  static constexpr int BYTES = SLOTS * SLOT;
  static constexpr int GROUPS = 160 * 1024 / BYTES;        // a CU
  static_assert(TF == TT && NI * 8 * NW == TF, "whole loads, operands alike");
  static_assert(OUT_TOKENS == 32 || OUT_TOKENS == 16, "passes of the results");
};

template <typename T, int FB, int TB, int WF, int WT>
__global__ __launch_bounds__(WF *WT * 64, 2) void is_k13_dense(const Args a) {
  using G = Tile<FB, TB, WF, WT>;
  typedef T T8 __attribute__((ext_vector_type(8)));
  __shared__ __attribute__((aligned(1024))) char lds[G::BYTES];
  lds_poison(lds, sizeof(lds));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n32 = lane & 31, half = lane >> 5, wf = wave % WF, wt = wave / WF;

  // An XCD's workgroups share one range of tiles and take them in turn: what they work
  // on at a time lies together.
  const int lo = (int)((int64_t)a.units * (blockIdx.x & 7) / 8), hi = (int)((int64_t)a.units * ((blockIdx.x & 7) + 1) / 8);
  const int stride = ((int)gridDim.x - (int)(blockIdx.x & 7) + 7) / 8;
  struct Place {
    int entry, split, rt, ft, in0, in1;
  };
  // Unit -> (part of the sum, entry, row tile, feature tile), features first within 8
  // row tiles.
  auto place_of = [&](int unit) {
    Place p;
    const int group = divide(unit, a.by_tiles), rest = unit - group * a.row_tiles * a.feature_tiles;
    p.entry = divide(group, a.by_splits);
    p.split = group - p.entry * a.splits;
    const int first = divide(rest, a.by_span) * 8, in_span = rest - first * a.feature_tiles;
    const int high = min(8, a.row_tiles - first);
    p.ft = high == 8 ? in_span >> 3 : divide(in_span, a.by_last);
    p.rt = first + in_span - p.ft * high;
    p.in0 = p.split * a.split_in;
    p.in1 = p.in0 + min(a.in - p.in0, a.split_in);      // (in0 + split_in may pass an int)
    return p;
  };
  auto steps_of = [](const Place &p) { return (p.in1 - p.in0 + 63) / 64; };

  // ---- Loads, across tiles. Operation i of this wave brings rows 8 (wave NI + i) .. + 7
  // of an operand's step. W of step t is half 2 t and X half 2 t + 1 of a stream that
  // goes round the five slots: while the products of step t run, both halves of t + 1
  // and W of t + 2 are there or on their way; the end of step t, which frees two slots,
  // asks for X of t + 2 and the start of step t + 1 for W of t + 3.
  constexpr int NI = G::NI;
  // The lane, as a value that the compiler cannot compute with ahead of a loop: what
  // follows from it would take registers throughout.
  auto fresh_lane = [&] {
    int l = lane;
    __asm__ volatile("" : "+v"(l));
    return l;
  };
  auto row_of = [&](int i, int l) { return (wave * NI + i) * 8 + (l >> 3); };
  auto chunk_of = [&](int i, int l) { return (l & 7) ^ ((row_of(i, l) >> 1) & 7); };     // of its row
  const unsigned lds_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)lds + wave * NI * 1024;
  struct Cursor {
    int unit, left, slot;      // the tile asked for, its inputs to come; bytes
    uint64_t at;
    unsigned off[NI];
    uintx4 rs;
  };
  auto tile = [&](Cursor &c, bool of_w) {
    // Past the last tile: loads without bytes, which only clear LDS.
    const Place p = place_of(min(c.unit, hi - 1));
    c.left = c.unit < hi ? p.in1 - p.in0 : 0;
    c.at = of_w ? (uint64_t)(uintptr_t)(static_cast<const T *>(a.w) + (int64_t)p.ft * G::TF * a.wr + p.in0)
                : (uint64_t)(uintptr_t)(static_cast<const T *>(a.x) + p.entry * a.xb + (int64_t)p.rt * G::TT * a.xr + p.in0);
    const int rows = of_w ? a.features - p.ft * G::TF : a.len - p.rt * G::TT, step = (int)(of_w ? a.wr : a.xr) * 2;
    // (Not a loop: the compiler would keep the array in memory and the cursor with it.)
    const int l = fresh_lane();
    static_for<NI>([&](auto i) {
      c.off[i] = row_of(i, l) < rows ? (unsigned)(row_of(i, l) * step + chunk_of(i, l) * 16) : kOutside;
    });
  };
  // Points a cursor to its next step; a tile's last step may end inside a row.
  auto next = [&](Cursor &c, bool of_w) {
    if (c.left <= 0) {
      c.unit += stride;
      tile(c, of_w);
    }
    if (c.left > 0 && c.left < 64) {
      const int l = fresh_lane();
      static_for<NI>([&](auto i) { c.off[i] = chunk_of(i, l) * 8 < c.left ? c.off[i] : kOutside; });
    }
    c.rs = buffer_at(c.at, c.left > 0 ? 0x80000000u : 0u);
    c.at += G::ROW;
    c.left -= 64;
    c.slot += 2 * G::SLOT;
    if (c.slot >= G::SLOTS * G::SLOT) c.slot -= G::SLOTS * G::SLOT;
  };
  auto ask = [&](const Cursor &c, auto op) {      // operation op of the step
    constexpr int I = decltype(op)::value;
    load_lds16<1>(c.rs, __builtin_amdgcn_readfirstlane(lds_at + c.slot + I * 1024), c.off + I);
  };

  // ---- Products.
  const int turn = (n32 >> 1) & 7;
  const char *wl = lds + (wf * 32 * FB + n32) * G::ROW, *xl = lds + (wt * 32 * TB + n32) * G::ROW;
  T8 fw[2][FB], fx[2][TB];
  floatx16 acc[FB][TB];
  // Operand o of quarter kk of the step in the slots ws and xs, tokens first.
  auto read = [&](int ws, int xs, int kk, auto o) {
    constexpr int O = decltype(o)::value;
    const int at = ((2 * kk + half) ^ turn) << 4;
    if constexpr (O < TB) fx[kk & 1][O] = *reinterpret_cast<const T8 *>(xl + xs + at + O * 32 * G::ROW);
    else fw[kk & 1][O - TB] = *reinterpret_cast<const T8 *>(wl + ws + at + (O - TB) * 32 * G::ROW);
  };
  constexpr int PRODUCTS = FB * TB, OPERANDS = FB + TB;
  // The products of a quarter, one at a time, and what `beside` puts after each of them.
  auto products = [&](int kk, auto &&beside) {
    static_for<PRODUCTS>([&](auto u) {
      constexpr int U = decltype(u)::value;
      acc[U / TB][U % TB] = mma32(fw[kk & 1][U / TB], fx[kk & 1][U % TB], acc[U / TB][U % TB]);
      beside(u);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // Operands or loads dealt to the products: those of slot u.
  auto deal = [](auto u, auto count, auto slots, auto &&f) {
    constexpr int U = decltype(u)::value, N = decltype(count)::value, S = decltype(slots)::value;
    constexpr int PER = (N + S - 1) / S;
    static_for<PER>([&](auto i) {
      constexpr int I = U * PER + decltype(i)::value;
      if constexpr (I < N) f(std::integral_constant<int, I>{});
    });
  };
  using Operands = std::integral_constant<int, OPERANDS>;
  using Loads = std::integral_constant<int, NI>;
  using Slots = std::integral_constant<int, PRODUCTS>;
  using Early = std::integral_constant<int, (PRODUCTS + 1) / 2>;

  // ---- Results: lane = token n32 of block j, features 32 i + 8 u + 4 half + (0..3). A
  // wave brings 32 features of 32 tokens at a time through LDS, so that residual and
  // output are touched by 4 lanes a token.
  auto slot = [](int c, int token) { return token * 128 + ((c ^ ((token >> 1) & 7)) << 4); };
  // Before tokens 16 s .. of block j are taken back: all 32 with the first 16 if they fit.
  auto stage = [&](auto i, auto j, auto s, char *mine, int l) {
    if constexpr (G::OUT_TOKENS == 32 && s == 1) return;
    __asm__ volatile("" ::: "memory");
    if (G::OUT_TOKENS == 32 || (l >> 4 & 1) == s) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<floatx4 *>(mine + slot(2 * e + (l >> 5), l & (G::OUT_TOKENS - 1))) =
            floatx4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
    }
    __asm__ volatile("" ::: "memory");
  };
  // Back: 4 lanes a token (lane & 3: which 8 features), 16 tokens at a time.
  auto unstage = [&](int s, const char *mine, float (&z)[8], int l) {
    const int token = (16 * s + (l >> 2)) & (G::OUT_TOKENS - 1), col = l & 3;
    *reinterpret_cast<floatx4 *>(z) = *reinterpret_cast<const floatx4 *>(mine + slot(2 * col, token));
    *reinterpret_cast<floatx4 *>(z + 4) = *reinterpret_cast<const floatx4 *>(mine + slot(2 * col + 1, token));
  };
  // The residual of 32 tokens is asked for at once, and that of the next 32 before the
  // stores of these, since loads wait for the stores before them. The bias is one value
  // a lane, and reaches the lanes that need it by permutes.
  auto finish = [&](const Place &p, char *mine, auto kind, auto with_residual) {
    constexpr int ACT = decltype(kind)::value;
    constexpr bool RES = decltype(with_residual)::value;
    typedef T uvec __attribute__((ext_vector_type(8), aligned(sizeof(T))));   // at any element
    const int l = fresh_lane(), col = l & 3;
    const int f = p.ft * G::TF + wf * 32 * FB, row0 = p.rt * G::TT + wt * 32 * TB + (l >> 2);
    const T *res = static_cast<const T *>(a.residual) + p.entry * a.rb + f + col * 8;
    T *out = static_cast<T *>(a.out) + p.entry * a.ob + f + col * 8;
    const int left = a.features - f - col * 8;        // features from this lane's first on
    float bias[(FB + 1) / 2];
    static_for<(FB + 1) / 2>([&](auto i) {
      const int e = 64 * i + l;
      bias[i] = a.bias && e < 32 * FB && f + e < a.features ? a.bias[f + e] : 0.f;
    });
    // Also the results' place: r of this block of tokens, then of the next.
    T8 r[2][FB][2];
    auto ask_residual = [&](auto j) {
      static_for<2 * FB>([&](auto u) {
        constexpr int I = decltype(u)::value >> 1;
        const int row = row0 + j * 32 + 16 * (u & 1);
        T8 &x = r[j & 1][I][u & 1];
        x = T8{};
        if (row >= a.len) return;
        const T *at = res + row * a.rr + I * 32;
        if (left >= I * 32 + 8) {
          x = *reinterpret_cast<const uvec *>(at);
        } else {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (I * 32 + e < left) x[e] = at[e];
        }
      });
    };
    if constexpr (RES) ask_residual(std::integral_constant<int, 0>{});
    static_for<TB>([&](auto j) {
      static_for<FB>([&](auto i) {
        float b[8];
        __asm__ volatile("" : "+v"(bias[i / 2]));     // permuted anew for every block: fewer registers
#pragma unroll
        for (int e = 0; e < 8; ++e)
          b[e] = __int_as_float(__builtin_amdgcn_ds_bpermute(((32 * (int)i + 8 * col + e) & 63) * 4,
                                                             __float_as_int(bias[i / 2])));
        static_for<2>([&](auto s) {
          float z[8];
          stage(i, j, s, mine, l);
          unstage(s, mine, z, l);
          T8 &x = r[j & 1][i][s];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = activated<ACT>(z[e] + b[e]);
            x[e] = (T)(RES ? (float)x[e] + y : y);
          }
          // Computed here, not beside its store, up to which every sum would be kept.
          uintx4 bits = __builtin_bit_cast(uintx4, x);
          __asm__ volatile("" : "+v"(bits));
          x = __builtin_bit_cast(T8, bits);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (RES && j + 1 < TB) ask_residual(std::integral_constant<int, j + 1>{});
      static_for<2 * FB>([&](auto u) {
        constexpr int I = decltype(u)::value >> 1;
        const int row = row0 + j * 32 + 16 * (u & 1);
        if (row >= a.len) return;
        const T8 &x = r[j & 1][I][u & 1];
        T *at = out + row * a.orow + I * 32;
        if (left >= I * 32 + 8) {
          *reinterpret_cast<uvec *>(at) = x;
        } else {
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (I * 32 + e < left) at[e] = x[e];
        }
      });
    });
  };
  // A part of a split sum, as it is.
  auto finish_part = [&](const Place &p, char *mine) {
    const int l = fresh_lane(), f = p.ft * G::TF + wf * 32 * FB + (l & 3) * 8;
    const int row0 = p.rt * G::TT + wt * 32 * TB + (l >> 2);
    float *to = a.part + ((int64_t)p.split * a.entries + p.entry) * a.len * a.part_row + f;
    static_for<FB * TB>([&](auto u) {
      constexpr int I = decltype(u)::value / TB, J = decltype(u)::value % TB;
      static_for<2>([&](auto s) {
        const int row = row0 + J * 32 + 16 * s;
        float z[8];
        stage(std::integral_constant<int, I>{}, std::integral_constant<int, J>{}, s, mine, l);
        unstage(s, mine, z, l);
        if (row < a.len && f + I * 32 < a.part_row) {
          floatx4 *at = reinterpret_cast<floatx4 *>(to + (int64_t)row * a.part_row + I * 32);
          at[0] = *reinterpret_cast<const floatx4 *>(z);
          at[1] = *reinterpret_cast<const floatx4 *>(z + 4);
        }
      });
    });
  };

  int unit = lo + (int)(blockIdx.x >> 3);
  if (unit >= hi) return;      // whole workgroups leave
  Cursor w, x;
  w.unit = x.unit = unit;
  w.slot = -2 * G::SLOT;
  x.slot = -G::SLOT;
  tile(w, true);
  tile(x, false);
  auto ask_all = [&](const Cursor &c) { static_for<NI>([&](auto i) { ask(c, i); }); };
  next(w, true), ask_all(w);
  next(x, false), ask_all(x);
  next(w, true), ask_all(w);
  next(x, false), ask_all(x);
  loads_left<2 * NI>();
  lds_barrier();
  int ws = 0, xs = G::SLOT;
  static_for<OPERANDS>([&](auto o) { read(ws, xs, 0, o); });
  for (; unit < hi; unit += stride) {
    const Place p = place_of(unit);
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
      for (int j = 0; j < TB; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    for (int left = steps_of(p); left > 0; --left) {
      next(w, true);
      static_for<3>([&](auto kk) {
        constexpr int KK = decltype(kk)::value;
        products(KK, [&](auto u) {
          deal(u, Operands{}, Early{}, [&](auto o) { read(ws, xs, KK + 1, o); });
          if constexpr (KK == 0) deal(u, Loads{}, Slots{}, [&](auto i) { ask(w, i); });
        });
      });
      loads_left<NI>();      // the next step has arrived (this wave's part; W of the one after need not)
      lds_barrier();         // and everyone's; this step's operands are all in registers
      ws += 2 * G::SLOT;
      if (ws >= G::SLOTS * G::SLOT) ws -= G::SLOTS * G::SLOT;
      xs += 2 * G::SLOT;
      if (xs >= G::SLOTS * G::SLOT) xs -= G::SLOTS * G::SLOT;
      next(x, false);
      products(3, [&](auto u) {
        deal(u, Operands{}, Early{}, [&](auto o) { read(ws, xs, 0, o); });
        deal(u, Loads{}, Slots{}, [&](auto i) { ask(x, i); });
      });
    }
    // The results pass the slot that W's next loads will take, a wave's own part of it.
    int free = w.slot + 2 * G::SLOT;
    if (free >= G::SLOTS * G::SLOT) free -= G::SLOTS * G::SLOT;
    char *mine = lds + free + wave * NI * 1024;
    if (a.splits > 1) finish_part(p, mine);
    else if (a.residual) for_activation(a.act, [&](auto kind) { finish(p, mine, kind, std::true_type{}); });
    else for_activation(a.act, [&](auto kind) { finish(p, mine, kind, std::false_type{}); });
    // Again (the registers were needed meanwhile).
    static_for<OPERANDS>([&](auto o) { read(ws, xs, 0, o); });
  }
  loads_left<0>();
}

// Adds the parts of 8 features of a row, in order.
template <typename T>
__global__ __launch_bounds__(256) void is_k13_dense_join(const Args a, int64_t items) {
  const int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  const int groups = a.part_row / 8, f = (int)(it % groups) * 8;
  const int64_t r = it / groups, entry = r / a.len, row = r - entry * a.len;
  const int64_t step = (int64_t)a.entries * a.len * a.part_row / 4;
  const floatx4 *p = reinterpret_cast<const floatx4 *>(a.part + r * a.part_row + f);
  floatx4 lo = p[0], hi = p[1];
#pragma unroll 4
  for (int s = 1; s < a.splits; ++s) {
    lo += p[s * step];
    hi += p[s * step + 1];
  }
  float z[8], bias[8];
  *reinterpret_cast<floatx4 *>(z) = lo;
  *reinterpret_cast<floatx4 *>(z + 4) = hi;
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = a.bias && f + e < a.features ? a.bias[f + e] : 0.f;
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
  // Workgroups start at different inputs: in step they would all read the same
  // columns of rows that lie far apart, and few memory channels at a time.
  const int turn = (int)((unsigned)ft * (NW * U) % (unsigned)chunks);
  // Two sets of U chunks: one on its way while the other is multiplied.
  T8 fw[2][U][FB], fx[2][U][TB];
  auto fetch = [&](int c0, auto set) {
    static_for<U>([&](auto u) {
      int c = c0 + u + turn;
      c = c >= chunks ? c - chunks : c;
      const bool in = c0 + u < chunks && c * 32 + quarter * 8 < a.in;
      static_for<FB>([&](auto i) { fw[set][u][i] = in ? *reinterpret_cast<const T8 *>(w + wo[i] + c * 32) : T8{}; });
      static_for<TB>([&](auto j) { fx[set][u][j] = in ? *reinterpret_cast<const T8 *>(x + xo[j] + c * 32) : T8{}; });
    });
  };
  auto multiply = [&](auto set) {
    static_for<U>([&](auto u) {
      static_for<FB>([&](auto i) {
        static_for<TB>([&](auto j) { acc[i][j] = mma16(fw[set][u][i], fx[set][u][j], acc[i][j]); });
      });
    });
  };
  using Set0 = std::integral_constant<int, 0>;
  using Set1 = std::integral_constant<int, 1>;
  int c0 = wave * U;
  if (c0 < chunks) fetch(c0, Set0{});
  while (c0 < chunks) {
    c0 += NW * U;
    if (c0 < chunks) fetch(c0, Set1{});
    multiply(Set0{});
    if (c0 >= chunks) break;
    c0 += NW * U;
    if (c0 < chunks) fetch(c0, Set0{});
    multiply(Set1{});
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
  int features, rows, waves, lds, groups;    // groups: workgroups a CU holds
};
template <int FB, int TB, int WF, int WT>
constexpr TileShape shape() {
  using G = Tile<FB, TB, WF, WT>;
  return {G::TF, G::TT, G::NW, G::BYTES, G::GROUPS};
}
constexpr TileShape kTiles[] = {shape<4, 2, 2, 4>(), shape<2, 2, 2, 2>(), shape<1, 1, 2, 2>()};

// Blocks of 16 features and of 16 rows of a few-rows workgroup, and chunks in flight.
struct FewShape {
  int features, rows;
};
constexpr FewShape kFew[] = {{1, 1}, {2, 1}, {2, 2}};
constexpr int kFewWaves = 8;
constexpr int kFewMost = 256;     // rows up to which they are looked at
constexpr double kMaxUnits = 2147483000.0;    // tiles of a call, counted in an int

// Workgroups for `units` tiles: as many as the device holds at a time, and a multiple
// of 8 (an XCD each). A workgroup without a tile leaves at once.
int64_t grid_of(int64_t units, int groups) {
  const int64_t held = (int64_t)persistent_grid(0x7fffffff, device_cu_count()) * groups;
  return units < held ? (units + 7) / 8 * 8 : held;
}

template <typename T>
hipError_t launch_t(const DensePlan &p, const Args &a, hipStream_t s) {
  const unsigned blocks = (unsigned)((int64_t)a.entries * p.row_tiles * p.feature_tiles * p.splits);
  if (p.few) {
    const dim3 grid((unsigned)blocks), block(p.block);
    switch (p.tile) {
      case 0: return launch_kernel(is_k13_dense_few<T, 1, 1, kFewWaves, 4>, grid, block, 0, s, a);
      case 1: return launch_kernel(is_k13_dense_few<T, 2, 1, kFewWaves, 2>, grid, block, 0, s, a);
      default: return launch_kernel(is_k13_dense_few<T, 2, 2, kFewWaves, 2>, grid, block, 0, s, a);
    }
  }
  hipError_t e;
  const dim3 grid((unsigned)grid_of(blocks, kTiles[p.tile].groups));
  switch (p.tile) {
    case 0: e = launch_kernel(is_k13_dense<T, 4, 2, 2, 4>, grid, dim3(p.block), 0, s, a); break;
    case 1: e = launch_kernel(is_k13_dense<T, 2, 2, 2, 2>, grid, dim3(p.block), 0, s, a); break;
    default: e = launch_kernel(is_k13_dense<T, 1, 1, 2, 2>, grid, dim3(p.block), 0, s, a); break;
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t items = (int64_t)a.entries * a.len * (a.part_row / 8);
  return launch_kernel(is_k13_dense_join<T>, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a, items);
}

}  // namespace

// How a call is cut, by an estimate of its time in microseconds fitted to runs of 16 to
// 65536 rows, 344 to 8192 inputs and 300 to 8192 features. Of 60 calls drawn from that range
// 41 come within 15% of it and all within 31%; short calls and those of one round of large
// tiles end sooner (33 said, 23 measured for 7200 rows, 512 to 2048), 128-squared tiles with
// more than 4000 inputs later.
//   tiles of 256, 128 and 64 squared, a step of 64 inputs: 1.0, 0.47 and 0.36 with one
//     workgroup on its CU and few CUs busy, 1.55, 0.95 and 0.80 with all of them (the clock
//     falls; two and four workgroups a CU for the smaller tiles); 4, 1.5 and 1 to fill the
//     buffers; 4, 3 and 1.5 for a tile's results, 10, 6 and 2 where all CUs write at once;
//     the read and write of everything at 5 TB/s, of which and the above the shorter is
//     hidden by two fifths;
//   few rows: a workgroup takes in 40 GB/s, two on a CU 30 each;
//   3 for a launch, 4 and the parts at 4 TB/s for joining.
// Measured on both sides: 7200 rows, 512 to 2048: 256 squared 21.6 us, 128 squared 24.4, 64
// squared 31.5; 300 rows, 4096 to 1024: 64 squared in four parts 17.5 us, 128 squared in four
// 19.4, unsplit 32.1 and 37.8.
double least_us(const dense_desc &d) {
  return 2.0 * ((double)d.in * d.features + (double)d.n * d.len * (d.in + d.features)) / 5.0e6;
}

double tile_us(const dense_desc &d, int tile, int splits) {
  static const double alone[] = {1.0, 0.47, 0.36}, all[] = {1.55, 0.95, 0.80}, start[] = {4.0, 1.5, 1.0};
  static const double end_alone[] = {4.0, 3.0, 1.5}, end_all[] = {10.0, 6.0, 2.0};
  const TileShape &t = kTiles[tile];
  const double rows = (double)d.n * d.len;
  const double units = d.n * ceil((double)d.len / t.rows) * ceil((double)d.features / t.features) * splits;
  const double held = 256.0 * t.groups, full = floor(units / held), rest = units - full * held;
  const double steps = ceil(ceil(d.in / 64.0) / splits);
  double us = start[tile] + full * (steps * all[tile] + end_all[tile]);
  if (rest > 0) {
    const double share = t.groups == 1 ? rest / 256.0 : rest > 256 ? (rest - 256.0) / (held - 256.0) : 0.0;
    us += steps * (alone[tile] + (all[tile] - alone[tile]) * share) + end_alone[tile] +
          (end_all[tile] - end_alone[tile]) * share;
  }
  const double least = least_us(d);
  us = 3.0 + (us > least ? us + 0.6 * least : least + 0.6 * us);
  return splits == 1 ? us : us + 4.0 + 8.0 * splits * rows * d.features / 4.0e6;
}

double few_us(const dense_desc &d, int shape) {
  const FewShape &f = kFew[shape];
  const double groups = d.n * ceil(d.len / (16.0 * f.rows)) * ceil(d.features / (16.0 * f.features));
  const double bytes = 32.0 * (f.features + f.rows) * d.in;
  const double us = groups <= 256 ? bytes / 40.0e3 : bytes / 30.0e3 * groups / 256.0, least = least_us(d);
  return 4.0 + (us > least ? us : least);
}

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
  const int64_t steps = ((int64_t)d.in + 63) / 64;
  p.splits = 1;
  p.split_in = (int)steps * 64;
  double best = 0.0;
  auto take = [&](double us) {
    const bool better = best == 0.0 || us < best;
    if (better) best = us;
    return better;
  };
  // Tiles of a call: a form that cannot be launched with so many is passed over.
  auto tiles = [&](int rows, int features) {
    return (double)d.n * ceil((double)d.len / rows) * ceil((double)d.features / features);
  };
  for (int i = 0; i < 3; ++i)
    for (int64_t n = 1; n <= 16 && n <= steps; n *= 2) {
      const int64_t per = (steps + n - 1) / n, parts = (steps + per - 1) / per;
      if (parts != n && n > 1) continue;
      if (tiles(kTiles[i].rows, kTiles[i].features) * parts > kMaxUnits) continue;
      const double join = (double)d.n * d.len * ((d.features + 7) / 8);      // its threads
      if (n > 1 && join > kMaxLaunchThreads - 256) continue;
      if (!take(tile_us(d, i, (int)parts))) continue;
      p.few = false;
      p.tile = i;
      p.splits = (int)parts;
      p.split_in = (int)per * 64;
    }
  for (int i = 0; i < 3 && d.len <= kFewMost; ++i) {
    if (tiles(16 * kFew[i].rows, 16 * kFew[i].features) * 64 * kFewWaves > kMaxLaunchThreads) continue;
    if (!take(few_us(d, i))) continue;
    p.few = true;
    p.tile = i;
    p.splits = 1;
    p.split_in = (int)steps * 64;
  }
  if (best == 0.0) return false;      // no form can be launched
  if (p.few) {
    p.tile_rows = 16 * kFew[p.tile].rows;
    p.tile_features = 16 * kFew[p.tile].features;
    p.block = 64 * kFewWaves;
    p.lds = kFewWaves * kFew[p.tile].rows * kFew[p.tile].features * 1024;
    p.name = "is_k13_dense_few";
  } else {
    p.tile_rows = kTiles[p.tile].rows;
    p.tile_features = kTiles[p.tile].features;
    p.block = 64 * kTiles[p.tile].waves;
    p.lds = kTiles[p.tile].lds;
    p.name = "is_k13_dense";
  }
  p.row_tiles = (d.len + p.tile_rows - 1) / p.tile_rows;
  p.feature_tiles = (d.features + p.tile_features - 1) / p.tile_features;
  return true;
}

size_t dense_workspace(const DensePlan &p) {
  return p.splits == 1 ? 0 : (size_t)p.splits * p.d.n * p.d.len * ((p.d.features + 7) / 8 * 8) * 4;
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
  a.part_row = (d.features + 7) / 8 * 8;
  a.row_tiles = (int)p.row_tiles;
  a.feature_tiles = (int)p.feature_tiles;
  a.units = (int)(d.n * p.row_tiles * p.feature_tiles * p.splits);
  a.by_tiles = divisor((unsigned)(p.row_tiles * p.feature_tiles));
  a.by_splits = divisor((unsigned)p.splits);
  a.by_span = divisor((unsigned)(8 * p.feature_tiles));
  a.by_last = divisor((unsigned)(p.row_tiles % 8 ? p.row_tiles % 8 : 8));
  return d.dtype == IS_F16 ? launch_t<_Float16>(p, a, s) : launch_t<__bf16>(p, a, s);
}

}  // namespace is

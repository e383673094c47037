// k10_rotary.hip -- rotary positions, alone or after the norm of each head.
//
//   y = R(pos) (norm(x) * w):  pair p of a head turns by the angle
//   2 pi * pos[p / Pa] * turns[p % Pa]; norm is none, x / sqrt(mean x^2 + eps)
//   or (x - mean) / sqrt(var + eps) over the head's d elements.
//
// Every element is read once and written once, so the kernel is bound by
// memory. A head belongs to 2^log_lanes neighbouring lanes; a lane holds both
// elements of its pairs, so that a pair turns in one lane and only the norm's
// sum crosses lanes:
//   half layout:        the lanes of the turning part have the V elements at
//                       V t of either half, the pairs V t .. V t + V - 1; the
//                       lanes after them take two neighbouring chunks each of
//                       what passes through;
//   interleaved layout: lane t has the chunks t and t + 2^log_lanes, V / 2 whole
//                       pairs in each (single elements: 2t and 2t + 1).
// V elements are 16 bytes, wherever they start: a half or a rest that V does not
// divide ends in a chunk that reaches back over its neighbour's elements (all
// loads of a wave's heads come before their stores, and both lanes store the
// same values). Parts shorter than a chunk run with fewer elements per access.
//
// All that a thread needs first (its elements of up to kHeadsAhead heads, the
// position, the frequencies, the norm's weights) is asked for at once, in vector
// loads and without branches, so one trip to memory starts a thread's work. A
// thread's sines serve all the heads it walks over.
//
// The angle is formed in turns in 64 bits, the whole turns are dropped inside the
// product (fma), and only the rest is rounded to 32 bits: off by 2^-26 turns and by
// 2^-53 of the whole angle, what a 64-bit frequency is short of (as much again from
// 2^27 turns on; 2^-24.7 turns at positions of 2^31).
// 16-bit results use the hardware sine of an angle in turns, fp32 results the
// library's sincospi of twice the angle.
#include "attention.hpp"
#include "common.hpp"

namespace is {
namespace {

constexpr int kThreads = kRotaryBlock;
constexpr int kHeadsAhead = 4;   // heads a thread loads before it computes

struct Part {
  const void *x;
  void *y;
  const float *weight;
  const int32_t *positions;
  int64_t pos_b, xb, xt, xh, yb, yt, yh;   // elements
  int len, heads;
  int log_slots;            // threads of a token: 2^log_slots groups of lanes
  unsigned blocks;          // blocks of one batch entry
  unsigned first;           // first block of the part
};

struct Args {
  Part part[2];
  int nparts;
  int d, rot, axes, per_axis;
  int log_lanes;            // lanes of a head
  int norm;
  float eps, magnitude;
  double turns[IS_MAX_HEAD_DIM / 2];   // of every pair
};

// Sum over the 2^log_lanes lanes of a head: after each step the lanes joined so
// far hold one value, so that mirrors serve as exchanges of 4 and 8.
__device__ __forceinline__ float head_sum(float v, int log_lanes) {
  auto add = [&](auto ctrl) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  if (log_lanes > 0) add(std::integral_constant<int, 0xB1>{});    // quad_perm [1, 0, 3, 2]
  if (log_lanes > 1) add(std::integral_constant<int, 0x4E>{});    // quad_perm [2, 3, 0, 1]
  if (log_lanes > 2) add(std::integral_constant<int, 0x141>{});   // row_half_mirror
  if (log_lanes > 3) add(std::integral_constant<int, 0x140>{});   // row_mirror
  if (log_lanes > 4) v += __shfl_xor(v, 16);
  if (log_lanes > 5) v += __shfl_xor(v, 32);
  return v;
}

template <typename T>
__device__ __forceinline__ void sine(double pos, double turns, float &s, float &c) {
  const float t = (float)fma(pos, turns, -rint(pos * turns));   // the rest of a turn, in [-1/2, 1/2]
  if constexpr (sizeof(T) == 4) {
    sincospif(2.f * t, &s, &c);
  } else {
    s = __builtin_amdgcn_sinf(t);
    c = __builtin_amdgcn_cosf(t);
  }
}

// NP: pair groups a lane holds (2 only for V = 1, where 64 lanes may be too few).
template <typename T, bool HALF, int V, int NP, bool NORM>
__global__ __launch_bounds__(kThreads) void is_k10_rotary(const Args a) {
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef T uvec __attribute__((ext_vector_type(V), aligned(sizeof(T))));   // at any element
  typedef float fvec __attribute__((ext_vector_type(V), aligned(4)));
  const int which = a.nparts == 2 && blockIdx.x >= a.part[1].first;
  const Part &p = a.part[which];
  const unsigned bid = blockIdx.x - p.first;
  const unsigned b = bid / p.blocks;
  const int lane = threadIdx.x & ((1 << a.log_lanes) - 1);
  const int64_t g = (int64_t)(bid - b * p.blocks) * (kThreads >> a.log_lanes) + (threadIdx.x >> a.log_lanes);
  const int slot = (int)(g & ((1 << p.log_slots) - 1));
  // Threads past the last token stay for the lane sums and touch no memory.
  const bool live = (g >> p.log_slots) < p.len;
  const int64_t token = live ? g >> p.log_slots : 0;
  const int pairs = a.rot / 2, rest = a.d - a.rot, turning = (pairs + V - 1) / V;

  int at0[NP], at1[NP];     // first element of the lane's two chunks
  int own0[NP], own1[NP];   // the first of each that is not also another lane's
  int first[NP], mid[NP];   // pairs of the first chunk; interleaved: of the second
  bool v0[NP], v1[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = lane + (i << a.log_lanes);
    if constexpr (HALF) {
      const bool turns = t < turning;
      const int u0 = 2 * (t - turning) * V, u1 = u0 + V;    // in what passes through
      first[i] = mid[i] = turns ? min(V * t, pairs - V) : pairs;
      at0[i] = turns ? first[i] : a.rot + min(u0, rest - V);
      at1[i] = turns ? first[i] + pairs : a.rot + min(u1, rest - V);
      own0[i] = turns ? V * t - first[i] : u0 - (at0[i] - a.rot);
      own1[i] = turns ? own0[i] : u1 - (at1[i] - a.rot);
      v0[i] = live && (turns || u0 < rest);
      v1[i] = live && (turns || u1 < rest);
    } else {
      at0[i] = V > 1 ? V * t : 2 * t;
      at1[i] = V > 1 ? at0[i] + (V << a.log_lanes) : at0[i] + 1;
      first[i] = at0[i] / 2;
      mid[i] = at1[i] / 2;
      own0[i] = own1[i] = 0;
      v0[i] = live && at0[i] < a.d;
      v1[i] = live && at1[i] < a.d;
    }
  }

  const T *x = static_cast<const T *>(p.x) + b * p.xb + token * p.xt;
  T *y = static_cast<T *>(p.y) + b * p.yb + token * p.yt;
  const int slots = 1 << p.log_slots;
  vec r0[kHeadsAhead][NP], r1[kHeadsAhead][NP];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeadsAhead; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int h = h0 + k * slots;
        r0[k][i] = r1[k][i] = vec{};
        if (h < p.heads && v0[i]) r0[k][i] = *reinterpret_cast<const uvec *>(x + h * p.xh + at0[i]);
        if (h < p.heads && v1[i]) r1[k][i] = *reinterpret_cast<const uvec *>(x + h * p.xh + at1[i]);
      }
  };
  load(slot);

  float sn[NP][V], cs[NP][V];
  fvec w0[NP], w1[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    w0[i] = w1[i] = fvec(1.f);
    if (NORM && p.weight) {
      if (v0[i]) w0[i] = *reinterpret_cast<const fvec *>(p.weight + at0[i]);
      if (v1[i]) w1[i] = *reinterpret_cast<const fvec *>(p.weight + at1[i]);
    }
  }
  if (a.rot > 0) {
    const int32_t *pos = p.positions + b * p.pos_b + token * a.axes;
    const int32_t q0 = pos[0], q1 = a.axes > 1 ? pos[1] : 0, q2 = a.axes > 2 ? pos[2] : 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      // Half layout: V pairs from first; interleaved: V / 2 from first and from mid.
      constexpr int N = HALF || V == 1 ? V : V / 2;
      typedef double dvec __attribute__((ext_vector_type(N), aligned(8)));
      const dvec f0 = *reinterpret_cast<const dvec *>(a.turns + min(first[i], IS_MAX_HEAD_DIM / 2 - N));
      const dvec f1 = *reinterpret_cast<const dvec *>(a.turns + min(mid[i], IS_MAX_HEAD_DIM / 2 - N));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int pair = j < N ? first[i] + j : mid[i] + j - N;
        const double f = j < N ? f0[j % N] : f1[j % N];
        const int32_t q = pair < a.per_axis ? q0 : pair < 2 * a.per_axis ? q1 : q2;
        sine<T>((double)q, f, sn[i][j], cs[i][j]);
        sn[i][j] *= a.magnitude;
        cs[i][j] *= a.magnitude;
      }
    }
  }

  const float inv_d = 1.f / (float)a.d;
  for (int h0 = slot; h0 < p.heads;) {
#pragma unroll
    for (int k = 0; k < kHeadsAhead; ++k) {
      const int h = h0 + k * slots;
      float e0[NP][V], e1[NP][V];
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          e0[i][j] = (float)r0[k][i][j];
          e1[i][j] = (float)r1[k][i][j];
        }
      if constexpr (NORM) {
        // Each element once: not in a chunk that does not exist, nor in the part
        // of one that belongs to its neighbour.
        auto sum_own = [&](auto f) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              sum += v0[i] && j >= own0[i] ? f(e0[i][j]) : 0.f;
              sum += v1[i] && j >= own1[i] ? f(e1[i][j]) : 0.f;
            }
          return head_sum(sum, a.log_lanes) * inv_d;
        };
        if (a.norm == IS_NORM_LAYER) {
          const float mean = sum_own([](float v) { return v; });
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              e0[i][j] -= mean;
              e1[i][j] -= mean;
            }
        }
        const float inv = rsqrtf(sum_own([](float v) { return v * v; }) + a.eps);   // also below the normal numbers
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            e0[i][j] *= inv * w0[i][j];
            e1[i][j] *= inv * w1[i][j];
          }
      }
      if (h >= p.heads) continue;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        vec o0, o1;
        if constexpr (HALF) {
          const bool turns = first[i] < pairs;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o0[j] = (T)(turns ? e0[i][j] * cs[i][j] - e1[i][j] * sn[i][j] : e0[i][j]);
            o1[j] = (T)(turns ? e0[i][j] * sn[i][j] + e1[i][j] * cs[i][j] : e1[i][j]);
          }
        } else {
          float e[2 * V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            e[j] = e0[i][j];
            e[V + j] = e1[i][j];
          }
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const bool turns = (V == 1 || j < V / 2 ? first[i] + j : mid[i] + j - V / 2) < pairs;
            const float u = e[2 * j], v = e[2 * j + 1];
            e[2 * j] = turns ? u * cs[i][j] - v * sn[i][j] : u;
            e[2 * j + 1] = turns ? u * sn[i][j] + v * cs[i][j] : v;
          }
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o0[j] = (T)e[j];
            o1[j] = (T)e[V + j];
          }
        }
        if (v0[i]) *reinterpret_cast<uvec *>(y + h * p.yh + at0[i]) = o0;
        if (v1[i]) *reinterpret_cast<uvec *>(y + h * p.yh + at1[i]) = o1;
      }
    }
    h0 += kHeadsAhead * slots;
    if (h0 < p.heads) load(h0);
  }
}

int ceil_log2(int64_t v) {
  int l = 0;
  while (((int64_t)1 << l) < v) ++l;
  return l;
}

// Lanes of a head (log2): those of the pairs, plus one for every two chunks
// that pass through; V = 1 folds more than 64 onto 64 lanes.
int log_lanes(const RotaryPlan &p, int vec) {
  const int turning = (p.d.rot / 2 + vec - 1) / vec, rest = (p.d.d - p.d.rot + vec - 1) / vec;
  const int need = p.d.layout == IS_ROTARY_HALF ? turning + (rest + 1) / 2 : (p.d.d / vec + 1) / 2;
  const int l = ceil_log2(need);
  return l > 6 ? 6 : l;
}

// Groups of lanes a token's heads are dealt to (log2). A group walks up to
// kHeadsAhead heads, whose loads are in flight together and whose sines are
// computed once, as long as that leaves every CU 128 threads; few tokens get a
// group per head. (Two frames of 3600 tokens, 8 + 8 heads of 64, with norm: 13.2 us
// with a group per head, 11.1 for two heads, 9.6 for four.)
int log_slots(const RotaryPlan &p, int vec, const is_tokens &t) {
  int l = ceil_log2(t.heads);
  const double lanes = (double)t.n * t.len * (double)((int64_t)1 << log_lanes(p, vec));
  for (int h = 1; h < kHeadsAhead && l > 0 && lanes * (double)((int64_t)1 << (l - 1)) >= 256.0 * 128; h *= 2) --l;
  return l;
}

int64_t blocks_per_entry(const RotaryPlan &p, int vec, const is_tokens &t) {
  const int64_t groups = (int64_t)t.len << log_slots(p, vec, t);
  const int per = kThreads >> log_lanes(p, vec);
  return (groups + per - 1) / per;
}

bool none(const is_tokens &t) { return t.n == 0 || t.len == 0 || t.heads == 0; }

template <typename T, int V, int NP>
hipError_t launch_t(bool half, const Args &a, unsigned blocks, hipStream_t s) {
  const dim3 g(blocks), t(kThreads);
  if (half)
    return a.norm ? launch_kernel(is_k10_rotary<T, true, V, NP, true>, g, t, 0, s, a)
                  : launch_kernel(is_k10_rotary<T, true, V, NP, false>, g, t, 0, s, a);
  return a.norm ? launch_kernel(is_k10_rotary<T, false, V, NP, true>, g, t, 0, s, a)
                : launch_kernel(is_k10_rotary<T, false, V, NP, false>, g, t, 0, s, a);
}

}  // namespace

// 16 bytes where the head's parts are at least that long (half layout) or made
// of such chunks (interleaved), else 8, else single elements. Where a head starts
// does not matter (a base is 16-byte aligned, the strides are free): the memory path
// takes a vector at any element.
int rotary_vector_width(const RotaryPlan &p, is_dtype dtype) {
  const int pairs = p.d.rot / 2, rest = p.d.d - p.d.rot;
  for (int v = dtype == IS_F32 ? 4 : 8; v >= 4; v /= 2) {
    const bool ok = p.d.layout == IS_ROTARY_HALF ? (pairs == 0 || pairs >= v) && (rest == 0 || rest >= v)
                                                 : p.d.d % v == 0;
    if (ok) return v;
  }
  return 1;
}

int64_t rotary_blocks(const RotaryPlan &p, int vec, const is_tokens &t) {
  return none(t) ? 0 : t.n * blocks_per_entry(p, vec, t);
}

hipError_t launch_rotary(const RotaryPlan &p, is_dtype dtype, int norm, float eps, const RotaryPart *parts,
                         int nparts, hipStream_t s) {
  const int vec = rotary_vector_width(p, dtype);
  Args a;
  a.nparts = 0;
  a.d = p.d.d;
  a.rot = p.d.rot;
  a.axes = p.d.axes;
  a.per_axis = p.per_axis;
  a.log_lanes = log_lanes(p, vec);
  a.norm = norm;
  a.eps = eps;
  a.magnitude = (float)p.d.magnitude;
  for (int i = 0; i < IS_MAX_HEAD_DIM / 2; ++i) a.turns[i] = p.turns[i];
  unsigned blocks = 0;
  for (int i = 0; i < nparts; ++i) {
    const RotaryPart &r = parts[i];
    if (none(r.xt)) continue;
    Part &q = a.part[a.nparts++];
    q = {r.x, r.y, r.weight, r.positions, r.pos_batch_stride, r.xt.batch_stride, r.xt.token_stride,
         r.xt.head_stride, r.yt.batch_stride, r.yt.token_stride, r.yt.head_stride, r.xt.len, r.xt.heads,
         log_slots(p, vec, r.xt), (unsigned)blocks_per_entry(p, vec, r.xt), blocks};
    blocks += (unsigned)(r.xt.n * (int64_t)q.blocks);
  }
  if (a.nparts == 1) a.part[1] = a.part[0];
  const bool half = p.d.layout == IS_ROTARY_HALF;
  if (dtype == IS_F32)
    return vec == 4 ? launch_t<float, 4, 1>(half, a, blocks, s) : launch_t<float, 1, 2>(half, a, blocks, s);
  if (dtype == IS_F16)
    return vec == 8   ? launch_t<_Float16, 8, 1>(half, a, blocks, s)
           : vec == 4 ? launch_t<_Float16, 4, 1>(half, a, blocks, s)
                      : launch_t<_Float16, 1, 2>(half, a, blocks, s);
  return vec == 8   ? launch_t<__bf16, 8, 1>(half, a, blocks, s)
         : vec == 4 ? launch_t<__bf16, 4, 1>(half, a, blocks, s)
                    : launch_t<__bf16, 1, 2>(half, a, blocks, s);
}

}  // namespace is

// k10_rotary.hip -- rotary positions, alone or after the norm of each head.
//
//   y = R(pos) (norm(x) * w):  pair p of a head turns by the angle
//   2 pi * pos[p / Pa] * turns[p % Pa]; norm is none, x / sqrt(mean x^2 + eps)
//   or (x - mean) / sqrt(var + eps) over the head's d elements.
//
// Every element is read once and written once, so the kernel is bound by
// memory. A head belongs to `lanes` neighbouring lanes (a power of two); a
// lane holds both elements of its pairs, so that a pair turns in one lane and
// only the norm's sum crosses lanes:
//   half layout:        lane t has the V-element chunks t and t + rot / 2 / V,
//                       the pairs V t .. V t + V - 1; lanes past the rotated
//                       part take two neighbouring chunks each and pass them on;
//   interleaved layout: lane t has the chunks 2t and 2t + 1, the same pairs.
// V = 8 (16-bit) or 4 (fp32) elements are 16 bytes. Shapes, strides or a
// rotated part that those chunks do not divide run with V = 4 (16-bit) or 1.
// A thread's sines serve all the heads it walks over (`slots` apart).
//
// The angle is formed in turns in 64 bits, the whole turns are dropped there,
// and only the rest is rounded to 32 bits: error 2^-26 turns at any position.
// 16-bit results use the hardware sine of an angle in turns, fp32 results the
// library's sincospi of twice the angle.
#include "attention.hpp"
#include "common.hpp"

namespace is {
namespace {

constexpr int kThreads = 256;
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
  double turns[IS_MAX_HEAD_DIM / 2];
};

// Sum over the 2^log_lanes lanes of a head.
__device__ __forceinline__ float head_sum(float v, int log_lanes) {
  for (int i = 0; i < log_lanes; ++i) v += __shfl_xor(v, 1 << i);
  return v;
}

template <typename T>
__device__ __forceinline__ void sine(double turns, float &s, float &c) {
  const float t = (float)(turns - rint(turns));   // the rest of a turn, in [-1/2, 1/2]
  if constexpr (sizeof(T) == 4) {
    sincospif(2.f * t, &s, &c);
  } else {
    s = __builtin_amdgcn_sinf(t);
    c = __builtin_amdgcn_cosf(t);
  }
}

// NP: pair groups a lane holds (2 only for V = 1, where 64 lanes may be too few).
template <typename T, bool HALF, int V, int NP>
__global__ __launch_bounds__(kThreads) void is_k10_rotary(const Args a) {
  typedef T vec __attribute__((ext_vector_type(V)));
  const int which = a.nparts == 2 && blockIdx.x >= a.part[1].first;
  const Part &p = a.part[which];
  const unsigned bid = blockIdx.x - p.first;
  const unsigned b = bid / p.blocks;
  const int lane = threadIdx.x & ((1 << a.log_lanes) - 1);
  const int64_t g = (int64_t)(bid - b * p.blocks) * (kThreads >> a.log_lanes) + (threadIdx.x >> a.log_lanes);
  const int slot = (int)(g & ((1 << p.log_slots) - 1));
  const int64_t token = g >> p.log_slots;
  // Threads past the last token stay for the lane sums and touch no memory.
  const bool live = token < p.len;
  const int chunks = a.d / V, turning = a.rot / 2 / V;

  int c0[NP], c1[NP];
  bool v0[NP], v1[NP];
  float sn[NP][V], cs[NP][V], w0[NP][V], w1[NP][V];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = lane + (i << a.log_lanes);
    const bool turns = HALF && t < turning;
    c0[i] = turns ? t : HALF ? 2 * turning + 2 * (t - turning) : 2 * t;
    c1[i] = turns ? t + turning : c0[i] + 1;
    v0[i] = live && c0[i] < chunks;
    v1[i] = live && c1[i] < chunks;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int pair = V * t + j;
      sn[i][j] = 0.f;
      cs[i][j] = 1.f;
      if (live && 2 * pair < a.rot) {
        const int axis = (pair >= a.per_axis) + (pair >= 2 * a.per_axis);
        const int32_t pos = p.positions[b * p.pos_b + token * a.axes + axis];
        sine<T>((double)pos * a.turns[pair - axis * a.per_axis], sn[i][j], cs[i][j]);
        sn[i][j] *= a.magnitude;
        cs[i][j] *= a.magnitude;
      }
      w0[i][j] = w1[i][j] = 1.f;
      if (a.norm && p.weight) {
        if (v0[i]) w0[i][j] = p.weight[c0[i] * V + j];
        if (v1[i]) w1[i][j] = p.weight[c1[i] * V + j];
      }
    }
  }

  const T *x = static_cast<const T *>(p.x) + b * p.xb + token * p.xt;
  T *y = static_cast<T *>(p.y) + b * p.yb + token * p.yt;
  const float inv_d = 1.f / (float)a.d;
  const int slots = 1 << p.log_slots;
  for (int h0 = slot; h0 < p.heads; h0 += kHeadsAhead * slots) {
    vec r0[kHeadsAhead][NP], r1[kHeadsAhead][NP];
#pragma unroll
    for (int k = 0; k < kHeadsAhead; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int h = h0 + k * slots;
        r0[k][i] = r1[k][i] = vec{};
        if (h < p.heads && v0[i]) r0[k][i] = *reinterpret_cast<const vec *>(x + h * p.xh + c0[i] * V);
        if (h < p.heads && v1[i]) r1[k][i] = *reinterpret_cast<const vec *>(x + h * p.xh + c1[i] * V);
      }
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
      if (a.norm) {
        if (a.norm == IS_NORM_LAYER) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) sum += e0[i][j] + e1[i][j];
          const float mean = head_sum(sum, a.log_lanes) * inv_d;
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              e0[i][j] = v0[i] ? e0[i][j] - mean : 0.f;   // chunks that do not exist stay 0
              e1[i][j] = v1[i] ? e1[i][j] - mean : 0.f;
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) sq += e0[i][j] * e0[i][j] + e1[i][j] * e1[i][j];
        const float inv = 1.f / sqrtf(head_sum(sq, a.log_lanes) * inv_d + a.eps);
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
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o0[j] = (T)(e0[i][j] * cs[i][j] - e1[i][j] * sn[i][j]);
            o1[j] = (T)(e0[i][j] * sn[i][j] + e1[i][j] * cs[i][j]);
          }
        } else {
          float e[2 * V], f[2 * V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            e[j] = e0[i][j];
            e[V + j] = e1[i][j];
          }
#pragma unroll
          for (int j = 0; j < V; ++j) {
            f[2 * j] = e[2 * j] * cs[i][j] - e[2 * j + 1] * sn[i][j];
            f[2 * j + 1] = e[2 * j] * sn[i][j] + e[2 * j + 1] * cs[i][j];
          }
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o0[j] = (T)f[j];
            o1[j] = (T)f[V + j];
          }
        }
        if (v0[i]) *reinterpret_cast<vec *>(y + h * p.yh + c0[i] * V) = o0;
        if (v1[i]) *reinterpret_cast<vec *>(y + h * p.yh + c1[i] * V) = o1;
      }
    }
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
  const int chunks = p.d.d / vec;
  const int turning = p.d.layout == IS_ROTARY_HALF ? p.d.rot / 2 / vec : 0;
  const int need = turning + (chunks - 2 * turning + 1) / 2;
  const int l = ceil_log2(need);
  return l > 6 ? 6 : l;
}

// Groups of lanes a token's heads are dealt to (log2). Few tokens: a group per
// head. Once every CU has 1024 threads that way, groups of up to
// kHeadsAhead heads, whose sines are then computed once.
int log_slots(const RotaryPlan &p, int vec, const is_tokens &t) {
  const int l = ceil_log2(t.heads);
  const double threads = (double)t.n * t.len * (double)((int64_t)1 << (l + log_lanes(p, vec)));
  const int few = ceil_log2(kHeadsAhead);
  return threads < 256.0 * 1024 * kHeadsAhead ? l : (l > few ? l - few : 0);
}

int64_t blocks_per_entry(const RotaryPlan &p, int vec, const is_tokens &t) {
  const int64_t groups = (int64_t)t.len << log_slots(p, vec, t);
  const int per = kThreads >> log_lanes(p, vec);
  return (groups + per - 1) / per;
}

bool none(const is_tokens &t) { return t.n == 0 || t.len == 0 || t.heads == 0; }

template <typename T, int V, int NP>
hipError_t launch_t(bool half, const Args &a, unsigned blocks, hipStream_t s) {
  return half ? launch_kernel(is_k10_rotary<T, true, V, NP>, dim3(blocks), dim3(kThreads), 0, s, a)
              : launch_kernel(is_k10_rotary<T, false, V, NP>, dim3(blocks), dim3(kThreads), 0, s, a);
}

}  // namespace

int rotary_vector_width(const RotaryPlan &p, is_dtype dtype, const RotaryPart *parts, int nparts) {
  for (int v = dtype == IS_F32 ? 4 : 8; v > 1; v /= 2) {
    if (v == 2) break;   // 8-byte chunks at least, or single elements
    bool ok = p.d.d % v == 0 && (p.d.layout == IS_ROTARY_INTERLEAVED || p.d.rot / 2 % v == 0);
    for (int i = 0; i < nparts && ok; ++i)
      for (const is_tokens *t : {&parts[i].xt, &parts[i].yt}) {
        if (none(*t)) continue;
        ok = ok && (t->n == 1 || t->batch_stride % v == 0) && (t->len == 1 || t->token_stride % v == 0) &&
             (t->heads == 1 || t->head_stride % v == 0);
      }
    if (ok) return v;
  }
  return 1;
}

int64_t rotary_blocks(const RotaryPlan &p, is_dtype, int vec, const is_tokens &t) {
  return none(t) ? 0 : t.n * blocks_per_entry(p, vec, t);
}

hipError_t launch_rotary(const RotaryPlan &p, is_dtype dtype, int norm, float eps, const RotaryPart *parts,
                         int nparts, hipStream_t s) {
  const int vec = rotary_vector_width(p, dtype, parts, nparts);
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

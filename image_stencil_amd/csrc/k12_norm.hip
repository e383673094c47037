// k12_norm.hip -- the sum and norm between two blocks, one pass over rows of c
// channels:
//   x' = x + s g post(y),   z = norm(x') w (1 + scale) + shift + b
// with both norms over the row (mean square, or mean and variance).
//
// A row belongs to TPR threads, 8 or 16 elements each, and stays in
// registers from its load to its stores: statistics are sums over the threads
// (two for a norm with a mean, whose variance is that of the differences). What
// multiplies and adds per channel is folded once for all rows of an entry:
//   x' = x + G yhat,  G = s g post_weight;   z = A xhat + B,  A = w (1 + scale).
// Groups of threads walk the rows of one entry, the next row's loads on their way
// while this one is summed. Rows may start at any element (the memory path takes a vector
// at any address); a vector across a row's end is taken by elements. Stores do not stay in
// the caches (16384 rows of 1024 bf16 channels, norm alone: 30.7 us without that, 25.0;
// an operator that reads them next loses nothing).
//
// Bound: one read and one write of every element. 8 x 16384 rows of 1024 bf16 channels
// with both norms and all vectors: 212 us, 5.07 TB/s, the rate of a large copy (213); two
// frames of 3600 rows of 512 fp16 channels: 9.3 us; 3063 rows of 1001 fp32 channels: 13.7
// (floor 9.8 and a launch); one row: 4.0 in a graph.
#include <math.h>

#include "blocks.hpp"
#include "common.hpp"
#include "divide.hpp"

namespace is {
namespace {

struct Args {
  NormPointers p;
  int64_t xb, xr, yb, yr, xob, xor_, ob, orow, gate_b, scale_b, shift_b;
  int entries, len, c, groups;   // groups of threads that share an entry's rows
  int norm, post;
  float eps, alpha, inv_c;
  Divisor by_groups;
};

// Threads of a workgroup: one row where waves share it (they meet at barriers), else
// four waves.
__host__ __device__ constexpr int block_of(int tpr) { return tpr > kWave ? tpr : 256; }

// The sum over the TPR threads of a row. Rows of one wave or less: lanes; else
// the waves' sums meet in LDS, in two places in turn, so that one barrier is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *shared, int &turn) {
#pragma unroll
  for (int m = 1; m < (TPR < kWave ? TPR : kWave); m *= 2) v += __shfl_xor(v, m);
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    float *at = shared + turn * W;
    turn ^= 1;
    if ((threadIdx.x & (kWave - 1)) == 0) at[threadIdx.x / kWave] = v;
    lds_barrier();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += at[i];
  }
  return v;
}

// E: elements of a thread.
template <typename T, int TPR, int E>
__global__ __launch_bounds__(block_of(TPR)) void is_k12_block_norm(const Args a) {
  constexpr int V = 16 / sizeof(T), NV = E / V, BLOCK = block_of(TPR);
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef T uvec __attribute__((ext_vector_type(V), aligned(sizeof(T))));   // at any element
  __shared__ float shared[TPR > kWave ? 2 * TPR / kWave : 1];
  lds_poison(shared, sizeof(shared));
  int turn = 0;
  const int lane = threadIdx.x % TPR;
  const unsigned g = blockIdx.x * (BLOCK / TPR) + threadIdx.x / TPR;      // under 2^32 threads / 16
  const int b = divide((int)g, a.by_groups);
  unsigned i = g - (unsigned)(b * a.groups);      // past the last row it may pass 2^31
  if (b >= a.entries) return;     // whole groups of threads leave

  // Vector v of a thread: elements at .. at + V - 1, the last one cut at c.
  auto load = [&](const T *row, int v) -> vec {
    const int at = (lane + v * TPR) * V;
    vec r = {};
    if (at + V <= a.c) {
      r = *reinterpret_cast<const uvec *>(row + at);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at + j < a.c) r[j] = row[at + j];
    }
    return r;
  };
  auto store = [&](T *row, int v, const float (&f)[V]) {
    const int at = (lane + v * TPR) * V;
    vec r;
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = (T)f[j];
    if (at + V <= a.c) {
      __builtin_nontemporal_store(r, reinterpret_cast<uvec *>(row + at));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at + j < a.c) row[at + j] = r[j];
    }
  };
  const T *x = static_cast<const T *>(a.p.x) + b * a.xb;
  const T *y = static_cast<const T *>(a.p.y) + b * a.yb;
  T *x_out = static_cast<T *>(a.p.x_out) + b * a.xob;
  T *out = static_cast<T *>(a.p.out) + b * a.ob;
  const bool has_y = a.p.y != nullptr;
  vec rx[NV] = {}, ry[NV] = {};
  auto fetch = [&](unsigned row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      rx[v] = load(x + row * a.xr, v);
      if (has_y) ry[v] = load(y + row * a.yr, v);
    }
  };
  fetch(i);

  // Vector v of what is given per channel (S: its type), or `none` everywhere.
  float G[NV][V], A[NV][V], B[NV][V];
  auto vector = [&](auto type, const void *p, int64_t offset, int v, float none, float (&f)[V]) {
    using S = decltype(type);
    typedef S svec __attribute__((ext_vector_type(V), aligned(sizeof(S))));
    const int at = (lane + v * TPR) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = none;
    if (!p) return;
    const S *q = static_cast<const S *>(p) + offset;
    if (at + V <= a.c) {
      const svec r = *reinterpret_cast<const svec *>(q + at);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = (float)r[j];
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (at + j < a.c) f[j] = (float)q[at + j];
    }
  };
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float t[V];
    vector(T{}, a.p.gate, b * a.gate_b, v, 1.f, G[v]);
    vector(0.f, a.post ? a.p.post_weight : nullptr, 0, v, 1.f, t);
#pragma unroll
    for (int j = 0; j < V; ++j) G[v][j] *= a.alpha * t[j];
    vector(0.f, a.p.weight, 0, v, 1.f, A[v]);
    vector(T{}, a.p.scale, b * a.scale_b, v, 0.f, t);
#pragma unroll
    for (int j = 0; j < V; ++j) A[v][j] *= 1.f + t[j];
    vector(T{}, a.p.shift, b * a.shift_b, v, 0.f, B[v]);
    vector(0.f, a.p.bias, 0, v, 0.f, t);
#pragma unroll
    for (int j = 0; j < V; ++j) B[v][j] += t[j];
  }

  // f in place normed: minus its mean (IS_NORM_LAYER), by its mean square.
  auto normed = [&](float (&f)[NV][V], int kind) {
    if (kind == IS_NORM_LAYER) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < V; ++j) sum += f[v][j];
      const float mean = row_sum<TPR>(sum, shared, turn) * a.inv_c;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < V; ++j) f[v][j] = (lane + v * TPR) * V + j < a.c ? f[v][j] - mean : 0.f;
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < V; ++j) sum += f[v][j] * f[v][j];
    const float inv = rsqrtf(row_sum<TPR>(sum, shared, turn) * a.inv_c + a.eps);   // also below the normal numbers
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < V; ++j) f[v][j] *= inv;
  };

  while (true) {
    float f[NV][V], h[NV][V];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[v][j] = (float)rx[v][j];
        h[v][j] = (float)ry[v][j];
      }
    const unsigned row = i;
    i += a.groups;
    if (E <= 16 && i < (unsigned)a.len) fetch(i);     // (32 elements leave no registers for more)
    if (has_y) {
      if (a.post) normed(h, a.post);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[v][j] += G[v][j] * h[v][j];
        if (a.p.x_out) store(x_out + row * a.xor_, v, f[v]);
      }
    }
    if (a.norm) {
      normed(f, a.norm);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[v][j] = f[v][j] * A[v][j] + B[v][j];
        store(out + row * a.orow, v, f[v]);
      }
    }
    if (i >= (unsigned)a.len) break;
    if constexpr (E > 16) fetch(i);
  }
}

// Threads of a row and the elements of each, the fewest threads first. (With 32
// elements a thread, registers leave a wave per SIMD: 4096 rows of 8192 bf16 channels
// with all vectors 80 us, with 16 elements 57. The last shape takes 32 all the same: 1024
// threads leave 128 registers each, and are slower.)
struct Shape {
  int tpr, e;
};
constexpr Shape kShapes[] = {{16, 8}, {64, 8}, {64, 16}, {128, 16}, {256, 16}, {512, 16}, {512, 32}};

int shape_of(const block_norm_desc &d) {
  int i = 0;
  while (kShapes[i].tpr * kShapes[i].e < d.c) ++i;
  return i;
}

// Groups of threads that share an entry's rows: a row each up to 4096 waves; beyond, as
// many as run at a time, so that what is loaded per channel serves many rows (131072
// rows of 1024 bf16 channels with all vectors: 2048 waves 212 us, 4096 220; 262144 rows
// of 64: 56 with 4096, 88 with 2048).
int groups_of(const block_norm_desc &d) {
  const Shape s = kShapes[shape_of(d)];
  const double rows = (double)d.x.n * d.x.len, waves = s.tpr / (double)kWave;
  const double most = (s.e <= 8 || rows * waves <= 4096.0 ? 4096.0 : 2048.0) / waves;
  double each = rows <= most ? 1.0 : ceil(rows / most);
  if (each > d.x.len) each = d.x.len;
  const int groups = (int)ceil(d.x.len / each);
  return groups < 1 ? 1 : groups;
}

int64_t blocks_of(const block_norm_desc &d) {
  const int tpr = kShapes[shape_of(d)].tpr, per = block_of(tpr) / tpr;
  return ((int64_t)d.x.n * groups_of(d) + per - 1) / per;
}

template <typename T>
hipError_t launch_t(const block_norm_desc &d, const Args &a, hipStream_t s) {
  const dim3 grid((unsigned)blocks_of(d));
  auto go = [&](auto tpr, auto e) {
    constexpr int TPR = decltype(tpr)::value;
    return launch_kernel(is_k12_block_norm<T, TPR, decltype(e)::value>, grid, dim3(block_of(TPR)), 0, s, a);
  };
#define IS_SHAPE(I) \
  case I: return go(std::integral_constant<int, kShapes[I].tpr>{}, std::integral_constant<int, kShapes[I].e>{})
  switch (shape_of(d)) {
    IS_SHAPE(0);
    IS_SHAPE(1);
    IS_SHAPE(2);
    IS_SHAPE(3);
    IS_SHAPE(4);
    IS_SHAPE(5);
    IS_SHAPE(6);
    default: return hipErrorInvalidValue;
  }
#undef IS_SHAPE
}

}  // namespace

double block_norm_threads(const block_norm_desc &d) {
  return (double)blocks_of(d) * block_of(kShapes[shape_of(d)].tpr);
}

hipError_t launch_block_norm(const block_norm_desc &d, const NormPointers &p, hipStream_t s) {
  Args a;
  a.p = p;
  a.xb = d.x.batch_stride;
  a.xr = d.x.row_stride;
  a.yb = p.y ? d.y.batch_stride : 0;
  a.yr = p.y ? d.y.row_stride : 0;
  a.xob = p.x_out ? d.x_out.batch_stride : 0;
  a.xor_ = p.x_out ? d.x_out.row_stride : 0;
  a.ob = p.out ? d.out.batch_stride : 0;
  a.orow = p.out ? d.out.row_stride : 0;
  a.gate_b = d.gate_stride;
  a.scale_b = d.scale_stride;
  a.shift_b = d.shift_stride;
  a.entries = d.x.n;
  a.len = d.x.len;
  a.c = d.c;
  a.groups = groups_of(d);
  a.by_groups = divisor((unsigned)a.groups);
  a.norm = d.norm;
  a.post = d.post;
  a.eps = d.eps;
  a.alpha = d.residual_scale;
  a.inv_c = 1.f / (float)d.c;
  switch (d.dtype) {
    case IS_F32: return launch_t<float>(d, a, s);
    case IS_F16: return launch_t<_Float16>(d, a, s);
    default: return launch_t<__bf16>(d, a, s);
  }
}

}  // namespace is

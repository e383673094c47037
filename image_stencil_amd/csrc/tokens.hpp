// tokens.hpp -- argument checks that the entry points on token tensors share
// (host only): address ranges, strides, overlaps.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "imgstencil.h"

namespace is {
namespace arguments {

constexpr double kMaxBytes = 7.0e13;       // one tensor's address range, under 2^46

inline int element_bytes(is_dtype t) { return t == IS_F32 ? 4 : 2; }

inline bool misaligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

// Address range of a strided tensor, as offsets from its base.
struct Range {
  const char *lo, *hi;
};
inline bool intersect(const Range &a, const Range &b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline bool empty(const is_tokens &t) { return t.n == 0 || t.len == 0 || t.heads == 0; }

// Bytes from a token tensor's base to the end of its last element.
inline double extent_bytes(const is_tokens &t, int d, int es) {
  if (empty(t)) return 0.0;
  return ((double)(t.n - 1) * t.batch_stride + (double)(t.len - 1) * t.token_stride +
          (double)(t.heads - 1) * t.head_stride + d) * es;
}

inline Range range(const void *p, const is_tokens &t, int d, int es) {
  const char *c = static_cast<const char *>(p);
  return {c, c + (size_t)extent_bytes(t, d, es)};
}

// Sizes, strides and address range of an input.
inline is_status check_tokens(const is_tokens &t, int d, int es) {
  if (t.n < 0 || t.len < 0 || t.heads < 0) return IS_ERR_INVALID_ARG;
  if (t.batch_stride < 0 || t.token_stride < 0 || t.head_stride < 0) return IS_ERR_INVALID_ARG;
  if (extent_bytes(t, d, es) > kMaxBytes) return IS_ERR_UNSUPPORTED;
  return IS_OK;
}

struct Dim {
  int64_t stride;
  int size;
};
// The dimensions of more than one step, the smallest stride first; returns their number.
inline int by_stride(const is_tokens &t, Dim *dims) {
  const Dim all[3] = {{t.batch_stride, t.n}, {t.token_stride, t.len}, {t.head_stride, t.heads}};
  int n = 0;
  for (const Dim &m : all) {
    if (m.size <= 1) continue;
    int i = n++;
    for (; i > 0 && dims[i - 1].stride > m.stride; --i) dims[i] = dims[i - 1];
    dims[i] = m;
  }
  return n;
}

// An output's elements must have addresses of their own: sorted by stride,
// every dimension steps over all that the smaller ones span. (A sufficient
// condition, met by every tensor sliced or permuted from a dense one.)
inline bool distinct(const is_tokens &t, int d) {
  Dim dims[3];
  double span = d;
  for (int i = 0, n = by_stride(t, dims); i < n; ++i) {
    if ((double)dims[i].stride < span) return false;
    span += (double)(dims[i].size - 1) * dims[i].stride;
  }
  return true;
}

// Of two tensors of one size; the stride of a single step says nothing.
inline bool same_strides(const is_tokens &a, const is_tokens &b) {
  return (a.n <= 1 || a.batch_stride == b.batch_stride) && (a.len <= 1 || a.token_stride == b.token_stride) &&
         (a.heads <= 1 || a.head_stride == b.head_stride);
}

// Every address from the first element to the last belongs to the tensor.
inline bool gapless(const is_tokens &t, int d) {
  Dim dims[3];
  double span = d;
  for (int i = 0, n = by_stride(t, dims); i < n; ++i) {
    if ((double)dims[i].stride > span) return false;
    span += (double)(dims[i].size - 1) * dims[i].stride;
  }
  return true;
}

// Two tensors certainly share an address: one base, or the base of one among
// the other's elements where those leave no gap. Slices of a packed buffer, which
// lie between each other, do not.
inline bool collide(const void *p, const is_tokens &tp, const void *q, const is_tokens &tq, int d, int es) {
  const Range a = range(p, tp, d, es), b = range(q, tq, d, es);
  if (!intersect(a, b)) return false;
  return a.lo == b.lo || (a.lo < b.lo ? gapless(tp, d) : gapless(tq, d));
}

inline is_tokens tokens(int n, int len, int heads, const int64_t *stride) {
  return {n, len, heads, stride[0], stride[1], stride[2]};
}

}  // namespace arguments
}  // namespace is

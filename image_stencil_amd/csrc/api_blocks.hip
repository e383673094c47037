// api_blocks.hip -- the C ABI of the sum and norm between blocks and of dense
// layers: argument checks, plans and launches, on the host and before any GPU call.
#include <math.h>
#include <string.h>

#include <new>

#include "blocks.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "tokens.hpp"

struct dense_plan_s {
  is::DensePlan p;
};

using namespace is::arguments;

namespace {

// Rows as token tensors of one head.
is_tokens rows(const is_rows &r) { return {r.n, r.len, 1, r.batch_stride, r.row_stride, 0}; }
is_tokens rows(int n, int len, const int64_t *stride) { return {n, len, 1, stride[0], stride[1], 0}; }

bool norm_kind(int k) { return k == 0 || k == IS_NORM_RMS || k == IS_NORM_LAYER; }

// n vectors of c elements, `stride` apart.
Range vectors(const void *p, int n, int64_t stride, int c, int es) {
  const char *b = static_cast<const char *>(p);
  return {b, b ? b + ((size_t)(n - 1) * stride + c) * es : b};
}

is_status run_norm(const block_norm_desc &d, const is::NormPointers &p, hipStream_t stream) {
  if (d.c < 1 || !norm_kind(d.norm) || !norm_kind(d.post)) return IS_ERR_INVALID_ARG;
  if (!(d.eps >= 0.f) || !isfinite(d.eps) || !isfinite(d.residual_scale)) return IS_ERR_INVALID_ARG;
  if (d.gate_stride < 0 || d.scale_stride < 0 || d.shift_stride < 0) return IS_ERR_INVALID_ARG;
  if (d.dtype != IS_F32 && d.dtype != IS_F16 && d.dtype != IS_BF16) return IS_ERR_UNSUPPORTED;
  if (d.c > IS_MAX_NORM_CHANNELS) return IS_ERR_UNSUPPORTED;
  const int es = element_bytes(d.dtype), c = d.c;
  const is_tokens tx = rows(d.x), ty = rows(d.y), txo = rows(d.x_out), to = rows(d.out);
  is_status st = check_tokens(tx, c, es);
  if (st != IS_OK) return st;
  if (d.x.n == 0 || d.x.len == 0) return IS_OK;
  // What is computed: a sum needs y, an output norm. Something must be written.
  if (!p.x || (p.x_out && !p.y) || (d.norm != 0) != (p.out != nullptr) || (!p.x_out && !p.out) || (d.post && !p.y) ||
      (p.gate && !p.y))
    return IS_ERR_INVALID_ARG;
  const struct {
    const void *p;
    const is_tokens &t;
    bool written;
  } others[3] = {{p.y, ty, false}, {p.x_out, txo, true}, {p.out, to, true}};
  for (const auto &o : others) {
    if (!o.p) continue;
    st = check_tokens(o.t, c, es);
    if (st != IS_OK) return st;
    if (o.t.n != tx.n || o.t.len != tx.len) return IS_ERR_INVALID_ARG;
    if (o.written && !distinct(o.t, c)) return IS_ERR_INVALID_ARG;
  }
  for (const void *q : {p.x, p.y, (const void *)p.x_out, (const void *)p.out})
    if (misaligned(q, 16)) return IS_ERR_MISALIGNED;
  for (const void *q : {p.gate, p.scale, p.shift})
    if (misaligned(q, es)) return IS_ERR_MISALIGNED;
  for (const float *q : {p.post_weight, p.weight, p.bias})
    if (misaligned(q, 4)) return IS_ERR_MISALIGNED;
  for (const int64_t s : {d.gate_stride, d.scale_stride, d.shift_stride})
    if ((double)(d.x.n - 1) * s * es > kMaxBytes) return IS_ERR_UNSUPPORTED;
  const Range read[6] = {vectors(p.gate, tx.n, d.gate_stride, c, es),   vectors(p.scale, tx.n, d.scale_stride, c, es),
                         vectors(p.shift, tx.n, d.shift_stride, c, es), vectors(p.post_weight, 1, 0, c, 4),
                         vectors(p.weight, 1, 0, c, 4),                 vectors(p.bias, 1, 0, c, 4)};
  Range written[2] = {{nullptr, nullptr}, {nullptr, nullptr}};
  for (int i = 0; i < 2; ++i) {
    const void *o = i ? p.out : p.x_out;
    const is_tokens &t = i ? to : txo;
    if (!o) continue;
    written[i] = range(o, t, c, es);
    for (const Range &r : read)
      if (intersect(written[i], r)) return IS_ERR_INVALID_ARG;
    if (!(o == p.x && same_strides(t, tx)) && intersect(written[i], range(p.x, tx, c, es))) return IS_ERR_INVALID_ARG;
    if (p.y && !(o == p.y && same_strides(t, ty)) && intersect(written[i], range(p.y, ty, c, es)))
      return IS_ERR_INVALID_ARG;
  }
  if (intersect(written[0], written[1])) return IS_ERR_INVALID_ARG;
  if (is::block_norm_threads(d) > is::kMaxLaunchThreads) return IS_ERR_UNSUPPORTED;
  return is::report_hip(is::launch_block_norm(d, p, stream));
}

constexpr int kMaxSize = 2147483000;

is_status check_dense(const dense_desc *d) {
  if (!d) return IS_ERR_INVALID_ARG;
  if (d->n < 0 || d->len < 0 || d->in < 1 || d->features < 1) return IS_ERR_INVALID_ARG;
  if (d->activation < IS_ACT_NONE || d->activation > IS_ACT_SILU || d->w_stride < 0) return IS_ERR_INVALID_ARG;
  if ((d->dtype != IS_F16 && d->dtype != IS_BF16) || d->in % 8) return IS_ERR_UNSUPPORTED;
  // Rounded up to whole tiles they are still ints.
  for (const int size : {d->len, d->in, d->features})
    if (size > kMaxSize) return IS_ERR_UNSUPPORTED;
  const is_tokens tx = rows(d->n, d->len, d->x_stride), tr = rows(d->n, d->len, d->residual_stride),
                  to = rows(d->n, d->len, d->out_stride);
  is_status st = check_tokens(tx, d->in, 2);
  if (st == IS_OK) st = check_tokens(tr, d->features, 2);
  if (st == IS_OK) st = check_tokens(to, d->features, 2);
  if (st != IS_OK) return st;
  if ((tx.n > 1 && tx.batch_stride % 8) || (tx.len > 1 && tx.token_stride % 8) || (d->features > 1 && d->w_stride % 8))
    return IS_ERR_MISALIGNED;
  const int64_t most = (int64_t)1 << 21;
  if ((tx.len > 1 && tx.token_stride > most) || (tx.len == 1 && tx.n > 1 && tx.batch_stride > most) ||
      (d->features > 1 && d->w_stride > most))
    return IS_ERR_UNSUPPORTED;
  if ((double)d->features * d->w_stride * 2 > kMaxBytes) return IS_ERR_UNSUPPORTED;
  if (!empty(to) && !distinct(to, d->features)) return IS_ERR_INVALID_ARG;
  return IS_OK;
}

is_status run_dense(const is::DensePlan &p, const dense_desc &d, const void *x, const void *w, const float *bias,
                    const void *residual, void *out, void *ws, size_t ws_bytes, hipStream_t stream) {
  const is_tokens tx = rows(d.n, d.len, d.x_stride), tr = rows(d.n, d.len, d.residual_stride),
                  to = rows(d.n, d.len, d.out_stride);
  if (empty(to)) return IS_OK;
  if (!x || !w || !out) return IS_ERR_INVALID_ARG;
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(out, 16) || misaligned(residual, 16) || misaligned(bias, 4))
    return IS_ERR_MISALIGNED;
  const size_t need = is::dense_workspace(p);
  if (need > 0) {
    if (!ws || ws_bytes < need) return IS_ERR_WORKSPACE;
    if (misaligned(ws, 16)) return IS_ERR_MISALIGNED;
  }
  const char *wp = static_cast<const char *>(w), *bp = reinterpret_cast<const char *>(bias),
             *sp = static_cast<const char *>(ws);
  const Range o = range(out, to, d.features, 2), s = {sp, need ? sp + need : sp};
  const Range read[3] = {range(x, tx, d.in, 2), {wp, wp + ((size_t)(d.features - 1) * d.w_stride + d.in) * 2},
                         {bp, bp ? bp + 4 * (size_t)d.features : bp}};
  for (const Range &r : read)
    if (intersect(o, r) || intersect(s, r)) return IS_ERR_INVALID_ARG;
  if (residual) {
    const Range r = range(residual, tr, d.features, 2);
    if (!(residual == out && same_strides(tr, to)) && intersect(o, r)) return IS_ERR_INVALID_ARG;
    if (intersect(s, r)) return IS_ERR_INVALID_ARG;
  }
  if (intersect(o, s)) return IS_ERR_INVALID_ARG;
  return is::report_hip(is::launch_dense(p, x, w, bias, residual, out, ws, stream));
}

}  // namespace

extern "C" {

is_status block_norm_forward(const block_norm_desc *d, const void *x, const void *y, const void *gate,
                             const float *post_weight, const float *weight, const float *bias, const void *scale,
                             const void *shift, void *x_out, void *out, hipStream_t stream) {
  if (!d) return IS_ERR_INVALID_ARG;
  return run_norm(*d, {x, y, gate, scale, shift, post_weight, weight, bias, x_out, out}, stream);
}

is_status dense_create(const dense_desc *d, dense_plan *out) {
  if (!out) return IS_ERR_INVALID_ARG;
  *out = nullptr;
  const is_status st = check_dense(d);
  if (st != IS_OK) return st;
  is::DensePlan p;
  memset(&p, 0, sizeof(p));
  p.asked = p.d = *d;
  if (!is::configure_dense(p)) return IS_ERR_UNSUPPORTED;
  dense_plan_s *h = new (std::nothrow) dense_plan_s;
  if (!h) return IS_ERR_NO_MEMORY;
  h->p = p;
  *out = h;
  return IS_OK;
}

void dense_destroy(dense_plan plan) { delete plan; }

is_status dense_workspace_size(dense_plan plan, size_t *bytes) {
  if (!plan || !bytes) return IS_ERR_INVALID_ARG;
  *bytes = is::dense_workspace(plan->p);
  return IS_OK;
}

is_status dense_get_plan_info(dense_plan plan, conv2d_plan_info *info) {
  if (!plan || !info) return IS_ERR_INVALID_ARG;
  const is::DensePlan &p = plan->p;
  const dense_desc &d = p.asked;
  memset(info, 0, sizeof(*info));
  strncpy(info->kernel, p.name, sizeof(info->kernel) - 1);
  info->grid_x = (int)(p.d.n * p.row_tiles * p.feature_tiles);
  info->grid_y = p.splits;
  info->grid_z = 1;
  info->block = p.block;
  info->lds_bytes = p.lds;
  info->tile_w = p.tile_features;
  info->tile_h = p.tile_rows;
  const double r = (double)d.n * d.len;
  info->flops = 2.0 * r * d.in * d.features;
  info->bytes = 2.0 * (r * d.in + (double)d.in * d.features + r * d.features);
  return IS_OK;
}

is_status dense_forward(dense_plan plan, const void *x, const void *w, const float *bias, const void *residual,
                        void *out, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!plan) return IS_ERR_INVALID_ARG;
  return run_dense(plan->p, plan->p.asked, x, w, bias, residual, out, workspace, workspace_bytes, stream);
}

}  // extern "C"

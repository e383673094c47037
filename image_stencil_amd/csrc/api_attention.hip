// api_attention.hip -- the C ABI of the attention operators: argument checks,
// plans and launches. Like the convolution entry points it validates on the
// host, before any GPU call, and only enqueues kernels.
#include <math.h>
#include <string.h>

#include <new>

#include "attention.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "tokens.hpp"

struct rotary_plan_s {
  is::RotaryPlan p;
};
struct cross_attention_plan_s {
  is::AttentionPlan p;
};

using namespace is::arguments;

namespace {

constexpr long double kTwoPi = 6.283185307179586476925286766559L;
is_status check_rotary(const rotary_desc *d) {
  if (!d) return IS_ERR_INVALID_ARG;
  if (d->d < 1 || d->rot < 0 || d->rot > d->d || (d->rot & 1) || d->axes < 1) return IS_ERR_INVALID_ARG;
  if (d->d > IS_MAX_HEAD_DIM || d->axes > 3) return IS_ERR_UNSUPPORTED;
  const int pairs = d->rot / 2;
  if (pairs % d->axes) return IS_ERR_INVALID_ARG;
  if (d->layout != IS_ROTARY_HALF && d->layout != IS_ROTARY_INTERLEAVED) return IS_ERR_INVALID_ARG;
  if (d->scaling < IS_ROTARY_UNSCALED || d->scaling > IS_ROTARY_RAMP) return IS_ERR_INVALID_ARG;
  if (!(d->base > 0.0) || !isfinite(d->base)) return IS_ERR_INVALID_ARG;
  if (!((float)d->magnitude > 0.f) || !isfinite((float)d->magnitude)) return IS_ERR_INVALID_ARG;   // used in fp32
  if (d->scaling != IS_ROTARY_UNSCALED && (!(d->factor >= 1.0) || !isfinite(d->factor))) return IS_ERR_INVALID_ARG;
  if (d->scaling == IS_ROTARY_NTK && pairs / d->axes == 1) return IS_ERR_UNSUPPORTED;
  if (d->scaling == IS_ROTARY_RAMP &&
      (d->original_len < 1 || !(d->ramp_low >= 0.0) || !(d->ramp_high > d->ramp_low) || !isfinite(d->ramp_high)))
    return IS_ERR_INVALID_ARG;
  return IS_OK;
}

// In 80 bits, and rounded once: in 64 the powers and quotients would be off by up to
// 9 halves of a last bit, which far positions multiply.
void frequencies(is::RotaryPlan &p) {
  typedef long double real;
  const rotary_desc &d = p.d;
  const int per = p.per_axis = d.rot / 2 / d.axes;
  const real base = d.scaling == IS_ROTARY_NTK && per > 1 ? d.base * powl(d.factor, (real)per / (per - 1)) : d.base;
  for (int i = 0; i < per; ++i) {
    real f = powl(base, -(real)i / per);
    if (d.scaling == IS_ROTARY_LINEAR) f /= d.factor;
    if (d.scaling == IS_ROTARY_RAMP) {
      real keep = (d.original_len * f / kTwoPi - d.ramp_low) / ((real)d.ramp_high - d.ramp_low);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      f = f * keep + f / d.factor * (1 - keep);
    }
    p.freq[i] = (double)f;
    // A position is a whole number: whole turns of it never count.
    const real turns = f / kTwoPi - rintl(f / kTwoPi);
    for (int axis = 0; axis < d.axes; ++axis) p.turns[axis * per + i] = (double)turns;
  }
}

bool dtype_ok(is_dtype t) { return t == IS_F32 || t == IS_F16 || t == IS_BF16; }

// Bytes of a part's position rows, and the range they are read from.
double positions_bytes(const is::RotaryPlan &p, const is::RotaryPart &a) {
  return 4.0 * ((double)(a.xt.n - 1) * a.pos_batch_stride + (double)a.xt.len * p.d.axes);
}
Range positions_range(const is::RotaryPlan &p, const is::RotaryPart &a) {
  const char *c = reinterpret_cast<const char *>(a.positions);
  return {c, p.d.rot > 0 ? c + (size_t)positions_bytes(p, a) : c};
}
Range weight_range(const is::RotaryPlan &p, const is::RotaryPart &a) {
  const char *c = reinterpret_cast<const char *>(a.weight);
  return {c, c ? c + 4 * (size_t)p.d.d : c};
}

// One tensor of a rotary call: its checks, before any GPU call.
is_status check_part(const is::RotaryPlan &p, is_dtype dtype, const is::RotaryPart &a) {
  const int es = element_bytes(dtype), d = p.d.d;
  is_status st = check_tokens(a.xt, d, es);
  if (st == IS_OK) st = check_tokens(a.yt, d, es);
  if (st != IS_OK) return st;
  if (a.xt.n != a.yt.n || a.xt.len != a.yt.len || a.xt.heads != a.yt.heads) return IS_ERR_INVALID_ARG;
  if (a.pos_batch_stride < 0) return IS_ERR_INVALID_ARG;
  if (empty(a.xt)) return IS_OK;
  if (!distinct(a.yt, d)) return IS_ERR_INVALID_ARG;
  if (!a.x || !a.y || (p.d.rot > 0 && !a.positions)) return IS_ERR_INVALID_ARG;
  if (misaligned(a.x, 16) || misaligned(a.y, 16) || misaligned(a.positions, 4) || misaligned(a.weight, 16))
    return IS_ERR_MISALIGNED;
  const Range out = range(a.y, a.yt, d, es);
  const bool in_place = a.x == a.y && same_strides(a.xt, a.yt);
  if (!in_place && intersect(range(a.x, a.xt, d, es), out)) return IS_ERR_INVALID_ARG;
  if (p.d.rot > 0 && positions_bytes(p, a) > kMaxBytes) return IS_ERR_UNSUPPORTED;
  const Range pos = positions_range(p, a), weight = weight_range(p, a);
  if (intersect(pos, out) || intersect(weight, out)) return IS_ERR_INVALID_ARG;
  return IS_OK;
}

// What one part writes must not be what the other reads or writes: they run in one
// launch, in no order.
bool apart(const is::RotaryPlan &p, is_dtype dtype, const is::RotaryPart &a, const is::RotaryPart &b) {
  if (empty(a.xt) || empty(b.xt)) return true;
  const int es = element_bytes(dtype), d = p.d.d;
  const Range out = range(a.y, a.yt, d, es);
  return !collide(a.y, a.yt, b.x, b.xt, d, es) && !collide(a.y, a.yt, b.y, b.yt, d, es) &&
         !intersect(out, positions_range(p, b)) && !intersect(out, weight_range(p, b));
}

is_status run_rotary(const is::RotaryPlan &p, is_dtype dtype, int norm, float eps, const is::RotaryPart *parts,
                     int nparts, hipStream_t stream) {
  for (int i = 0; i < nparts; ++i) {
    const is_status st = check_part(p, dtype, parts[i]);
    if (st != IS_OK) return st;
  }
  if (nparts == 2 && !(apart(p, dtype, parts[0], parts[1]) && apart(p, dtype, parts[1], parts[0])))
    return IS_ERR_INVALID_ARG;
  const int vec = is::rotary_vector_width(p, dtype);
  double blocks = 0.0;
  for (int i = 0; i < nparts; ++i) blocks += (double)is::rotary_blocks(p, vec, parts[i].xt);
  if (blocks * is::kRotaryBlock > is::kMaxThreads) return IS_ERR_UNSUPPORTED;
  if (blocks == 0.0) return IS_OK;
  return is::report_hip(is::launch_rotary(p, dtype, norm, eps, parts, nparts, stream));
}

is_status check_attention(const cross_attention_desc *d) {
  if (!d) return IS_ERR_INVALID_ARG;
  if (d->n < 0 || d->lq < 0 || d->lk < 0 || d->hq < 1 || d->hkv < 1 || d->hq % d->hkv || d->d < 1)
    return IS_ERR_INVALID_ARG;
  if (!isfinite(is::score_factor(d->scale)) || d->mask_batch_stride < 0) return IS_ERR_INVALID_ARG;
  if ((d->dtype != IS_F16 && d->dtype != IS_BF16) || d->d % 8 || d->d > IS_MAX_HEAD_DIM) return IS_ERR_UNSUPPORTED;
  const is_tokens t[4] = {tokens(d->n, d->lq, d->hq, d->q_stride), tokens(d->n, d->lk, d->hkv, d->k_stride),
                          tokens(d->n, d->lk, d->hkv, d->v_stride), tokens(d->n, d->lq, d->hq, d->out_stride)};
  for (const is_tokens &x : t) {
    const is_status st = check_tokens(x, d->d, 2);
    if (st != IS_OK) return st;
  }
  for (const is_tokens &x : t)
    if ((x.n > 1 && x.batch_stride % 8) || (x.len > 1 && x.token_stride % 8) || (x.heads > 1 && x.head_stride % 8))
      return IS_ERR_MISALIGNED;
  if (!empty(t[3]) && !distinct(t[3], d->d)) return IS_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 23;
  if (d->lk > 1 && (d->k_stride[1] > most || d->v_stride[1] > most)) return IS_ERR_UNSUPPORTED;
  if ((double)d->lq * (d->hq / d->hkv) > 2147483000.0 || (double)d->lk > 2147483000.0) return IS_ERR_UNSUPPORTED;
  if ((double)d->n * d->mask_batch_stride > kMaxBytes) return IS_ERR_UNSUPPORTED;
  return IS_OK;
}

is_status run_attention(const is::AttentionPlan &p, const void *q, const void *k, const void *v,
                        const uint8_t *mask, const int32_t *lengths, void *out, float *lse, void *ws,
                        size_t ws_bytes, hipStream_t stream) {
  const cross_attention_desc &d = p.d;
  const is_tokens tq = tokens(d.n, d.lq, d.hq, d.q_stride), tk = tokens(d.n, d.lk, d.hkv, d.k_stride),
                  tv = tokens(d.n, d.lk, d.hkv, d.v_stride), to = tokens(d.n, d.lq, d.hq, d.out_stride);
  if (empty(to)) return IS_OK;
  if (!q || !out || (d.lk > 0 && (!k || !v))) return IS_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(lengths, 4) ||
      (d.lk > 0 && (misaligned(k, 16) || misaligned(v, 16))))
    return IS_ERR_MISALIGNED;
  const size_t need = is::attention_workspace(p);
  if (need > 0) {
    if (!ws || ws_bytes < need) return IS_ERR_WORKSPACE;
    if (misaligned(ws, 16)) return IS_ERR_MISALIGNED;
  }
  const char *l = reinterpret_cast<const char *>(lse), *w = static_cast<const char *>(ws);
  const char *m = reinterpret_cast<const char *>(mask), *n = reinterpret_cast<const char *>(lengths);
  const Range written[3] = {range(out, to, d.d, 2),
                            {l, l ? l + 4 * (size_t)d.n * d.hq * d.lq : l},
                            {w, need ? w + need : w}};
  const Range read[5] = {range(q, tq, d.d, 2), range(k, tk, d.d, 2), range(v, tv, d.d, 2),
                         {m, m ? m + (size_t)(d.n - 1) * d.mask_batch_stride + d.lk : m},
                         {n, n ? n + 4 * (size_t)d.n : n}};
  for (int i = 0; i < 3; ++i) {
    for (const Range &r : read)
      if (intersect(written[i], r)) return IS_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (intersect(written[i], written[j])) return IS_ERR_INVALID_ARG;
  }
  return is::report_hip(is::launch_attention(p, q, k, v, mask, lengths, out, lse, ws, stream));
}

}  // namespace

extern "C" {

is_status rotary_create(const rotary_desc *d, rotary_plan *out) {
  if (!out) return IS_ERR_INVALID_ARG;
  *out = nullptr;
  const is_status st = check_rotary(d);
  if (st != IS_OK) return st;
  rotary_plan_s *h = new (std::nothrow) rotary_plan_s;
  if (!h) return IS_ERR_NO_MEMORY;
  memset(&h->p, 0, sizeof(h->p));
  h->p.d = *d;
  frequencies(h->p);
  *out = h;
  return IS_OK;
}

void rotary_destroy(rotary_plan plan) { delete plan; }

is_status rotary_get_frequencies(rotary_plan plan, double *f, int max, int *count) {
  if (!plan || !count || max < 0 || (max > 0 && !f)) return IS_ERR_INVALID_ARG;
  *count = plan->p.per_axis;
  for (int i = 0; i < plan->p.per_axis && i < max; ++i) f[i] = plan->p.freq[i];
  return IS_OK;
}

is_status rotary_forward(rotary_plan plan, is_dtype dtype, const is_tokens *xt, const void *x,
                         const int32_t *positions, int64_t pos_batch_stride, const is_tokens *yt, void *y,
                         hipStream_t stream) {
  if (!plan || !xt || !yt) return IS_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return IS_ERR_UNSUPPORTED;
  const is::RotaryPart part = {x, y, nullptr, positions, pos_batch_stride, *xt, *yt};
  return run_rotary(plan->p, dtype, 0, 0.f, &part, 1, stream);
}

is_status qk_norm_rotary_forward(rotary_plan plan, const qk_norm_desc *d, const void *q, const void *k,
                                 const float *q_weight, const float *k_weight, const int32_t *q_positions,
                                 const int32_t *k_positions, void *q_out, void *k_out, hipStream_t stream) {
  if (!plan || !d) return IS_ERR_INVALID_ARG;
  if (!dtype_ok(d->dtype)) return IS_ERR_UNSUPPORTED;
  if ((d->norm != IS_NORM_RMS && d->norm != IS_NORM_LAYER) || !(d->eps >= 0.f) || !isfinite(d->eps))
    return IS_ERR_INVALID_ARG;
  const is::RotaryPart parts[2] = {{q, q_out, q_weight, q_positions, d->q_pos_batch_stride, d->q, d->q_out},
                                   {k, k_out, k_weight, k_positions, d->k_pos_batch_stride, d->k, d->k_out}};
  return run_rotary(plan->p, d->dtype, d->norm, d->eps, parts, 2, stream);
}

is_status cross_attention_create(const cross_attention_desc *d, cross_attention_plan *out) {
  if (!out) return IS_ERR_INVALID_ARG;
  *out = nullptr;
  const is_status st = check_attention(d);
  if (st != IS_OK) return st;
  is::AttentionPlan p;
  memset(&p, 0, sizeof(p));
  p.d = *d;
  p.scale = d->scale != 0.f ? d->scale : (float)(1.0 / sqrt((double)d->d));
  if (!is::configure_attention(p)) return IS_ERR_UNSUPPORTED;
  cross_attention_plan_s *h = new (std::nothrow) cross_attention_plan_s;
  if (!h) return IS_ERR_NO_MEMORY;
  h->p = p;
  *out = h;
  return IS_OK;
}

void cross_attention_destroy(cross_attention_plan plan) { delete plan; }

is_status cross_attention_workspace_size(cross_attention_plan plan, size_t *bytes) {
  if (!plan || !bytes) return IS_ERR_INVALID_ARG;
  *bytes = is::attention_workspace(plan->p);
  return IS_OK;
}

is_status cross_attention_get_plan_info(cross_attention_plan plan, conv2d_plan_info *info) {
  if (!plan || !info) return IS_ERR_INVALID_ARG;
  const is::AttentionPlan &p = plan->p;
  const cross_attention_desc &d = p.d;
  memset(info, 0, sizeof(*info));
  strncpy(info->kernel, p.name, sizeof(info->kernel) - 1);
  info->grid_x = (int)p.workgroups;
  info->grid_y = p.splits;
  info->grid_z = 1;
  info->block = p.block;
  info->lds_bytes = p.lds;
  info->tile_w = p.split_keys;
  info->tile_h = p.tile_rows;
  info->flops = 4.0 * d.n * d.lq * (double)d.lk * d.hq * d.d;
  info->bytes = 4.0 * d.n * ((double)d.lq * d.hq + (double)d.lk * d.hkv) * d.d;
  return IS_OK;
}

is_status cross_attention_forward(cross_attention_plan plan, const void *q, const void *k, const void *v,
                                  const uint8_t *key_mask, const int32_t *key_lengths, void *out, float *lse,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!plan) return IS_ERR_INVALID_ARG;
  return run_attention(plan->p, q, k, v, key_mask, key_lengths, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"

// api_held.hip -- the C ABI of states held in 8 bits and of the attention to them:
// argument checks, plans and launches, on the host and before any GPU call.
#include <math.h>
#include <string.h>

#include <new>

#include "common.hpp"
#include "held.hpp"
#include "internal.hpp"
#include "tokens.hpp"

struct held_attention_plan_s {
  is::HeldPlan p;
};

using namespace is::arguments;

namespace {

is_status check_states(const held_states_desc *d) {
  if (!d) return IS_ERR_INVALID_ARG;
  if (d->n < 0 || d->len < 0 || d->heads < 1 || d->d < 1) return IS_ERR_INVALID_ARG;
  if ((d->dtype != IS_F16 && d->dtype != IS_BF16) || d->d % 8 || d->d > IS_MAX_HEAD_DIM) return IS_ERR_UNSUPPORTED;
  const double records = (double)d->n * d->heads * is::held_blocks(d->len);
  if (records * 256.0 > is::kMaxThreads || (double)d->len > 2147483000.0) return IS_ERR_UNSUPPORTED;
  if (records * 64 * is::held_padded(d->d) > kMaxBytes) return IS_ERR_UNSUPPORTED;
  return IS_OK;
}

Range store_range(const held_states_desc &d, const void *held) {
  const char *p = static_cast<const char *>(held);
  return {p, p ? p + is::held_bytes(d) : p};
}

is_status check_store(const held_states_desc &d, const void *held, size_t bytes) {
  if (is::held_bytes(d) == 0) return IS_OK;
  if (!held) return IS_ERR_INVALID_ARG;
  if (misaligned(held, 16)) return IS_ERR_MISALIGNED;
  return bytes < is::held_bytes(d) ? IS_ERR_WORKSPACE : IS_OK;
}

// The tensors of a store or load and the place in the states they stand for.
is_status check_sides(const held_states_desc &d, const is_tokens *kt, const void *k, const is_tokens *vt, const void *v,
                      int at) {
  if (!kt || !vt) return IS_ERR_INVALID_ARG;
  const is_tokens *t[2] = {kt, vt};
  for (const is_tokens *x : t) {
    const is_status st = check_tokens(*x, d.d, 2);
    if (st != IS_OK) return st;
    if (x->n != d.n || x->heads != d.heads || x->len != kt->len) return IS_ERR_INVALID_ARG;
  }
  if (at < 0 || at > d.len || kt->len > d.len - at) return IS_ERR_INVALID_ARG;
  if (empty(*kt)) return IS_OK;
  if (!k || !v) return IS_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16)) return IS_ERR_MISALIGNED;
  return IS_OK;
}

is::HeldSide side(const is_tokens &t, const void *p) { return {p, t.batch_stride, t.token_stride, t.head_stride}; }

is_status check_attention(const held_attention_desc *d) {
  if (!d) return IS_ERR_INVALID_ARG;
  const is_status st = check_states(&d->held);
  if (st != IS_OK) return st;
  const held_states_desc &h = d->held;
  if (d->lq < 0 || d->hq < 1 || d->hq % h.heads) return IS_ERR_INVALID_ARG;
  if (!isfinite(is::score_factor(d->scale)) || d->mask_batch_stride < 0) return IS_ERR_INVALID_ARG;
  const is_tokens q = tokens(h.n, d->lq, d->hq, d->q_stride), o = tokens(h.n, d->lq, d->hq, d->out_stride);
  for (const is_tokens *x : {&q, &o}) {
    const is_status s = check_tokens(*x, h.d, 2);
    if (s != IS_OK) return s;
    if ((x->n > 1 && x->batch_stride % 8) || (x->len > 1 && x->token_stride % 8) || (x->heads > 1 && x->head_stride % 8))
      return IS_ERR_MISALIGNED;
  }
  if (!empty(o) && !distinct(o, h.d)) return IS_ERR_INVALID_ARG;
  if ((double)d->lq * (d->hq / h.heads) > 2147483000.0) return IS_ERR_UNSUPPORTED;
  if ((double)h.n * d->mask_batch_stride > kMaxBytes) return IS_ERR_UNSUPPORTED;
  return IS_OK;
}

is_status run_attention(const is::HeldPlan &p, const void *q, const void *held, size_t held_size, const uint8_t *mask,
                        const int32_t *lengths, void *out, float *lse, void *ws, size_t ws_bytes, hipStream_t stream) {
  const held_attention_desc &d = p.d;
  const held_states_desc &h = d.held;
  const is_tokens tq = tokens(h.n, d.lq, d.hq, d.q_stride), to = tokens(h.n, d.lq, d.hq, d.out_stride);
  if (empty(to)) return IS_OK;
  const is_status st = check_store(h, held, held_size);
  if (st != IS_OK) return st;
  if (!q || !out) return IS_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(lengths, 4)) return IS_ERR_MISALIGNED;
  const size_t need = is::held_workspace(p);
  if (need > 0) {
    if (!ws || ws_bytes < need) return IS_ERR_WORKSPACE;
    if (misaligned(ws, 16)) return IS_ERR_MISALIGNED;
  }
  const char *l = reinterpret_cast<const char *>(lse), *w = static_cast<const char *>(ws);
  const char *m = reinterpret_cast<const char *>(mask), *n = reinterpret_cast<const char *>(lengths);
  const Range written[3] = {range(out, to, h.d, 2),
                            {l, l ? l + 4 * (size_t)h.n * d.hq * d.lq : l},
                            {w, need ? w + need : w}};
  const Range read[4] = {range(q, tq, h.d, 2), store_range(h, held),
                         {m, m ? m + (size_t)(h.n - 1) * d.mask_batch_stride + h.len : m},
                         {n, n ? n + 4 * (size_t)h.n : n}};
  for (int i = 0; i < 3; ++i) {
    for (const Range &r : read)
      if (intersect(written[i], r)) return IS_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (intersect(written[i], written[j])) return IS_ERR_INVALID_ARG;
  }
  return is::report_hip(is::launch_held_attention(p, q, held, mask, lengths, out, lse, ws, stream));
}

}  // namespace

extern "C" {

is_status held_states_size(const held_states_desc *d, size_t *bytes) {
  if (!bytes) return IS_ERR_INVALID_ARG;
  const is_status st = check_states(d);
  if (st == IS_OK) *bytes = is::held_bytes(*d);
  return st;
}

is_status held_store(const held_states_desc *d, const is_tokens *kt, const void *k, const is_tokens *vt, const void *v,
                     const uint8_t *key_mask, int64_t key_mask_stride, const int32_t *key_lengths, int at, void *held,
                     size_t held_size, hipStream_t stream) {
  is_status st = check_states(d);
  if (st == IS_OK) st = check_sides(*d, kt, k, vt, v, at);
  if (st != IS_OK) return st;
  if (at % IS_HELD_BLOCK || key_mask_stride < 0) return IS_ERR_INVALID_ARG;
  if ((double)d->n * key_mask_stride > kMaxBytes) return IS_ERR_UNSUPPORTED;
  if (misaligned(key_lengths, 4)) return IS_ERR_MISALIGNED;
  if (empty(*kt)) return IS_OK;
  st = check_store(*d, held, held_size);
  if (st != IS_OK) return st;
  const char *m = reinterpret_cast<const char *>(key_mask), *n = reinterpret_cast<const char *>(key_lengths);
  const Range to = store_range(*d, held);
  for (const Range &r : {range(k, *kt, d->d, 2), range(v, *vt, d->d, 2),
                         Range{m, m ? m + (size_t)(d->n - 1) * key_mask_stride + kt->len : m},
                         Range{n, n ? n + 4 * (size_t)d->n : n}})
    if (intersect(to, r)) return IS_ERR_INVALID_ARG;
  return is::report_hip(is::launch_held_store(*d, side(*kt, k), side(*vt, v), kt->len, at, key_mask, key_mask_stride,
                                              key_lengths, held, stream));
}

is_status held_load(const held_states_desc *d, const void *held, size_t held_size, int at, const is_tokens *kt,
                    void *k, const is_tokens *vt, void *v, hipStream_t stream) {
  is_status st = check_states(d);
  if (st == IS_OK) st = check_sides(*d, kt, k, vt, v, at);
  if (st != IS_OK) return st;
  if (empty(*kt)) return IS_OK;
  st = check_store(*d, held, held_size);
  if (st != IS_OK) return st;
  if (!distinct(*kt, d->d) || !distinct(*vt, d->d)) return IS_ERR_INVALID_ARG;
  const Range rk = range(k, *kt, d->d, 2), rv = range(v, *vt, d->d, 2), from = store_range(*d, held);
  // Slices of one packed buffer lie between each other; that they are apart is the caller's.
  if (intersect(rk, from) || intersect(rv, from) || collide(k, *kt, v, *vt, d->d, 2)) return IS_ERR_INVALID_ARG;
  return is::report_hip(is::launch_held_load(*d, held, at, kt->len, side(*kt, k), side(*vt, v), false, stream));
}

is_status held_attention_create(const held_attention_desc *d, held_attention_plan *out) {
  if (!out) return IS_ERR_INVALID_ARG;
  *out = nullptr;
  const is_status st = check_attention(d);
  if (st != IS_OK) return st;
  is::HeldPlan p;
  memset(&p, 0, sizeof(p));
  p.d = *d;
  p.scale = d->scale != 0.f ? d->scale : (float)(1.0 / sqrt((double)d->held.d));
  if (!is::configure_held(p)) return IS_ERR_UNSUPPORTED;
  held_attention_plan_s *h = new (std::nothrow) held_attention_plan_s;
  if (!h) return IS_ERR_NO_MEMORY;
  h->p = p;
  *out = h;
  return IS_OK;
}

void held_attention_destroy(held_attention_plan plan) { delete plan; }

is_status held_attention_workspace_size(held_attention_plan plan, size_t *bytes) {
  if (!plan || !bytes) return IS_ERR_INVALID_ARG;
  *bytes = is::held_workspace(plan->p);
  return IS_OK;
}

is_status held_attention_get_plan_info(held_attention_plan plan, conv2d_plan_info *info) {
  if (!plan || !info) return IS_ERR_INVALID_ARG;
  const is::HeldPlan &p = plan->p;
  const held_states_desc &h = p.d.held;
  memset(info, 0, sizeof(*info));
  strncpy(info->kernel, p.name, sizeof(info->kernel) - 1);
  info->grid_x = (int)(p.direct ? p.workgroups : p.loaded.workgroups);
  info->grid_y = p.direct ? p.splits : p.loaded.splits;
  info->grid_z = 1;
  info->block = p.direct ? p.block : p.loaded.block;
  info->lds_bytes = p.direct ? p.lds : p.loaded.lds;
  info->tile_w = p.direct ? p.split_blocks * IS_HELD_BLOCK : p.loaded.split_keys;
  info->tile_h = p.direct ? 32 : p.loaded.tile_rows;
  info->flops = 4.0 * h.n * p.d.lq * (double)h.len * p.d.hq * h.d;
  info->bytes = 4.0 * h.n * p.d.lq * (double)p.d.hq * h.d + 2.0 * h.n * (double)h.len * h.heads * h.d;
  return IS_OK;
}

is_status held_attention_forward(held_attention_plan plan, const void *q, const void *held, size_t held_size,
                                 const uint8_t *key_mask, const int32_t *key_lengths, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!plan) return IS_ERR_INVALID_ARG;
  return run_attention(plan->p, q, held, held_size, key_mask, key_lengths, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"

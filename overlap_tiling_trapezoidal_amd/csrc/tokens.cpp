// Host side of the token operators: a plan's sequences, the rotation's
// frequency table, argument checks and workspace sizes.  Plain C++, no GPU
// code, so it builds with a host compiler too.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <new>

#include "layer_internal.h"

namespace tdp {

int check_seqs(const char* fn, const char* name, const tdp_seqs* s, SeqsDev* out) {
  if (!s) return fail(TDP_EINVAL, "%s: null %s", fn, name);
  if (s->num_seqs < 1 || s->len_group < 1)
    return fail(TDP_EINVAL, "%s: %s needs num_seqs >= 1 and len_group >= 1 (got %d, %d)", fn, name, s->num_seqs,
                s->len_group);
  if (s->max_rows < 1 || s->max_rows > (1 << 24))
    return fail(TDP_ESHAPE, "%s: %s.max_rows %d outside [1, 2^24]", fn, name, s->max_rows);
  if (s->total_rows < 1 || s->total_rows > INT32_MAX)
    return fail(TDP_ESHAPE, "%s: %s.total_rows %lld outside [1, 2^31)", fn, name, (long long)s->total_rows);
  if (!s->row_range && s->total_rows != (int64_t)s->num_seqs * s->max_rows)
    return fail(TDP_EINVAL, "%s: %s without row_range needs total_rows = num_seqs * max_rows (got %lld, %d * %d)", fn,
                name, (long long)s->total_rows, s->num_seqs, s->max_rows);
  if ((reinterpret_cast<uintptr_t>(s->row_range) & 7) || (reinterpret_cast<uintptr_t>(s->seq_len) & 3))
    return fail(TDP_EINVAL, "%s: %s.row_range must be 8-byte aligned and seq_len 4-byte aligned", fn, name);
  if (out) {
    out->S = s->num_seqs;
    out->max_rows = s->max_rows;
    out->total = s->total_rows;
    out->range = s->row_range;
    out->len = s->seq_len;
    out->by_group = make_fastdiv((uint32_t)s->len_group);
  }
  return TDP_OK;
}

int check_heads(const char* fn, const char* name, const tdp_heads* t, const tdp_seqs* s, int32_t head_dim,
                int32_t dtype, HeadsDev* out) {
  if (!t || !t->data) return fail(TDP_EINVAL, "%s: null %s", fn, name);
  if (reinterpret_cast<uintptr_t>(t->data) & 15) return fail(TDP_EINVAL, "%s: %s must be 16-byte aligned", fn, name);
  if (t->heads < 1 || t->heads > kMaxHeads)
    return fail(TDP_ESHAPE, "%s: %s.heads %d outside [1, %d]", fn, name, t->heads, kMaxHeads);
  const int64_t unit = 16 / dtype_bytes(dtype);
  const int64_t st[3] = {t->seq_stride, t->row_stride, t->head_stride};
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % unit != 0 || st[i] > (int64_t)1 << 40)
      return fail(TDP_EINVAL, "%s: %s's strides must be multiples of 16 bytes (%lld elements) in [0, 2^40], got %lld",
                  fn, name, (long long)unit, (long long)st[i]);
  out->data = static_cast<char*>(t->data);
  out->seq_stride = t->seq_stride;
  out->row_stride = t->row_stride;
  out->head_stride = t->head_stride;
  out->heads = t->heads;
  return TDP_OK;
}

int check_head_counts(const char* fn, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
  if (q_heads < 1 || k_heads < 1 || q_heads > kMaxHeads || q_heads % k_heads != 0 || head_dim < 8)
    return fail(TDP_ESHAPE, "%s: needs heads in [1, %d], q's a multiple of k's, and head_dim >= 8 (got %d, %d, %d)", fn,
                kMaxHeads, q_heads, k_heads, head_dim);
  return TDP_OK;
}

int check_weights(const char* fn, const tdp_seqs* seqs, int32_t num_weights) {
  if (seqs->num_seqs > (1 << 30))
    return fail(TDP_ESHAPE, "%s: num_seqs %d exceeds 2^30", fn, seqs->num_seqs);
  if (num_weights < 1 || num_weights > seqs->num_seqs)
    return fail(TDP_EINVAL, "%s: num_weights must be in [1, num_seqs] (got %d of %d)", fn, num_weights,
                seqs->num_seqs);
  return TDP_OK;
}

int check_product(const char* fn, const tdp_seqs* seqs, int32_t num_weights, int32_t in_features,
                  int32_t out_features) {
  const int st = check_seqs(fn, "seqs", seqs, nullptr);
  if (st != TDP_OK) return st;
  for (const int32_t f : {in_features, out_features})
    if (f < 8 || f % 8 != 0 || f > TDP_MAX_FEATURES)
      return fail(TDP_ESHAPE, "%s: features must be multiples of 8 in [8, %d] (got %d and %d)", fn, TDP_MAX_FEATURES,
                  in_features, out_features);
  return check_weights(fn, seqs, num_weights);
}

int check_window(const char* fn, const tdp_window* w) {
  if (!w) return fail(TDP_EINVAL, "%s: null window", fn);
  if (w->step < 1 || w->step > (1 << 24))
    return fail(TDP_ESHAPE, "%s: window.step %d outside [1, 2^24]", fn, w->step);
  if (w->back < 0 || w->ahead < 0 || w->sinks < 0 || w->back > TDP_WINDOW_ALL || w->ahead > TDP_WINDOW_ALL ||
      w->sinks > TDP_WINDOW_ALL)
    return fail(TDP_EINVAL, "%s: window.back, ahead and sinks must be in [0, 2^30] (got %d, %d, %d)", fn, w->back,
                w->ahead, w->sinks);
  return TDP_OK;
}

int check_rows(const char* fn, const char* name, const tdp_rows* t, int32_t dtype, HeadsDev* out) {
  if (!t || !t->data) return fail(TDP_EINVAL, "%s: null %s", fn, name);
  if (reinterpret_cast<uintptr_t>(t->data) & 15) return fail(TDP_EINVAL, "%s: %s must be 16-byte aligned", fn, name);
  const int64_t unit = 16 / dtype_bytes(dtype);
  const int64_t st[2] = {t->seq_stride, t->row_stride};
  for (int i = 0; i < 2; ++i)
    if (st[i] < 0 || st[i] % unit != 0 || st[i] > (int64_t)1 << 40)
      return fail(TDP_EINVAL, "%s: %s's strides must be multiples of 16 bytes (%lld elements) in [0, 2^40], got %lld",
                  fn, name, (long long)unit, (long long)st[i]);
  out->data = static_cast<char*>(t->data);
  out->seq_stride = t->seq_stride;
  out->row_stride = t->row_stride;
  out->head_stride = 0;
  out->heads = 1;
  return TDP_OK;
}

}  // namespace tdp

using namespace tdp;

extern "C" {

int tdp_plan_sequences(const tdp_plan* plan, int64_t* row_range) {
  if (!plan || !row_range) return fail(TDP_EINVAL, "tdp_plan_sequences: null argument");
  const PlanDev& p = plan->dev;
  int64_t s = 0;
  for (int slot = 0; slot < p.T_local; ++slot) {
    int i, j, k;
    tile_grid(p, p.rank + slot * p.world, i, j, k);
    const TileSlot ts = tile_slot(p, i, j, k);
    for (int b = 0; b < p.B; ++b, ++s) {
      row_range[2 * s] = ts.row_base + (int64_t)b * ts.cap;
      row_range[2 * s + 1] = row_range[2 * s] + ts.cap;
    }
  }
  return TDP_OK;
}

int tdp_rope_create(const tdp_rope_config* cfg, const double* freqs, tdp_rope** out) {
  if (!cfg || !out) return fail(TDP_EINVAL, "tdp_rope_create: null argument");
  *out = nullptr;
  const tdp_rope_config c = *cfg;
  if (c.head_dim < 8 || c.head_dim % 8 != 0 || c.head_dim > TDP_MAX_ROPE_DIM)
    return fail(TDP_ESHAPE, "head_dim must be a multiple of 8 in [8, %d] (got %d)", TDP_MAX_ROPE_DIM, c.head_dim);
  int64_t sum = 0;
  for (int a = 0; a < 3; ++a) {
    if (c.rot_dim[a] < 0 || c.rot_dim[a] % 2 != 0)
      return fail(TDP_ESHAPE, "rot_dim[%d] must be even and >= 0 (got %d)", a, c.rot_dim[a]);
    sum += c.rot_dim[a];
  }
  if (sum > c.head_dim)
    return fail(TDP_ESHAPE, "rot_dim adds up to %lld, more than head_dim %d", (long long)sum, c.head_dim);
  if (c.pairing != TDP_PAIR_INTERLEAVED && c.pairing != TDP_PAIR_HALVES)
    return fail(TDP_EINVAL, "unknown pairing %d", c.pairing);
  if (c.point != TDP_POINT_MIDDLE && c.point != TDP_POINT_START)
    return fail(TDP_EINVAL, "unknown point %d", c.point);
  if (sum && !freqs) return fail(TDP_EINVAL, "tdp_rope_create: null freqs");
  tdp_rope* r = new (std::nothrow) tdp_rope;
  if (!r) return fail(TDP_EINVAL, "out of host memory");
  memset(r, 0, sizeof *r);
  r->cfg = c;
  RopeDev& d = r->dev;
  d.D = c.head_dim;
  d.pairs = (int32_t)(sum / 2);
  for (int a = 0; a < 3; ++a) d.half[a] = c.rot_dim[a] / 2;
  d.pair_end[0] = d.half[0];
  d.pair_end[1] = d.half[0] + d.half[1];
  d.pairing = c.pairing;
  d.point = c.point;
  for (int i = 0; i < d.pairs; ++i) {
    if (!isfinite(freqs[i]) || fabs(freqs[i]) > 1e6) {
      delete r;
      return fail(TDP_EINVAL, "freqs[%d] must be finite and at most 1e6 radians per unit", i);
    }
    const double turns = freqs[i] / 6.283185307179586476925286766559 * (c.point == TDP_POINT_MIDDLE ? 0.5 : 1.0);
    d.hi[i] = (float)turns;
    d.lo[i] = (float)(turns - (double)d.hi[i]);
  }
  *out = r;
  return TDP_OK;
}

void tdp_rope_destroy(tdp_rope* rope) { delete rope; }

int64_t tdp_qk_norm_rope_workspace(const tdp_rope* rope, const tdp_seqs* seqs, int32_t q_heads, int32_t k_heads) {
  if (!rope || q_heads < 1 || k_heads < 1 || check_seqs("tdp_qk_norm_rope_workspace", "seqs", seqs, nullptr) != TDP_OK)
    return 0;
  const NormParts n = norm_parts(*seqs, q_heads, k_heads);
  return align256((int64_t)(n.q + n.k) * rope->cfg.head_dim * 4);
}

int64_t tdp_attention_workspace(const tdp_seqs* q_seqs, const tdp_seqs* k_seqs, int32_t q_heads, int32_t k_heads,
                                int32_t head_dim) {
  const char* fn = "tdp_attention_workspace";
  if (check_seqs(fn, "q_seqs", q_seqs, nullptr) != TDP_OK || check_seqs(fn, "k_seqs", k_seqs, nullptr) != TDP_OK ||
      check_head_counts(fn, q_heads, k_heads, head_dim) != TDP_OK)
    return 0;
  return attention_workspace(*q_seqs, *k_seqs, nullptr, q_heads, k_heads, head_dim);
}

int64_t tdp_attention_backward_workspace(const tdp_seqs* q_seqs, const tdp_seqs* k_seqs, int32_t q_heads,
                                         int32_t k_heads, int32_t head_dim) {
  const char* fn = "tdp_attention_backward_workspace";
  if (check_seqs(fn, "q_seqs", q_seqs, nullptr) != TDP_OK || check_seqs(fn, "k_seqs", k_seqs, nullptr) != TDP_OK ||
      check_head_counts(fn, q_heads, k_heads, head_dim) != TDP_OK)
    return 0;
  return backward_workspace(*q_seqs, *k_seqs, nullptr, q_heads, k_heads, head_dim);
}

int64_t tdp_window_attention_workspace(const tdp_seqs* q_seqs, const tdp_seqs* k_seqs, const tdp_window* window,
                                       int32_t q_heads, int32_t k_heads, int32_t head_dim) {
  const char* fn = "tdp_window_attention_workspace";
  if (check_window(fn, window) != TDP_OK || check_seqs(fn, "q_seqs", q_seqs, nullptr) != TDP_OK ||
      check_seqs(fn, "k_seqs", k_seqs, nullptr) != TDP_OK ||
      check_head_counts(fn, q_heads, k_heads, head_dim) != TDP_OK)
    return 0;
  return attention_workspace(*q_seqs, *k_seqs, window, q_heads, k_heads, head_dim);
}

int64_t tdp_window_attention_backward_workspace(const tdp_seqs* q_seqs, const tdp_seqs* k_seqs,
                                                const tdp_window* window, int32_t q_heads, int32_t k_heads,
                                                int32_t head_dim) {
  const char* fn = "tdp_window_attention_backward_workspace";
  if (check_window(fn, window) != TDP_OK || check_seqs(fn, "q_seqs", q_seqs, nullptr) != TDP_OK ||
      check_seqs(fn, "k_seqs", k_seqs, nullptr) != TDP_OK ||
      check_head_counts(fn, q_heads, k_heads, head_dim) != TDP_OK)
    return 0;
  return backward_workspace(*q_seqs, *k_seqs, window, q_heads, k_heads, head_dim);
}

int64_t tdp_layer_norm_workspace(const tdp_seqs* seqs, int32_t channels, int32_t num_weights) {
  const char* fn = "tdp_layer_norm_workspace";
  if (check_seqs(fn, "seqs", seqs, nullptr) != TDP_OK) return 0;
  if (channels < 8 || channels % 8 != 0 || channels > TDP_MAX_CHANNELS) {
    fail(TDP_ESHAPE, "%s: channels %d out of range", fn, channels);
    return 0;
  }
  if (check_weights(fn, seqs, num_weights) != TDP_OK) return 0;
  return align256(layer_norm_parts(*seqs, channels, num_weights) * num_weights * 2 * channels * 4);
}

int64_t tdp_grouped_product_workspace(const tdp_seqs* seqs, int32_t num_weights, int32_t in_features,
                                      int32_t out_features, int32_t dtype) {
  const char* fn = "tdp_grouped_product_workspace";
  if (check_product(fn, seqs, num_weights, in_features, out_features) != TDP_OK || !dtype_bytes(dtype)) return 0;
  return rows_workspace(*seqs, out_features, in_features, dtype, kNarrowY, flat_rows(*seqs, num_weights));
}

int64_t tdp_grouped_product_backward_workspace(const tdp_seqs* seqs, int32_t num_weights, int32_t in_features,
                                               int32_t out_features, int32_t dtype) {
  const char* fn = "tdp_grouped_product_backward_workspace";
  if (check_product(fn, seqs, num_weights, in_features, out_features) != TDP_OK || !dtype_bytes(dtype)) return 0;
  const int64_t a = rows_workspace(*seqs, in_features, out_features, dtype, kNarrowDx, flat_rows(*seqs, num_weights));
  const int64_t b = weight_workspace(*seqs, num_weights, in_features, out_features, dtype);
  return a > b ? a : b;  // dx and dW take turns
}

}  // extern "C"

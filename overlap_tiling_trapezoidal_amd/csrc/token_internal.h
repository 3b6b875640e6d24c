// The token operators' host objects and the forms their kernels take:
// sequences of rows, strided (rows, heads, head_dim) tensors and the
// rotation's frequencies.  Shared by the host side (tokens.cpp) and the
// kernels (rope.hip, attention.hip).
#pragma once

#include <stdint.h>

#include "plan_internal.h"

namespace tdp {

constexpr int kMaxPairs = TDP_MAX_ROPE_DIM / 2;

struct SeqsDev {
  int32_t S, max_rows;
  int64_t total;
  const int64_t* range;
  const int32_t* len;
  FastDiv by_group;
};

struct HeadsDev {
  char* data;
  int64_t seq_stride, row_stride, head_stride;  // elements
  int32_t heads;
};

// The rotation, passed by value.  Frequencies are turns per position unit as
// two floats (hi + lo), for the point actually summed: half of them for the
// middle, whose kernel adds start + end.
struct RopeDev {
  int32_t D, pairs;    // head_dim; pairs that turn
  int32_t pair_end[2];  // pairs of the time axis; of time and height
  int32_t half[3];     // pairs per axis
  int32_t pairing, point;
  float hi[kMaxPairs], lo[kMaxPairs];
};

// A sliding window (step 0: none).
struct WindowDev {
  int32_t step, back, ahead, sinks;
  FastDiv by_step;
};
TDP_HD int64_t window_step(const WindowDev& w, int p) {  // floor(p / step), p > -2^30
  return p >= 0 ? (int64_t)fastdiv((uint32_t)p, w.by_step)
                : -(int64_t)fastdiv((uint32_t)(w.step - 1 - p), w.by_step);
}
TDP_HD int clamp_row(int64_t x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : (int)x; }
// Keys [lo, hi) that the query at place p among `len` keys sees, besides the
// first rows below hi.
struct KeySpan {
  int lo, hi;
};
TDP_HD KeySpan key_span(const WindowDev& w, int p, int len) {
  const int64_t t = window_step(w, p);
  KeySpan k;
  k.hi = clamp_row((t + 1 + w.ahead) * w.step, 0, len);
  k.lo = clamp_row((t - w.back) * w.step, 0, k.hi);
  return k;
}
// Rows [lo, hi) of `len` queries that see key j; query i stands at i + off.
struct RowSpan {
  int lo, hi;
};
TDP_HD RowSpan row_span(const WindowDev& w, int j, int off, int len) {
  const int64_t t = window_step(w, j);
  RowSpan r;
  r.lo = clamp_row((t - w.ahead) * w.step - off, 0, len);
  r.hi = j < w.sinks ? len : clamp_row((t + w.back + 1) * w.step - off, r.lo, len);
  return r;
}
inline WindowDev window_dev(const tdp_window& w) {
  return {w.step, w.back, w.ahead, w.sinks, make_fastdiv((uint32_t)w.step)};
}
int check_window(const char* fn, const tdp_window* w);

// Host checks: TDP_OK and the device form, or the status with its message.
int check_seqs(const char* fn, const char* name, const tdp_seqs* s, SeqsDev* out);
int check_heads(const char* fn, const char* name, const tdp_heads* t, const tdp_seqs* s, int32_t head_dim,
                int32_t dtype, HeadsDev* out);
int check_rows(const char* fn, const char* name, const tdp_rows* t, int32_t dtype, HeadsDev* out);
constexpr int32_t kMaxHeads = 65536;
int check_head_counts(const char* fn, int32_t q_heads, int32_t k_heads, int32_t head_dim);
// Workgroups of `rows`-row blocks over every sequence: S * ceil(max_rows / rows).
inline int64_t seq_blocks(const tdp_seqs& s, int rows) {
  return (int64_t)s.num_seqs * ((s.max_rows + rows - 1) / rows);
}

// Partial sums of the norm weights' gradients: one row of head_dim floats per
// workgroup of the backward launch.  A workgroup takes queries or keys; they
// share at most kNormParts workgroups in proportion to their heads (three per
// CU, what its registers allow at once: 187 us on 35 840 rows of 16 + 16 heads of
// 128 against 195 with 2048).
constexpr int kNormParts = 768;
constexpr int kNormRowsPerWg = 4;  // one row per wave
struct NormParts {
  int q, k;
};
inline NormParts norm_parts(const tdp_seqs& s, int32_t q_heads, int32_t k_heads) {
  const int64_t b = seq_blocks(s, kNormRowsPerWg);
  int64_t q = (int64_t)kNormParts * q_heads / ((int64_t)q_heads + k_heads);
  q = q < 1 ? 1 : (q > kNormParts - 1 ? kNormParts - 1 : q);
  const int64_t k = kNormParts - q;
  return {(int)(b < q ? b : q), (int)(b < k ? b : k)};
}

// Attention blocks.  The query axis of a key head is its group's query heads
// and rows together (entry m is row m / group, head m % group), so a shared
// key head's rows are read once for the whole group.
constexpr int kAttnBlockQ = 128;  // query entries per workgroup of the forward and dq kernels
constexpr int kAttnBlockK = 64;   // keys per step

// Key splits of the forward: few query blocks would leave most of the 256
// CUs idle while each walks all keys, so the keys are cut into parts of at
// least kAttnSplitKeys until about kAttnSplitBlocks workgroups run (one query row
// of 2 x 32 heads on 24 576 keys of 8 heads of 128: 44 us against 448 unsplit).
constexpr int kAttnSplitBlocks = 512;
constexpr int kAttnSplitKeys = 256;
constexpr int kAttnMaxSplits = 64;
// `per` blocks for each head of each sequence.  More of these than any launch holds
// are returned as they are, which is refused too and keeps products in 64 bits.
inline int64_t head_blocks(const tdp_seqs& s, int32_t heads, int64_t per) {
  const int64_t n = (int64_t)s.num_seqs * heads;
  return n > (1 << 24) ? n : n * per;
}
inline int64_t attention_blocks(const tdp_seqs& q, int32_t q_heads, int32_t k_heads) {
  const int64_t m = (int64_t)q.max_rows * (q_heads / k_heads);
  return head_blocks(q, k_heads, (m + kAttnBlockQ - 1) / kAttnBlockQ);
}
// Keys that a block of queries walks at most.
inline int64_t window_keys(const tdp_window* w, const tdp_seqs& q, const tdp_seqs& k) {
  if (!w) return k.max_rows;
  const int64_t rows = q.max_rows < kAttnBlockQ ? q.max_rows : kAttnBlockQ;
  const int64_t n = ((int64_t)w->back + w->ahead + 1 + (rows + w->step - 1) / w->step) * w->step + w->sinks;
  return n < k.max_rows ? n : k.max_rows;
}
inline int attention_splits(const tdp_seqs& q, int64_t keys, int32_t q_heads, int32_t k_heads) {
  const int64_t blocks = attention_blocks(q, q_heads, k_heads);
  if (blocks * 2 > kAttnSplitBlocks) return 1;
  int64_t n = kAttnSplitBlocks / blocks;
  const int64_t by_keys = keys / kAttnSplitKeys;
  if (n > by_keys) n = by_keys;
  if (n > kAttnMaxSplits) n = kAttnMaxSplits;
  return n < 2 ? 1 : (int)n;
}
// head_dim between them pays for the next (forward, 4 x 2240 rows, 16 bf16 heads:
// 40 dims 102 us, 64 105; 72 157, 96 165).
inline int attention_padded_dim(int32_t head_dim) { return head_dim <= 32 ? 32 : head_dim <= 64 ? 64 : 128; }
// Per split, sequence, key head and query entry: the unscaled sum (padded
// head_dim floats), then the maximum and the sum of weights (2 floats).
inline int64_t attention_workspace(const tdp_seqs& q, const tdp_seqs& k, const tdp_window* w, int32_t q_heads,
                                   int32_t k_heads, int32_t head_dim) {
  const int n = attention_splits(q, window_keys(w, q, k), q_heads, k_heads);
  if (n == 1) return 0;
  return align256((int64_t)n * q.num_seqs * q_heads * q.max_rows * (attention_padded_dim(head_dim) + 2) * 4);
}

// Row splits of the dk and dv kernel, for the same reason: parts of at least
// kDkvSplitRows query rows, until about kAttnSplitBlocks workgroups run (backward
// of 4 x 8960 rows, 16 heads on 4 of 64, a 77-token prompt: 130 us against 708).
constexpr int kDkvSplitRows = 512;
inline int64_t dkv_blocks(const tdp_seqs& k, int32_t k_heads) {
  return head_blocks(k, k_heads, (k.max_rows + kAttnBlockQ - 1) / kAttnBlockQ);
}
inline int dkv_splits(const tdp_seqs& k, int64_t rows, int32_t q_heads, int32_t k_heads) {
  const int64_t blocks = dkv_blocks(k, k_heads);
  if (blocks * 2 > kAttnSplitBlocks) return 1;
  int64_t n = kAttnSplitBlocks / blocks;
  const int64_t by_rows = rows * (q_heads / k_heads) / kDkvSplitRows;
  if (n > by_rows) n = by_rows;
  if (n > kAttnMaxSplits) n = kAttnMaxSplits;
  return n < 2 ? 1 : (int)n;
}
// With a window only the blocks that hold its first rows may be worth splitting:
// every later query sees them, where another key's rows span the window.  They
// are cut into parts of about a window's rows.
struct DkvSplit {
  int n;           // parts of the blocks that are split
  int64_t blocks;  // of a head's keys, the first ones, that are
  int64_t rows;    // their keys
};
inline DkvSplit dkv_split(const tdp_window* w, const tdp_seqs& q, const tdp_seqs& k, int32_t q_heads,
                          int32_t k_heads) {
  const int64_t all = ((int64_t)k.max_rows + kAttnBlockQ - 1) / kAttnBlockQ;
  int64_t seen = q.max_rows;  // rows that a key meets
  if (w) {
    const int64_t n = ((int64_t)w->back + w->ahead + 1) * w->step + kAttnBlockQ;
    seen = n < seen ? n : seen;
  }
  DkvSplit sp = {dkv_splits(k, w && w->sinks ? q.max_rows : seen, q_heads, k_heads), all, k.max_rows};
  if (sp.n == 1 && w && w->sinks) {
    const int64_t lead = ((int64_t)w->sinks + kAttnBlockQ - 1) / kAttnBlockQ, heavy = head_blocks(k, k_heads, lead);
    const int64_t part = seen > kDkvSplitRows ? seen : kDkvSplitRows;
    int64_t n = q.max_rows / part;
    if (n > 2 * kAttnSplitBlocks / heavy) n = 2 * kAttnSplitBlocks / heavy;  // many blocks fill the GPU unsplit
    if (n > kAttnMaxSplits) n = kAttnMaxSplits;
    if (n > 1 && lead < all) {
      sp.n = (int)n;
      sp.blocks = lead;
      sp.rows = lead * kAttnBlockQ;
    }
  }
  return sp;
}
// The backward's workspace: lse and delta, two floats per (query head, row), then per
// split, sequence, key head and key padded rows of dk, and the same of dv.
inline int64_t stats_bytes(const tdp_seqs& q, int32_t q_heads) {
  return align256((int64_t)q_heads * q.total_rows * 8);
}
inline int64_t backward_workspace(const tdp_seqs& q, const tdp_seqs& k, const tdp_window* w, int32_t q_heads,
                                  int32_t k_heads, int32_t head_dim) {
  const DkvSplit sp = dkv_split(w, q, k, q_heads, k_heads);
  const int64_t parts =
      sp.n == 1 ? 0 : (int64_t)sp.n * k.num_seqs * k_heads * sp.rows * attention_padded_dim(head_dim) * 8;
  return stats_bytes(q, q_heads) + align256(parts);
}

}  // namespace tdp

struct tdp_rope {
  tdp_rope_config cfg;
  tdp::RopeDev dev;
};

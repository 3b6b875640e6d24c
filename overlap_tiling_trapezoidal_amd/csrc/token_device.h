// Device helpers of the token operators: a sequence's rows and a tensor's
// addresses.
#pragma once

#include "device_common.h"
#include "token_internal.h"

namespace tdp {

// A sequence's first row, the rows its range spans, the rows outputs cover
// and the rows in use.  Values read from device memory are clamped, so no
// index leaves the tensors whatever the arrays hold.
struct SeqRows {
  int64_t row0;
  int span, cap, len;
};
__device__ inline SeqRows seq_rows(const SeqsDev& q, int s) {
  SeqRows r;
  if (q.range) {
    int64_t a = q.range[2 * (int64_t)s], b = q.range[2 * (int64_t)s + 1];
    a = a < 0 ? 0 : (a > q.total ? q.total : a);
    b = b < a ? a : (b > q.total ? q.total : b);
    r.row0 = a;
    r.span = (int)(b - a);  // total < 2^31
    r.cap = r.span < q.max_rows ? r.span : q.max_rows;
  } else {
    r.row0 = (int64_t)s * q.max_rows;
    r.span = r.cap = q.max_rows;
  }
  r.len = r.cap;
  if (q.len) {
    const int l = q.len[fastdiv((uint32_t)s, q.by_group)];
    r.len = l < 0 ? 0 : (l < r.cap ? l : r.cap);
  }
  return r;
}

// Element offset of a sequence's first row.
__device__ inline int64_t seq_base(const SeqsDev& q, const HeadsDev& t, int s, const SeqRows& r) {
  return q.range ? r.row0 * t.row_stride : (int64_t)s * t.seq_stride;
}

// Eight consecutive elements of a tensor as floats, and back (16 bytes of
// bf16, 32 of fp32; `e` is a multiple of 16 bytes).
template <int T>
__device__ inline void load8(const char* base, int64_t e, float* x) {
  if constexpr (T == TDP_BF16) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(base + 2 * e);
    InVec<TDP_BF16>::unpack(v, x);
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(base + 4 * e);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  }
}
template <int T>
__device__ inline void store8(char* base, int64_t e, const float* x) {
  if constexpr (T == TDP_BF16) {
    u32x4 v;
    v.x = pack_bf16x2(x[0], x[1]);
    v.y = pack_bf16x2(x[2], x[3]);
    v.z = pack_bf16x2(x[4], x[5]);
    v.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<u32x4*>(base + 2 * e) = v;
  } else {
    f32x4* p = reinterpret_cast<f32x4*>(base + 4 * e);
    p[0] = f32x4{x[0], x[1], x[2], x[3]};
    p[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
}

}  // namespace tdp

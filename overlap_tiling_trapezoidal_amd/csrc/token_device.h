// Device helpers of the token operators: a sequence's rows, a tensor's
// addresses, a lane's elements of a row and sums over lanes.
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

// The dims of a lane: bf16, eight in a row; fp32, four in each half of the
// head, so that each 16-byte access of neighbouring lanes is contiguous.
template <int T>
__device__ inline int lane_dim(int D, int chunk, int e) {
  return T == TDP_BF16 ? chunk * 8 + e : chunk * 4 + (e & 3) + (e >> 2) * (D / 2);
}
template <int T>
struct Raw {
  u32x4 v[T == TDP_BF16 ? 1 : 2];
  // p: the lane's first dim; half: bytes from the first quad to the second (fp32)
  __device__ inline void load(const char* p, int half, bool on) {
    v[0] = u32x4{0, 0, 0, 0};
    if constexpr (T == TDP_F32) v[1] = u32x4{0, 0, 0, 0};
    if (on) {
      v[0] = ld_nt(reinterpret_cast<const u32x4*>(p));
      if constexpr (T == TDP_F32) v[1] = ld_nt(reinterpret_cast<const u32x4*>(p + half));
    }
  }
  __device__ inline void unpack(float* x) const {
    InVec<T>::unpack(v[0], x);
    if constexpr (T == TDP_F32) InVec<T>::unpack(v[1], x + 4);
  }
  __device__ static inline void store(char* p, int half, const float* x) {
    if constexpr (T == TDP_BF16) {
      store_out<TDP_BF16, 8>(p, 0, x);
    } else {
      st_nt(reinterpret_cast<f32x4*>(p), f32x4{x[0], x[1], x[2], x[3]});
      st_nt(reinterpret_cast<f32x4*>(p + half), f32x4{x[4], x[5], x[6], x[7]});
    }
  }
};

template <int CTRL>
__device__ inline float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Sum over aligned groups of G lanes: quads by permutes, then mirrors of 8 and
// 16 lanes, then the swaps of neighbouring rows of 16 and of the wave's halves.
template <int G>
__device__ inline float group_sum(float v) {
  if constexpr (G >= 2) v += dpp<0xB1>(v);
  if constexpr (G >= 4) v += dpp<0x4E>(v);
  if constexpr (G >= 8) v += dpp<0x141>(v);
  if constexpr (G >= 16) v += dpp<0x140>(v);
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (G >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

}  // namespace tdp

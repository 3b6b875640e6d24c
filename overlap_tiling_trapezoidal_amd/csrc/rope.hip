// Rotation by three position axes, and the per-head norms of queries and
// keys with that rotation in the same pass, with their gradients (gfx950).
//
// Source of the positions: LTX-2 docs, "Tiled Data Parallelism (TDP)",
// "Position normalization" (each tile hands the model its own zero-based
// [start, end) intervals on time, height and width).
//
// All three kernels are bound by HBM bandwidth: a few operations per element
// read and written once.  A wave owns one row (token) at a time, all its heads:
// its lanes compute the row's angles once, one pair each, into LDS, and every
// head reuses them, so no table of cosines is stored or read (24 bytes of
// positions per row instead of 4 * head_dim).  A lane moves eight elements of
// a head (16 bytes of bf16), G lanes share a head (G = the power of two at or
// above head_dim / 8) and 64 / G heads go through the wave at once; the norm's
// sums run over the G lanes by cross-lane moves.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "token_device.h"

namespace tdp {
namespace {

constexpr int kWaves = 4;
constexpr int kTok = 64 * kWaves;

// cos and sin of 2*pi*(u * f), u = start + end or start, f = hi + lo turns per
// unit.  Whole turns leave the exact product u * hi inside one fma, before any
// rounding, and the parts that fp32 dropped (of start + end by the two-sum, of f
// in lo) are added to what remains, so the angle is good to about 2^-25 turns
// however far the position is.
__device__ inline void turn(float a, float b, bool middle, float hi, float lo, float* c, float* s) {
  float u = a, ue = 0.0f;
  if (middle) {
    u = a + b;
    const float bb = u - a;
    ue = (a - (u - bb)) + (b - bb);
  }
  const float t = fmaf(u, hi, -rintf(u * hi)) + fmaf(u, lo, ue * hi);
  sincospif(2.0f * t, s, c);
}

__device__ inline int pair_axis(const RopeDev& r, int p) { return (p >= r.pair_end[0]) + (p >= r.pair_end[1]); }

// One wave's cos/sin of a row: pair p at [p], and (1, 0) for the unturned dims
// at [pairs] and up (to pair 128).
struct Angles {
  float c[kMaxPairs + 1], s[kMaxPairs + 1];
};

__device__ inline void wave_lds_fence() {
  // LDS operations of one wave complete in order; only the compiler has to
  // keep the order, no other wave shares this memory.
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ inline void fill_angles(const RopeDev& r, const float* pos, const SeqRows& sr, int i, int lane, Angles* a) {
  const f32x2* base = reinterpret_cast<const f32x2*>(pos) + 3 * sr.row0 + i;
  for (int p = lane; p < r.D / 2 + 1; p += 64) {
    float c = 1.0f, s = 0.0f;
    if (p < r.pairs) {
      const f32x2 iv = base[(int64_t)pair_axis(r, p) * sr.span];
      turn(iv.x, iv.y, r.point == TDP_POINT_MIDDLE, r.hi[p], r.lo[p], &c, &s);
    }
    a->c[p] = c;
    a->s[p] = s;
  }
}

// Which angle and which partner each of a lane's eight dims uses.
template <bool HALVES>
struct LanePairs {
  int pair[HALVES ? 8 : 4];
  int src[HALVES ? 8 : 1];     // slot of the partner in the wave's exchange buffer
  float sign[HALVES ? 8 : 1];  // -1 on the first half of a section
  __device__ inline LanePairs(const RopeDev& r, int chunk, int group_lane0) {
    if constexpr (!HALVES) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = chunk * 4 + e;
        pair[e] = p < r.D / 2 ? p : r.D / 2;  // entries past `pairs` hold (1, 0)
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = chunk * 8 + e;
        pair[e] = r.D / 2;
        src[e] = e * 64 + group_lane0 + chunk;
        sign[e] = 0.0f;
        if (d < 2 * r.pairs) {
          const int ax = pair_axis(r, d / 2);
          const int first = ax == 0 ? 0 : r.pair_end[ax - 1];
          const int j = d - 2 * first, h = r.half[ax];
          const bool lower = j < h;
          const int dp = lower ? d + h : d - h;
          pair[e] = first + (lower ? j : j - h);
          src[e] = (dp & 7) * 64 + group_lane0 + (dp >> 3);
          sign[e] = lower ? -1.0f : 1.0f;
        }
      }
    }
  }
};

// The cos and signed sin of a lane's dims for one row.
template <bool HALVES>
struct LaneAngles {
  float c[HALVES ? 8 : 4], s[HALVES ? 8 : 4];
  __device__ inline LaneAngles(const LanePairs<HALVES>& lp, const Angles* a, float dir) {
#pragma unroll
    for (int e = 0; e < (HALVES ? 8 : 4); ++e) {
      c[e] = a->c[lp.pair[e]];
      s[e] = a->s[lp.pair[e]] * dir;
      if constexpr (HALVES) s[e] *= lp.sign[e];
    }
  }
};

template <bool HALVES>
__device__ inline void rotate8(const LanePairs<HALVES>& lp, const LaneAngles<HALVES>& la, float* ex, int lane,
                               float* x) {
  if constexpr (!HALVES) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = x[2 * e], b = x[2 * e + 1];
      x[2 * e] = fmaf(a, la.c[e], -b * la.s[e]);
      x[2 * e + 1] = fmaf(b, la.c[e], a * la.s[e]);
    }
  } else {
    // partners sit in other lanes: element e of lane l at e * 64 + l, so
    // writes and reads touch consecutive banks
    wave_lds_fence();
#pragma unroll
    for (int e = 0; e < 8; ++e) ex[e * 64 + lane] = x[e];
    wave_lds_fence();
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], la.c[e], ex[lp.src[e]] * la.s[e]);
  }
}

template <int G>
__device__ inline float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

struct RopeArgs {
  RopeDev rope;
  SeqsDev seqs;
  const float* pos;
  HeadsDev in[2], out[2];  // queries and keys (heads 0: none)
  const float* w[2];       // norm weights or null
  HeadsDev grad[2];        // backward: the outputs' gradients
  float* parts;            // backward: partial weight gradients
  float eps, dir;          // dir -1: inverse rotation
  uint32_t blocks;         // row blocks per sequence
};

// One row (sequence s, row i) per wave; workgroups cover every row once.
template <int T, int G, bool HALVES, bool NORM>
__global__ __launch_bounds__(kTok) void rope_kernel(const RopeArgs A) {
  __shared__ Angles ang[kWaves];
  __shared__ float exch[HALVES ? kWaves : 1][HALVES ? 512 : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int s = blockIdx.x / A.blocks;
  const int i = (blockIdx.x - s * A.blocks) * kWaves + wave;
  const SeqRows sr = seq_rows(A.seqs, s);
  if (i >= sr.cap) return;
  const int chunk = lane % G, grp = lane / G;
  const bool on = chunk * 8 < A.rope.D;
  const int nq = A.in[0].heads, H = nq + A.in[1].heads;
  constexpr int kPer = 64 / G;
  int64_t ib[2], ob[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    ib[t] = seq_base(A.seqs, A.in[t], s, sr) + i * A.in[t].row_stride + chunk * 8;
    ob[t] = seq_base(A.seqs, A.out[t], s, sr) + i * A.out[t].row_stride + chunk * 8;
  }
  if (i >= sr.len) {
    const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int h = grp; h < H; h += kPer) {
      const int t = h >= nq, hh = t ? h - nq : h;
      if (on) store8<T>(A.out[t].data, ob[t] + hh * A.out[t].head_stride, z);
    }
    return;
  }
  fill_angles(A.rope, A.pos, sr, i, lane, &ang[wave]);
  const LanePairs<HALVES> lp(A.rope, chunk, lane - chunk);
  wave_lds_fence();
  const LaneAngles<HALVES> la(lp, &ang[wave], A.dir);
  float w[2][8];
  if constexpr (NORM) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) w[t][e] = A.w[t] && on ? A.w[t][chunk * 8 + e] : 1.0f;
  }
  constexpr int U = 4;  // heads in flight per lane
  for (int h0 = 0; h0 < H; h0 += kPer * U) {
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * kPer + grp;
      const int t = h >= nq, hh = t ? h - nq : h;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = 0.0f;
      if (on && h < H) load8<T>(A.in[t].data, ib[t] + hh * A.in[t].head_stride, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * kPer + grp;
      const int t = h >= nq, hh = t ? h - nq : h;
      if constexpr (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[u][e], x[u][e], ss);
        ss = group_sum<G>(ss);
        const float r = 1.0f / sqrtf(ss / (float)A.rope.D + A.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] *= r * (t ? w[1][e] : w[0][e]);
      }
      rotate8<HALVES>(lp, la, exch[HALVES ? wave : 0], lane, x[u]);
      if (on && h < H) store8<T>(A.out[t].data, ob[t] + hh * A.out[t].head_stride, x[u]);
    }
  }
}

// Gradient of the norm and rotation: dx per row, and each workgroup's sums of
// the weights' gradients over its rows, in a fixed order.
template <int T, int G, bool HALVES>
__global__ __launch_bounds__(kTok) void norm_backward_kernel(const RopeArgs A) {
  __shared__ Angles ang[kWaves];
  __shared__ float exch[HALVES ? kWaves : 1][HALVES ? 512 : 1];
  __shared__ float red[kWaves][2][TDP_MAX_ROPE_DIM];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int chunk = lane % G, grp = lane / G;
  const bool on = chunk * 8 < A.rope.D;
  const int nq = A.in[0].heads, H = nq + A.in[1].heads;
  constexpr int kPer = 64 / G;
  const LanePairs<HALVES> lp(A.rope, chunk, lane - chunk);
  float w[2][8], dw[2][8];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[t][e] = A.w[t] && on ? A.w[t][chunk * 8 + e] : 1.0f;
      dw[t][e] = 0.0f;
    }
  const uint32_t nblk = A.blocks * (uint32_t)A.seqs.S;
  for (uint32_t blk = blockIdx.x; blk < nblk; blk += gridDim.x) {
    const int s = blk / A.blocks;
    const int i = (blk - s * A.blocks) * kWaves + wave;
    const SeqRows sr = seq_rows(A.seqs, s);
    if (i >= sr.cap) continue;
    int64_t ib[2], gb[2], ob[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      ib[t] = seq_base(A.seqs, A.in[t], s, sr) + i * A.in[t].row_stride + chunk * 8;
      gb[t] = seq_base(A.seqs, A.grad[t], s, sr) + i * A.grad[t].row_stride + chunk * 8;
      ob[t] = seq_base(A.seqs, A.out[t], s, sr) + i * A.out[t].row_stride + chunk * 8;
    }
    if (i >= sr.len) {
      const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int h = grp; h < H; h += kPer) {
        const int t = h >= nq, hh = t ? h - nq : h;
        if (on) store8<T>(A.out[t].data, ob[t] + hh * A.out[t].head_stride, z);
      }
      continue;
    }
    wave_lds_fence();
    fill_angles(A.rope, A.pos, sr, i, lane, &ang[wave]);
    wave_lds_fence();
    const LaneAngles<HALVES> la(lp, &ang[wave], -1.0f);
    constexpr int U = 2;
    for (int h0 = 0; h0 < H; h0 += kPer * U) {
      float x[U][8], g[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kPer + grp;
        const int t = h >= nq, hh = t ? h - nq : h;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = g[u][e] = 0.0f;
        if (on && h < H) {
          load8<T>(A.in[t].data, ib[t] + hh * A.in[t].head_stride, x[u]);
          load8<T>(A.grad[t].data, gb[t] + hh * A.grad[t].head_stride, g[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kPer + grp;
        const int t = h >= nq, hh = t ? h - nq : h;
        rotate8<HALVES>(lp, la, exch[HALVES ? wave : 0], lane, g[u]);
        float ss = 0.0f, gx = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[u][e], x[u][e], ss);
          gx = fmaf(g[u][e] * (t ? w[1][e] : w[0][e]), x[u][e], gx);
        }
        ss = group_sum<G>(ss);
        gx = group_sum<G>(gx);
        const float inv = 1.0f / (float)A.rope.D;
        const float r = 1.0f / sqrtf(ss * inv + A.eps);
        const float m = gx * inv * r * r;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float nx = g[u][e] * (x[u][e] * r);
          dw[0][e] += t ? 0.0f : nx;
          dw[1][e] += t ? nx : 0.0f;
          y[e] = r * fmaf(g[u][e], t ? w[1][e] : w[0][e], -x[u][e] * m);
        }
        if (on && h < H) store8<T>(A.out[t].data, ob[t] + hh * A.out[t].head_stride, y);
      }
    }
  }
  // the wave's groups, then its four waves
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = G; o < 64; o <<= 1) dw[t][e] += __shfl_xor(dw[t][e], o);
      if (grp == 0 && on) red[wave][t][chunk * 8 + e] = dw[t][e];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * A.rope.D; c += kTok) {
    const int t = c >= A.rope.D, d = t ? c - A.rope.D : c;
    A.parts[(int64_t)blockIdx.x * 2 * A.rope.D + c] = (red[0][t][d] + red[1][t][d]) + (red[2][t][d] + red[3][t][d]);
  }
}

// Sum the workgroups' partial rows: 16 columns per workgroup, 16 strided row
// sums per column joined in order.
__global__ __launch_bounds__(kTok) void norm_weights_kernel(const float* parts, int n, int D, float* dwq, float* dwk) {
  __shared__ float red[16][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;
  float v = 0.0f;
  if (c < 2 * D)
    for (int r = row; r < n; r += 16) v += parts[(int64_t)r * 2 * D + c];
  red[row][col] = v;
  __syncthreads();
  if (row == 0 && c < 2 * D) {
    float sum = 0.0f;
    for (int r = 0; r < 16; ++r) sum += red[r][col];
    float* out = c < D ? dwq : dwk;
    if (out) out[c < D ? c : c - D] = sum;
  }
}

template <int T, int G, bool NORM>
void launch_forward(const RopeArgs& a, uint32_t grid, hipStream_t st) {
  if (a.rope.pairing == TDP_PAIR_HALVES)
    hipLaunchKernelGGL((rope_kernel<T, G, true, NORM>), dim3(grid), dim3(kTok), 0, st, a);
  else
    hipLaunchKernelGGL((rope_kernel<T, G, false, NORM>), dim3(grid), dim3(kTok), 0, st, a);
}
template <int T, int G>
void launch_backward(const RopeArgs& a, uint32_t grid, hipStream_t st) {
  if (a.rope.pairing == TDP_PAIR_HALVES)
    hipLaunchKernelGGL((norm_backward_kernel<T, G, true>), dim3(grid), dim3(kTok), 0, st, a);
  else
    hipLaunchKernelGGL((norm_backward_kernel<T, G, false>), dim3(grid), dim3(kTok), 0, st, a);
}

enum class Mode { kRope, kNorm, kBackward };

template <int T, int G>
void launch_mode(Mode m, const RopeArgs& a, uint32_t grid, hipStream_t st) {
  if (m == Mode::kRope) launch_forward<T, G, false>(a, grid, st);
  if (m == Mode::kNorm) launch_forward<T, G, true>(a, grid, st);
  if (m == Mode::kBackward) launch_backward<T, G>(a, grid, st);
}
template <int T>
void launch_group(Mode m, const RopeArgs& a, uint32_t grid, hipStream_t st) {
  const int chunks = a.rope.D / 8;
  if (chunks == 1) launch_mode<T, 1>(m, a, grid, st);
  else if (chunks == 2) launch_mode<T, 2>(m, a, grid, st);
  else if (chunks <= 4) launch_mode<T, 4>(m, a, grid, st);
  else if (chunks <= 8) launch_mode<T, 8>(m, a, grid, st);
  else if (chunks <= 16) launch_mode<T, 16>(m, a, grid, st);
  else launch_mode<T, 32>(m, a, grid, st);
}

// Checks shared by the calls; fills everything but the tensors.
int begin(const char* fn, const tdp_rope* rope, const tdp_seqs* seqs, const float* pos, int32_t dtype, RopeArgs* a) {
  if (!rope) return fail(TDP_EINVAL, "%s: null rope", fn);
  if (!dtype_bytes(dtype)) return fail(TDP_EINVAL, "%s: dtype must be TDP_F32 or TDP_BF16 (got %d)", fn, dtype);
  const int st = check_seqs(fn, "seqs", seqs, &a->seqs);
  if (st != TDP_OK) return st;
  a->rope = rope->dev;
  if (rope->dev.pairs && (!pos || (reinterpret_cast<uintptr_t>(pos) & 7)))
    return fail(TDP_EINVAL, "%s: pos must be an 8-byte aligned device pointer", fn);
  a->pos = pos;
  a->blocks = (uint32_t)((seqs->max_rows + kWaves - 1) / kWaves);
  const int64_t items = seq_blocks(*seqs, kWaves) * kTok;
  if (items > 0xffffffffLL)
    return fail(TDP_ESHAPE, "%s: %lld work-items, more than one HIP launch holds", fn, (long long)items);
  return TDP_OK;
}

int check_in_place(const char* fn, const char* out_name, const tdp_heads* in, const tdp_heads* out) {
  if (in->heads != out->heads)
    return fail(TDP_EINVAL, "%s: %s has %d heads, its input %d", fn, out_name, out->heads, in->heads);
  if (in->data == out->data && (in->seq_stride != out->seq_stride || in->row_stride != out->row_stride ||
                                in->head_stride != out->head_stride))
    return fail(TDP_EINVAL, "%s: %s in place needs its input's strides", fn, out_name);
  return TDP_OK;
}

int check_pair(const char* fn, const char* in_name, const char* out_name, const tdp_heads* in, const tdp_heads* out,
               const tdp_seqs* seqs, int32_t dim, int32_t dtype, HeadsDev* di, HeadsDev* dout) {
  int st = check_heads(fn, in_name, in, seqs, dim, dtype, di);
  if (st == TDP_OK) st = check_heads(fn, out_name, out, seqs, dim, dtype, dout);
  if (st == TDP_OK) st = check_in_place(fn, out_name, in, out);
  return st;
}

int run(const char* fn, Mode m, const RopeArgs& a, int32_t dtype, uint32_t grid, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == TDP_BF16)
    launch_group<TDP_BF16>(m, a, grid, st);
  else
    launch_group<TDP_F32>(m, a, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

}  // namespace
}  // namespace tdp

using namespace tdp;

extern "C" {

int tdp_rope_apply(const tdp_rope* rope, const tdp_seqs* seqs, const float* pos, const tdp_heads* x,
                   const tdp_heads* y, int32_t dtype, int32_t inverse, void* stream) {
  const char* fn = "tdp_rope_apply";
  RopeArgs a = {};
  int st = begin(fn, rope, seqs, pos, dtype, &a);
  if (st == TDP_OK) st = check_pair(fn, "x", "y", x, y, seqs, rope->cfg.head_dim, dtype, &a.in[0], &a.out[0]);
  if (st != TDP_OK) return st;
  a.dir = inverse ? -1.0f : 1.0f;
  return run(fn, Mode::kRope, a, dtype, (uint32_t)seq_blocks(*seqs, kWaves), stream);
}

static int check_norm(const char* fn, float eps, const float* wq, const float* wk) {
  if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(TDP_EINVAL, "%s: eps must be finite and >= 0", fn);
  if ((reinterpret_cast<uintptr_t>(wq) | reinterpret_cast<uintptr_t>(wk)) & 3)
    return fail(TDP_EINVAL, "%s: weights must be 4-byte aligned", fn);
  return TDP_OK;
}

int tdp_qk_norm_rope(const tdp_rope* rope, const tdp_seqs* seqs, const float* pos, const tdp_heads* q,
                     const tdp_heads* k, const float* q_weight, const float* k_weight, const tdp_heads* q_out,
                     const tdp_heads* k_out, float eps, int32_t dtype, void* stream) {
  const char* fn = "tdp_qk_norm_rope";
  RopeArgs a = {};
  int st = begin(fn, rope, seqs, pos, dtype, &a);
  if (st == TDP_OK) st = check_pair(fn, "q", "q_out", q, q_out, seqs, rope->cfg.head_dim, dtype, &a.in[0], &a.out[0]);
  if (st == TDP_OK) st = check_pair(fn, "k", "k_out", k, k_out, seqs, rope->cfg.head_dim, dtype, &a.in[1], &a.out[1]);
  if (st == TDP_OK) st = check_norm(fn, eps, q_weight, k_weight);
  if (st != TDP_OK) return st;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.eps = eps;
  a.dir = 1.0f;
  return run(fn, Mode::kNorm, a, dtype, (uint32_t)seq_blocks(*seqs, kWaves), stream);
}

int tdp_qk_norm_rope_backward(const tdp_rope* rope, const tdp_seqs* seqs, const float* pos, const tdp_heads* q,
                              const tdp_heads* k, const float* q_weight, const float* k_weight,
                              const tdp_heads* dq_out, const tdp_heads* dk_out, const tdp_heads* dq,
                              const tdp_heads* dk, float* dq_weight, float* dk_weight, float eps, int32_t dtype,
                              void* workspace, void* stream) {
  const char* fn = "tdp_qk_norm_rope_backward";
  RopeArgs a = {};
  int st = begin(fn, rope, seqs, pos, dtype, &a);
  const int32_t D = st == TDP_OK ? rope->cfg.head_dim : 0;
  if (st == TDP_OK) st = check_heads(fn, "q", q, seqs, D, dtype, &a.in[0]);
  if (st == TDP_OK) st = check_heads(fn, "k", k, seqs, D, dtype, &a.in[1]);
  if (st == TDP_OK) st = check_pair(fn, "dq_out", "dq", dq_out, dq, seqs, D, dtype, &a.grad[0], &a.out[0]);
  if (st == TDP_OK) st = check_pair(fn, "dk_out", "dk", dk_out, dk, seqs, D, dtype, &a.grad[1], &a.out[1]);
  if (st == TDP_OK && (q->heads != dq->heads || k->heads != dk->heads))
    st = fail(TDP_EINVAL, "%s: dq and dk need the heads of q and k", fn);
  if (st == TDP_OK) st = check_norm(fn, eps, q_weight, k_weight);
  if (st == TDP_OK) st = check_norm(fn, eps, dq_weight, dk_weight);
  if (st == TDP_OK && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    st = fail(TDP_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
  if (st != TDP_OK) return st;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.eps = eps;
  a.parts = static_cast<float*>(workspace);
  const int parts = norm_parts(*seqs);
  st = run(fn, Mode::kBackward, a, dtype, (uint32_t)parts, stream);
  if (st != TDP_OK || (!dq_weight && !dk_weight)) return st;
  hipLaunchKernelGGL(norm_weights_kernel, dim3((2 * D + 15) / 16), dim3(kTok), 0,
                     reinterpret_cast<hipStream_t>(stream), a.parts, parts, D, dq_weight, dk_weight);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

}  // extern "C"

// Layer norm of rows and its gradients (gfx950).
//
//   y = (x - mean) r w + b,  r = 1 / sqrt(mean((x - mean)^2) + eps)
//   with n = (x - mean) r and g = dy w:
//   dx = r (g - mean(g) - n mean(g n)),  dw = sum of dy n,  db = sum of dy
//
// Bound by HBM bandwidth: a row is read once, stays in registers for its three
// sums, and is written once.  The sum of the elements alone leaves the mean off by
// a few 2^-24 of the row's offset, which every difference would carry (rows around
// 10^4 with a spread of 1: up to 10^-3).  The mean of the differences is that
// error, so they are lowered by it before their squares are summed, and an offset
// of the row costs no digits (taken from the squares' sum instead, it would cancel
// in rows of nearly one value).  The third sum costs up to 2 % in bf16 and 5 % in
// fp32 rows of 2048 and more (35840 of them 114 us against 109).  G lanes share a
// row, eight elements of it per lane NV times; rows wider than one wave holds take
// the workgroup.  A workgroup takes several blocks of rows, the next one's loads in
// flight while this one is worked on, and keeps the weights in registers.  247296
// rows of 2048 bf16 (2.03 GB) take 358 us, 5.7 TB/s of the 5.96 that a plain copy
// reaches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "layer_internal.h"
#include "token_device.h"

namespace tdp {
namespace {

constexpr int kTok = 256;

struct NormArgs {
  SeqsDev seqs;
  HeadsDev x, y, dy;  // y: the output; of the gradients dx
  const float *w, *b;
  float* parts;  // backward: (sets, parts, 2, C) sums of dw and db
  int32_t C, sets;
  uint32_t blocks, per_wg;  // row blocks per sequence; forward: blocks per workgroup
  uint32_t nparts;          // backward: workgroups per set of weights
  float eps;
};

// Sum over the G lanes of a row.  A row of the whole workgroup passes through
// `red`, one array per sum of a row: two barriers lie between two uses of one.
template <int G>
__device__ inline float row_sum(float v, float* red) {
  if constexpr (G <= 64) {
    return group_sum<G>(v);
  } else {
    v = group_sum<64>(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
  }
}
template <int G>
__device__ inline void row_sums(float& a, float& b, float* red) {
  if constexpr (G <= 64) {
    a = group_sum<G>(a);
    b = group_sum<G>(b);
  } else {
    a = group_sum<64>(a);
    b = group_sum<64>(b);
    if ((threadIdx.x & 63) == 0) {
      red[threadIdx.x >> 6] = a;
      red[4 + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = (red[0] + red[1]) + (red[2] + red[3]);
    b = (red[4] + red[5]) + (red[6] + red[7]);
  }
}

// A lane's part of rows: chunks lane, lane + G, ... of eight elements.
template <int T, int G, int NV>
struct Lane {
  static constexpr int R = kTok / G;  // rows of a block
  int chunk, sub, C, half;
  bool on[NV];
  __device__ inline Lane(int channels) {
    chunk = threadIdx.x % G;
    sub = threadIdx.x / G;
    C = channels;
    half = C * 2;
#pragma unroll
    for (int v = 0; v < NV; ++v) on[v] = (chunk + G * v) * 8 < C;
  }
  __device__ inline int dim(int v, int e) const { return lane_dim<T>(C, chunk + G * v, e); }
  __device__ inline char* at(const SeqsDev& q, const HeadsDev& t, int s, const SeqRows& r, int i) const {
    constexpr int eb = T == TDP_BF16 ? 2 : 4;
    return t.data + eb * (seq_base(q, t, s, r) + i * t.row_stride) + chunk * 16;
  }
  __device__ inline void load(const char* p, bool live, Raw<T>* raw) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v].load(p + v * G * 16, half, live && on[v]);
  }
  __device__ inline void store(char* p, bool owned, const float (*y)[8]) const {
    if (!owned) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (on[v]) Raw<T>::store(p + v * G * 16, half, y[v]);
  }
  // a row's differences from its mean: from the sum's, then from what that left
  __device__ inline void center(float (*x)[8], float m, float inv_c, float* red) const {
    float left = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[v][e] = on[v] ? x[v][e] - m : 0.0f;
        left += x[v][e];
      }
    left = row_sum<G>(left, red) * inv_c;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] = on[v] ? x[v][e] - left : 0.0f;
  }
  // a vector of weights (null: all `value`)
  __device__ inline void weights(const float* w, float value, float (*out)[8]) const {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) out[v][e] = w && on[v] ? w[dim(v, e)] : value;
  }
};

// A lane's row of a block: block t of the sequences s0, s0 + step, ...
struct RowOf {
  int s, i;
  SeqRows sr;
  __device__ inline void seek(const SeqsDev& q, uint32_t blocks, uint32_t t, int s0, int step, int rows, int sub) {
    const uint32_t n = t / blocks;
    s = s0 + step * (int)n;
    i = (int)(t - n * blocks) * rows + sub;
    sr = seq_rows(q, s);
  }
  __device__ inline bool live() const { return i < sr.len; }
  __device__ inline bool owned() const { return i < sr.cap; }
};

template <int T, int G, int NV>
__global__ __launch_bounds__(kTok) void layer_norm_kernel(const NormArgs A) {
  typedef Lane<T, G, NV> L;
  __shared__ float red[3][4];
  const L ln(A.C);
  const float inv_c = 1.0f / (float)A.C;
  const uint32_t n = A.blocks * (uint32_t)A.seqs.S;
  const uint32_t b0 = blockIdx.x * A.per_wg, b1 = b0 + A.per_wg < n ? b0 + A.per_wg : n;
  float w[NV][8], b[NV][8];
  int set = -1;
  RowOf nx;
  Raw<T> raw[NV];
  auto fetch = [&](uint32_t t) __attribute__((always_inline)) {
    nx.seek(A.seqs, A.blocks, t, 0, 1, L::R, ln.sub);
    ln.load(ln.at(A.seqs, A.x, nx.s, nx.sr, nx.i), nx.live(), raw);
  };
  fetch(b0);
  for (uint32_t t = b0; t < b1; ++t) {
    const RowOf at = nx;
    float x[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v].unpack(x[v]);
    if (t + 1 < b1) fetch(t + 1);
    if (at.i - ln.sub >= at.sr.cap) continue;  // no row of the block
    const int need = at.s % A.sets;
    if (need != set) {
      set = need;
      ln.weights(A.w ? A.w + (int64_t)set * A.C : nullptr, 1.0f, w);
      ln.weights(A.b ? A.b + (int64_t)set * A.C : nullptr, 0.0f, b);
    }
    float m = 0.0f, q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) m += x[v][e];
    m = row_sum<G>(m, red[0]) * inv_c;
    ln.center(x, m, inv_c, red[1]);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(x[v][e], x[v][e], q);
    const float r = __builtin_amdgcn_rsqf(fmaf(row_sum<G>(q, red[2]), inv_c, A.eps));
    const bool live = at.live();
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] = live ? fmaf(x[v][e] * r, w[v][e], b[v][e]) : 0.0f;
    ln.store(ln.at(A.seqs, A.y, at.s, at.sr, at.i), at.owned(), x);
  }
}

// dx, and each workgroup's sums of dw and db over its rows, fp32 in a fixed
// order.  A workgroup keeps to one set of weights.  On 35840 rows of 2048 bf16
// (440 MB) 82 us with the join, 5.4 TB/s; a workgroup per row, whose eight elements
// per lane need fewer registers, takes 99 for the barriers of its sums.
template <int T, int G, int NV>
__global__ __launch_bounds__(kTok) void layer_norm_backward_kernel(const NormArgs A) {
  typedef Lane<T, G, NV> L;
  __shared__ float red[3][8];
  __shared__ float join[G < 256 ? 4 : 1][G < 256 ? 8 * 64 : 1];
  const L ln(A.C);
  const float inv_c = 1.0f / (float)A.C;
  const int set = blockIdx.x / A.nparts;
  const uint32_t part = blockIdx.x - set * A.nparts;
  const uint32_t n = A.blocks * (uint32_t)((A.seqs.S - set + A.sets - 1) / A.sets);
  float w[NV][8], dw[NV][8], db[NV][8];
  ln.weights(A.w ? A.w + (int64_t)set * A.C : nullptr, 1.0f, w);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
  RowOf nx;
  Raw<T> rx[NV], rg[NV];
  auto fetch = [&](uint32_t t) __attribute__((always_inline)) {
    nx.seek(A.seqs, A.blocks, t, set, A.sets, L::R, ln.sub);
    ln.load(ln.at(A.seqs, A.x, nx.s, nx.sr, nx.i), nx.live(), rx);
    ln.load(ln.at(A.seqs, A.dy, nx.s, nx.sr, nx.i), nx.live(), rg);
  };
  if (part < n) fetch(part);
  for (uint32_t t = part; t < n; t += A.nparts) {
    const RowOf at = nx;
    float x[NV][8], g[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      rx[v].unpack(x[v]);
      rg[v].unpack(g[v]);
    }
    if (n - t > A.nparts) fetch(t + A.nparts);
    if (at.i - ln.sub >= at.sr.cap) continue;
    float m = 0.0f, mg = 0.0f, q = 0.0f, gx = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m += x[v][e];
        mg = fmaf(g[v][e], w[v][e], mg);
      }
    row_sums<G>(m, mg, red[0]);
    mg *= inv_c;
    ln.center(x, m * inv_c, inv_c, red[1]);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        q = fmaf(x[v][e], x[v][e], q);
        gx = fmaf(g[v][e] * w[v][e], x[v][e], gx);
      }
    row_sums<G>(q, gx, red[2]);
    const bool live = at.live();
    // a row past the end holds zeros, whose r is infinite when eps is 0
    const float r = live ? __builtin_amdgcn_rsqf(fmaf(q, inv_c, A.eps)) : 0.0f;
    const float c = gx * inv_c * r * r;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[v][e] = fmaf(g[v][e], x[v][e] * r, dw[v][e]);
        db[v][e] += g[v][e];
        x[v][e] = live ? r * (fmaf(g[v][e], w[v][e], -mg) - x[v][e] * c) : 0.0f;
      }
    ln.store(ln.at(A.seqs, A.y, at.s, at.sr, at.i), at.owned(), x);
  }
  // the wave's groups, then its four waves
  float* out = A.parts + (int64_t)blockIdx.x * 2 * A.C;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (G < 256) {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float a = k ? db[v][e] : dw[v][e];
#pragma unroll
          for (int o = G; o < 64; o <<= 1) a += __shfl_xor(a, o);
          join[wave][e * 64 + lane] = a;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * G; i += kTok) {
          const int slot = (i / G) * 64 + i % G, c = i % G + G * v;
          if (c * 8 < A.C)
            out[k * A.C + lane_dim<T>(A.C, c, i / G)] =
                (join[0][slot] + join[1][slot]) + (join[2][slot] + join[3][slot]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ln.on[v]) out[k * A.C + ln.dim(v, e)] = k ? db[v][e] : dw[v][e];
      }
    }
}

// Sum the workgroups' partial rows: 16 columns per workgroup, 16 strided row
// sums per column joined in order.
__global__ __launch_bounds__(kTok) void layer_norm_join_kernel(const float* parts, int nparts, int C, float* dw,
                                                               float* db) {
  __shared__ float red[16][17];
  const int per = (2 * C + 15) / 16;  // C is a multiple of 8: a block holds columns of both sums at most
  const int set = blockIdx.x / per;
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4, c = (blockIdx.x - set * per) * 16 + col;
  float v = 0.0f;
  if (c < 2 * C)
#pragma unroll 8
    for (int r = row; r < nparts; r += 16) v += parts[((int64_t)set * nparts + r) * 2 * C + c];
  red[row][col] = v;
  __syncthreads();
  if (row || c >= 2 * C) return;
  float* out = c < C ? dw : db;
  if (!out) return;
  float sum = 0.0f;
  for (int r = 0; r < 16; ++r) sum += red[r][col];
  out[(int64_t)set * C + (c < C ? c : c - C)] = sum;
}

#define TDP_NORM_LANES(call, T)                      \
  do {                                               \
    const int chunks = channels / 8;                 \
    if (chunks <= 8) call(T, 8, 1);                  \
    else if (chunks <= 16) call(T, 16, 1);           \
    else if (chunks <= 32) call(T, 32, 1);           \
    else if (chunks <= 64) call(T, 64, 1);           \
    else if (chunks <= 128) call(T, 64, 2);          \
    else if (chunks <= 256) call(T, 64, 4);          \
    else if (chunks <= 512) call(T, 256, 2);         \
    else call(T, 256, 4);                            \
  } while (0)

int begin(const char* fn, const tdp_seqs* seqs, const tdp_rows* x, const float* weight, int32_t num_weights,
          float eps, int32_t channels, int32_t dtype, NormArgs* A) {
  if (!dtype_bytes(dtype)) return fail(TDP_EINVAL, "%s: dtype must be TDP_F32 or TDP_BF16 (got %d)", fn, dtype);
  if (channels < 8 || channels % 8 != 0 || channels > TDP_MAX_CHANNELS)
    return fail(TDP_ESHAPE, "%s: channels must be a multiple of 8 in [8, %d] (got %d)", fn, TDP_MAX_CHANNELS,
                channels);
  if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(TDP_EINVAL, "%s: eps must be finite and >= 0", fn);
  int st = check_seqs(fn, "seqs", seqs, &A->seqs);
  if (st == TDP_OK) st = check_rows(fn, "x", x, dtype, &A->x);
  if (st != TDP_OK) return st;
  st = check_weights(fn, seqs, num_weights);
  if (st != TDP_OK) return st;
  if (reinterpret_cast<uintptr_t>(weight) & 3) return fail(TDP_EINVAL, "%s: weight must be 4-byte aligned", fn);
  A->w = weight;
  A->C = channels;
  A->sets = num_weights;
  A->eps = eps;
  A->blocks = (uint32_t)norm_blocks(seqs->max_rows, channels);
  return TDP_OK;
}

int check_same(const char* fn, const char* name, const tdp_rows* in, const tdp_rows* out) {
  if (in->data == out->data && (in->seq_stride != out->seq_stride || in->row_stride != out->row_stride))
    return fail(TDP_EINVAL, "%s: %s in place needs its input's strides", fn, name);
  return TDP_OK;
}

}  // namespace
}  // namespace tdp

using namespace tdp;

extern "C" {

int tdp_layer_norm(const tdp_seqs* seqs, const tdp_rows* x, const float* weight, const float* bias,
                   int32_t num_weights, const tdp_rows* y, float eps, int32_t channels, int32_t dtype,
                   void* stream) {
  const char* fn = "tdp_layer_norm";
  NormArgs A = {};
  int st = begin(fn, seqs, x, weight, num_weights, eps, channels, dtype, &A);
  if (st == TDP_OK) st = check_rows(fn, "y", y, dtype, &A.y);
  if (st == TDP_OK) st = check_same(fn, "y", x, y);
  if (st != TDP_OK) return st;
  if (reinterpret_cast<uintptr_t>(bias) & 3) return fail(TDP_EINVAL, "%s: bias must be 4-byte aligned", fn);
  A.b = bias;
  const int64_t blocks = (int64_t)A.blocks * seqs->num_seqs;
  // Blocks per workgroup, as long as 16 workgroups per CU remain: one leaves the
  // weights to be read again for every row, many leave few workgroups to even out
  // (247296 rows of 2048 bf16: 446 us with 1, 382 with 2, 357 with 4, 375 with 8).
  int64_t per = blocks / 4096;
  per = per < 1 ? 1 : per > 4 ? 4 : per;
  A.per_wg = (uint32_t)per;
  const int64_t grid = (blocks + per - 1) / per;
  if (blocks > INT32_MAX || grid * kTok > 0xffffffffLL)
    return fail(TDP_ESHAPE, "%s: %lld workgroups, more work-items than one HIP launch holds", fn, (long long)grid);
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
#define CALL(T, G, NV) hipLaunchKernelGGL((layer_norm_kernel<T, G, NV>), dim3((unsigned)grid), dim3(kTok), 0, hs, A)
  if (dtype == TDP_BF16) TDP_NORM_LANES(CALL, TDP_BF16);
  else TDP_NORM_LANES(CALL, TDP_F32);
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

int tdp_layer_norm_backward(const tdp_seqs* seqs, const tdp_rows* x, const float* weight, int32_t num_weights,
                            const tdp_rows* dy, const tdp_rows* dx, float* dweight, float* dbias, float eps,
                            int32_t channels, int32_t dtype, void* workspace, void* stream) {
  const char* fn = "tdp_layer_norm_backward";
  NormArgs A = {};
  int st = begin(fn, seqs, x, weight, num_weights, eps, channels, dtype, &A);
  if (st == TDP_OK) st = check_rows(fn, "dy", dy, dtype, &A.dy);
  if (st == TDP_OK) st = check_rows(fn, "dx", dx, dtype, &A.y);
  if (st == TDP_OK) st = check_same(fn, "dx", dy, dx);
  if (st == TDP_OK) st = check_same(fn, "dx", x, dx);
  if (st != TDP_OK) return st;
  if ((reinterpret_cast<uintptr_t>(dweight) | reinterpret_cast<uintptr_t>(dbias)) & 3)
    return fail(TDP_EINVAL, "%s: dweight and dbias must be 4-byte aligned", fn);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return fail(TDP_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
  if ((int64_t)A.blocks * seqs->num_seqs > INT32_MAX)
    return fail(TDP_ESHAPE, "%s: %lld blocks of rows, more than 2^31 - 1", fn,
                (long long)A.blocks * seqs->num_seqs);
  A.parts = static_cast<float*>(workspace);
  A.nparts = (uint32_t)layer_norm_parts(*seqs, channels, num_weights);
  const int64_t grid = (int64_t)A.nparts * num_weights, join = (int64_t)num_weights * ((2 * channels + 15) / 16);
  if ((grid > join ? grid : join) * kTok > 0xffffffffLL)
    return fail(TDP_ESHAPE, "%s: %lld workgroups, more work-items than one HIP launch holds", fn,
                (long long)(grid > join ? grid : join));
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
#define CALL(T, G, NV) \
  hipLaunchKernelGGL((layer_norm_backward_kernel<T, G, NV>), dim3((unsigned)grid), dim3(kTok), 0, hs, A)
  if (dtype == TDP_BF16) TDP_NORM_LANES(CALL, TDP_BF16);
  else TDP_NORM_LANES(CALL, TDP_F32);
#undef CALL
  if (dweight || dbias)
    hipLaunchKernelGGL(layer_norm_join_kernel, dim3((unsigned)join), dim3(kTok), 0, hs, A.parts, (int)A.nparts,
                       channels, dweight, dbias);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

}  // extern "C"

// Rotation by three position axes, and the per-head norms of queries and
// keys with that rotation in the same pass, with their gradients (gfx950).
//
// Source of the positions: LTX-2 docs, "Tiled Data Parallelism (TDP)",
// "Position normalization" (each tile hands the model its own zero-based
// [start, end) intervals on time, height and width).
//
// All kernels are bound by HBM bandwidth: a few operations per element read
// and written once.  A wave owns one row (token) at a time, all its heads: its
// lanes compute the row's angles once, one pair each, into LDS, and every head
// reuses them, so no table of cosines is stored or read (24 bytes of positions
// per row instead of 4 * head_dim).  A lane moves eight elements of a head in
// 16-byte pieces, G lanes share a head (G = the power of two at or above
// head_dim / 8) and 64 / G heads go through the wave at once; the norm's sums
// run over the G lanes by DPP moves.  A batch of U such passes is loaded ahead
// of the one being worked on, across rows too: a workgroup takes several
// consecutive blocks of four rows, so what does not depend on the row (weights,
// frequencies, partners) is set up once.
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

// One wave's row of angles, per dim that turns: the factor of the dim itself and
// of its partner, y[d] = x[d] c[d] + x[partner] s[d] (s carries the pair's sign).
struct Angles {
  float c[TDP_MAX_ROPE_DIM], s[TDP_MAX_ROPE_DIM];
};

__device__ inline void wave_lds_fence() {
  // LDS operations of one wave complete in order; only the compiler has to
  // keep the order, no other wave shares this memory.
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A lane's pairs of a row: p = lane and lane + 64 (head_dim > 128).
template <bool HALVES, int G>
struct LaneTurns {
  static constexpr int N = G > 16 ? 2 : 1;
  float hi[N], lo[N];
  int axis[N], d0[N], d1[N];
  bool on[N];
  __device__ inline LaneTurns(const RopeDev& r, int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int p = lane + 64 * n;
      on[n] = p < r.pairs;
      axis[n] = on[n] ? pair_axis(r, p) : 0;
      hi[n] = on[n] ? r.hi[p] : 0.0f;
      lo[n] = on[n] ? r.lo[p] : 0.0f;
      d0[n] = 2 * p;
      d1[n] = 2 * p + 1;
      if (HALVES && on[n]) {
        d0[n] = p + (axis[n] == 0 ? 0 : r.pair_end[axis[n] - 1]);
        d1[n] = d0[n] + r.half[axis[n]];
      }
    }
  }
  __device__ inline void load(const float* pos, const SeqRows& sr, int i, f32x2* iv) const {
    const f32x2* base = reinterpret_cast<const f32x2*>(pos) + 3 * sr.row0 + i;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (on[n]) iv[n] = base[(int64_t)axis[n] * sr.span];
  }
  __device__ inline void fill(const f32x2* iv, bool middle, float dir, Angles* a) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (!on[n]) continue;
      float c, s;
      turn(iv[n].x, iv[n].y, middle, hi[n], lo[n], &c, &s);
      s *= dir;
      a->c[d0[n]] = a->c[d1[n]] = c;
      a->s[d0[n]] = -s;
      a->s[d1[n]] = s;
    }
  }
};

// The dims of a lane: bf16, eight in a row; fp32, four in each half of the
// head, so that each 16-byte access of neighbouring lanes is contiguous.
template <int T>
__device__ inline int lane_dim(int D, int chunk, int e) {
  return T == TDP_BF16 ? chunk * 8 + e : chunk * 4 + (e & 3) + (e >> 2) * (D / 2);
}
// Inverse of it: the slot e * 64 + chunk of dim d in a wave's exchange buffer.
template <int T>
__device__ inline int dim_slot(int D, int d) {
  if (T == TDP_BF16) return (d & 7) * 64 + (d >> 3);
  const int up = d >= D / 2, q = d - up * (D / 2);
  return ((q & 3) + 4 * up) * 64 + (q >> 2);
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

// Where the partners of a lane's dims pass through a wave's exchange buffer
// (half-split pairs; the other pairs lie in one lane), and with PART, for heads of
// which only the first dims turn, how many turn from the lane's first dim on and
// from its fifth.  Dims that do not turn are kept by selection: factors of 1 and 0
// would make a NaN of an infinity, their own or a neighbour's.  Heads that turn
// whole have kernels of their own, without the selection: as one kernel, a branch
// or masks cost up to 6 or 30 % there (norm gradients of 8 + 4 fp32 heads of 64,
// conditioned: 519 us, with them 548 or 672).
template <int T, bool HALVES, bool PART>
struct Partners {
  int left[2];
  int src[HALVES ? 8 : 1];
  // an even count turns, so a dim and the next turn or pass together
  __device__ inline bool turns(int e) const { return !PART || (e & 2) < left[e >> 2]; }
  __device__ inline Partners(const RopeDev& r, int chunk, int group_lane0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) left[i] = 2 * r.pairs - lane_dim<T>(r.D, chunk, 4 * i);
    if constexpr (HALVES) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = lane_dim<T>(r.D, chunk, e);
        src[e] = e * 64 + group_lane0 + chunk;
        if (chunk * 8 < r.D && d < 2 * r.pairs) {
          const int ax = pair_axis(r, d / 2);
          const int j = d - (ax == 0 ? 0 : 2 * r.pair_end[ax - 1]);
          src[e] = dim_slot<T>(r.D, j < r.half[ax] ? d + r.half[ax] : d - r.half[ax]) + group_lane0;
        }
      }
    }
  }
};

// The factors of a lane's dims for one row; a pair inside the lane needs them
// once.
template <int T, bool HALVES>
struct LaneAngles {
  static constexpr int N = HALVES ? 8 : 4;
  float c[N], s[N];
  __device__ inline void read(int D, int chunk, bool on, const float* ac, const float* as) {
    const int d0 = on ? lane_dim<T>(D, chunk, 0) : 0, d1 = on ? lane_dim<T>(D, chunk, 4) : 0;
    float cc[8], ss[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cc[e] = ac[d0 + e];
      cc[4 + e] = ac[d1 + e];
      ss[e] = as[d0 + e];
      ss[4 + e] = as[d1 + e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      c[e] = cc[HALVES ? e : 2 * e];
      s[e] = ss[HALVES ? e : 2 * e + 1];
    }
  }
};

// Turn the first n of U vectors.  Half-split partners sit in other lanes: they
// pass through LDS, element e of lane l at e * 64 + l, so writes and reads touch
// consecutive banks; all vectors are written before the first is read.
template <int T, bool HALVES, bool PART, int U>
__device__ inline void rotate(const Partners<T, HALVES, PART>& pt, const LaneAngles<T, HALVES>& la, float* ex, int lane,
                              int n, float (*x)[8]) {
  if constexpr (!HALVES) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= n) break;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float a = x[u][e], b = x[u][e + 1];
        x[u][e] = pt.turns(e) ? fmaf(a, la.c[e / 2], -b * la.s[e / 2]) : a;
        x[u][e + 1] = pt.turns(e) ? fmaf(b, la.c[e / 2], a * la.s[e / 2]) : b;
      }
    }
  } else {
    wave_lds_fence();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= n) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) ex[u * 512 + e * 64 + lane] = x[u][e];
    }
    wave_lds_fence();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= n) break;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[u][e] = pt.turns(e) ? fmaf(x[u][e], la.c[e], ex[u * 512 + pt.src[e]] * la.s[e]) : x[u][e];
    }
  }
}

template <int CTRL>
__device__ inline float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Sum over aligned groups of G lanes: quads by permutes, then mirrors of 8 and
// 16 lanes, then the swap of neighbouring rows of 16.
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
  uint32_t per_wg;         // forward: row blocks per workgroup
  int32_t rows;            // forward: rows a wave takes side by side
  uint32_t q_wgs;          // backward: workgroups on queries, the others take keys
};

// The rows of one wave: block blk of the launch is rows 4 k .. 4 k + 3 of a
// sequence, one per wave of the workgroup.
struct RowAt {
  uint32_t blk;
  int s, i;
  SeqRows sr;
  __device__ inline void seek(const SeqsDev& q, uint32_t blocks, uint32_t b, int wave) {
    blk = b;
    s = b / blocks;
    i = (b - s * blocks) * kWaves + wave;
    sr = seq_rows(q, s);
  }
  __device__ inline void next(const SeqsDev& q, uint32_t blocks, int wave) {
    ++blk;
    i += kWaves;
    if (blk == (uint32_t)(s + 1) * blocks) {
      ++s;
      i = wave;
      sr = seq_rows(q, s);
    }
  }
  __device__ inline bool owned() const { return i < sr.cap; }
  __device__ inline bool live() const { return i < sr.len; }
};

// A tensor as a wave sees it: the lane's share of a head, and the row's base
// (the same for the whole wave).
template <int T, int G>
struct Lanes {
  static constexpr int eb = T == TDP_BF16 ? 2 : 4, kPer = 64 / G;
  char* lane0;
  int64_t row_step, head_step, seq_step;
  int heads;
  __device__ inline Lanes(const HeadsDev& t, int chunk, int grp)
      : lane0(t.data + eb * (grp * t.head_stride + chunk * (T == TDP_BF16 ? 8 : 4))),
        row_step(t.row_stride * eb), head_step(t.head_stride * eb), seq_step(t.seq_stride * eb), heads(t.heads) {}
  __device__ inline char* at(const SeqsDev& q, const RowAt& r, int head) const {
    const int64_t base = q.range ? (r.sr.row0 + r.i) * row_step : r.s * seq_step + r.i * row_step;
    return lane0 + (base + head * head_step);
  }
  __device__ inline void zero(const SeqsDev& q, const RowAt& r, int half, int grp, bool on) const {
    const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int h = 0; h < heads; h += kPer)
      if (on && h + grp < heads) Raw<T>::store(at(q, r, h), half, z);
  }
};

template <int T, int G, bool HALVES, bool PART, bool NORM, int U>
__global__ __launch_bounds__(kTok, U == 2 ? 4 : 3) void rope_kernel(const RopeArgs A) {
  constexpr int kPer = 64 / G;
  __shared__ Angles ang[kWaves];
  __shared__ float exch[HALVES ? kWaves : 1][HALVES ? U * 512 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int chunk = lane % G, grp = lane / G, half = A.rope.D * 2;
  const bool on = chunk * 8 < A.rope.D;
  const uint32_t nblk = A.blocks * (uint32_t)A.seqs.S;
  const uint32_t b0 = blockIdx.x * A.per_wg, b1 = b0 + A.per_wg < nblk ? b0 + A.per_wg : nblk;
  const Lanes<T, G> iq(A.in[0], chunk, grp), ik(A.in[1], chunk, grp), oq(A.out[0], chunk, grp), ok(A.out[1], chunk, grp);
  const int nq = (iq.heads + kPer * U - 1) / (kPer * U), nk = (ik.heads + kPer * U - 1) / (kPer * U);
  const LaneTurns<HALVES, G> turns(A.rope, lane);
  const Partners<T, HALVES, PART> pt(A.rope, chunk, lane - chunk);
  const float inv_d = 1.0f / (float)A.rope.D;
  float wq[8], wk[8];
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = lane_dim<T>(A.rope.D, chunk, e);
      wq[e] = A.w[0] && on ? A.w[0][d] : 1.0f;
      wk[e] = A.w[1] && on ? A.w[1][d] : 1.0f;
    }
  }
  RowAt nx;
  Raw<T> raw[U];
  f32x2 iv[LaneTurns<HALVES, G>::N];
  auto fetch = [&](const RowAt& r, int b) {
    const bool k = b >= nq;  // the same for the whole wave
    const int h0 = (k ? b - nq : b) * kPer * U, heads = k ? ik.heads : iq.heads;
    const char* p = k ? ik.at(A.seqs, r, h0) : iq.at(A.seqs, r, h0);
    const int64_t step = (k ? ik.head_step : iq.head_step) * kPer;
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(p + u * step, half, on && h0 + u * kPer + grp < heads);
  };
  auto begin_row = [&]() {
    if (nx.live()) {
      fetch(nx, 0);
      turns.load(A.pos, nx.sr, nx.i, iv);
    }
  };
  nx.seek(A.seqs, A.blocks, b0, wave);
  begin_row();
  for (uint32_t blk = b0; blk < b1; ++blk) {
    const RowAt at = nx;
    if (!at.live()) {
      if (at.owned()) {
        oq.zero(A.seqs, at, half, grp, on);
        ok.zero(A.seqs, at, half, grp, on);
      }
      if (blk + 1 < b1) {
        nx.next(A.seqs, A.blocks, wave);
        begin_row();
      }
      continue;
    }
    wave_lds_fence();
    turns.fill(iv, A.rope.point == TDP_POINT_MIDDLE, A.dir, &ang[wave]);
    wave_lds_fence();
    LaneAngles<T, HALVES> la;
    la.read(A.rope.D, chunk, on, ang[wave].c, ang[wave].s);
    for (int b = 0; b < nq + nk; ++b) {
      const bool k = b >= nq;
      const int heads = k ? ik.heads : iq.heads;
      const int hb = (k ? b - nq : b) * kPer * U;
      const int n = (heads - hb + kPer - 1) / kPer;  // passes with a head left, the same for the whole wave
      float x[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u].unpack(x[u]);
      if (b + 1 < nq + nk) {
        fetch(at, b + 1);
      } else if (blk + 1 < b1) {
        nx.next(A.seqs, A.blocks, wave);
        begin_row();
      }
      if constexpr (NORM) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = k ? wk[e] : wq[e];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u >= n) break;
          float ss = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[u][e], x[u][e], ss);
          const float r = __builtin_amdgcn_rsqf(fmaf(group_sum<G>(ss), inv_d, A.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][e] *= r * w[e];
        }
      }
      rotate<T, HALVES, PART, U>(pt, la, exch[HALVES ? wave : 0], lane, n, x);
      char* p = k ? ok.at(A.seqs, at, hb) : oq.at(A.seqs, at, hb);
      const int64_t step = (k ? ok.head_step : oq.head_step) * kPer;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on && hb + u * kPer + grp < heads) Raw<T>::store(p + u * step, half, x[u]);
    }
  }
}

// The same for few heads: a row of fewer heads than the wave's lanes hold leaves
// most lanes idle, so the wave takes P rows of a sequence side by side, one pass
// for queries and one for keys (hslots heads per row, P * hslots = 64 / G).
template <int T, int G, bool HALVES, bool PART, bool NORM>
__global__ __launch_bounds__(kTok, 4) void rope_few_kernel(const RopeArgs A) {
  constexpr int kPer = 64 / G, kDims = kPer * 8 * G, N = kDims / 2 / 64;  // dims and pairs of P rows at most
  __shared__ float angc[kWaves][kDims], angs[kWaves][kDims];
  __shared__ float exch[HALVES ? kWaves : 1][HALVES ? 512 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int chunk = lane % G, grp = lane / G, D = A.rope.D, half = D * 2;
  const int P = A.rows, hslots = kPer / P, sub = grp / hslots, head = grp - sub * hslots;
  const uint32_t nblk = A.blocks * (uint32_t)A.seqs.S;
  const uint32_t b0 = blockIdx.x * A.per_wg, b1 = b0 + A.per_wg < nblk ? b0 + A.per_wg : nblk;
  const bool on = chunk * 8 < D;
  const Lanes<T, G> in[2] = {Lanes<T, G>(A.in[0], chunk, head), Lanes<T, G>(A.in[1], chunk, head)};
  const Lanes<T, G> out[2] = {Lanes<T, G>(A.out[0], chunk, head), Lanes<T, G>(A.out[1], chunk, head)};
  const Partners<T, HALVES, PART> pt(A.rope, chunk, lane - chunk);
  const float inv_d = 1.0f / (float)D;
  // this lane's pairs: slot lane + 64 n is pair p of row r
  const int pairs = D / 2;
  for (uint32_t blk = b0; blk < b1; ++blk) {
    RowAt at;
    at.s = blk / A.blocks;
    at.i = (int)(blk - at.s * A.blocks) * kWaves * P + wave * P;
    at.sr = seq_rows(A.seqs, at.s);
    if (!at.owned()) continue;
    const bool owned = at.i + sub < at.sr.cap, live = at.i + sub < at.sr.len;
    Raw<T> raw[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      raw[t].load(in[t].at(A.seqs, at, 0) + sub * in[t].row_step, half, on && live && head < in[t].heads);
    wave_lds_fence();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int slot = lane + 64 * n, r = slot / pairs, q = slot - r * pairs;
      if (r >= P) break;
      if (PART && q >= A.rope.pairs) continue;
      const int ax = pair_axis(A.rope, q);
      int d0 = 2 * q, d1 = d0 + 1;
      if (HALVES) {
        d0 = q + (ax == 0 ? 0 : A.rope.pair_end[ax - 1]);
        d1 = d0 + A.rope.half[ax];
      }
      float c = 1.0f, si = 0.0f;
      if (at.i + r < at.sr.len) {
        const f32x2 iv = (reinterpret_cast<const f32x2*>(A.pos) + 3 * at.sr.row0 + at.i + r)[(int64_t)ax * at.sr.span];
        turn(iv.x, iv.y, A.rope.point == TDP_POINT_MIDDLE, A.rope.hi[q], A.rope.lo[q], &c, &si);
        si *= A.dir;
      }
      angc[wave][r * D + d0] = angc[wave][r * D + d1] = c;
      angs[wave][r * D + d0] = -si;
      angs[wave][r * D + d1] = si;
    }
    wave_lds_fence();
    LaneAngles<T, HALVES> la;
    la.read(D, chunk, on, angc[wave] + sub * D, angs[wave] + sub * D);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t && A.in[1].heads == 0) break;
      float x[1][8];
      raw[t].unpack(x[0]);
      if constexpr (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[0][e], x[0][e], ss);
        const float r = __builtin_amdgcn_rsqf(fmaf(group_sum<G>(ss), inv_d, A.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[0][e] *= r * (A.w[t] && on ? A.w[t][lane_dim<T>(D, chunk, e)] : 1.0f);
      }
      rotate<T, HALVES, PART, 1>(pt, la, exch[HALVES ? wave : 0], lane, 1, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[0][e] = live ? x[0][e] : 0.0f;
      if (on && owned && head < out[t].heads) Raw<T>::store(out[t].at(A.seqs, at, 0) + sub * out[t].row_step, half, x[0]);
    }
  }
}

// Gradient of the norm and rotation: dx per row, and each workgroup's sums of
// the weight's gradient over its rows, fp32 in a fixed order.  A workgroup takes
// queries or keys (the first q_wgs take queries), which keeps one tensor's sums
// and weights in registers.  With three waves per SIMD, bf16 holds everything in
// registers (16 + 16 heads of 128, 882 MB: 183 us); fp32 spills 6 to 14 of them
// with interleaved pairs and 27 to 34 with half-split ones (16 + 16 heads of 128,
// 1.76 GB: 347 and 357 us; 8 + 4 heads of 64, half-split, 1.18 GB: 517 us).
template <int T, int G, bool HALVES, bool PART>
__global__ __launch_bounds__(kTok, 3) void norm_backward_kernel(const RopeArgs A) {
  constexpr int kPer = 64 / G, U = 2;
  __shared__ Angles ang[kWaves];
  __shared__ float exch[HALVES ? kWaves : 1][HALVES ? U * 512 : 1];
  __shared__ float red[kWaves][TDP_MAX_ROPE_DIM];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int chunk = lane % G, grp = lane / G, half = A.rope.D * 2;
  const bool on = chunk * 8 < A.rope.D;
  const bool keys = blockIdx.x >= A.q_wgs;
  const Lanes<T, G> in(keys ? A.in[1] : A.in[0], chunk, grp), gr(keys ? A.grad[1] : A.grad[0], chunk, grp),
      out(keys ? A.out[1] : A.out[0], chunk, grp);
  const float* wp = keys ? A.w[1] : A.w[0];
  const uint32_t nblk = A.blocks * (uint32_t)A.seqs.S;
  const uint32_t wg = keys ? blockIdx.x - A.q_wgs : blockIdx.x, wgs = keys ? gridDim.x - A.q_wgs : A.q_wgs;
  const uint32_t b0 = (uint32_t)((uint64_t)nblk * wg / wgs), b1 = (uint32_t)((uint64_t)nblk * (wg + 1) / wgs);
  const int nb = (in.heads + kPer * U - 1) / (kPer * U);
  const LaneTurns<HALVES, G> turns(A.rope, lane);
  const Partners<T, HALVES, PART> pt(A.rope, chunk, lane - chunk);
  const float inv_d = 1.0f / (float)A.rope.D;
  float w[8], dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = wp && on ? wp[lane_dim<T>(A.rope.D, chunk, e)] : 1.0f;
    dw[e] = 0.0f;
  }
  RowAt nx;
  Raw<T> rx[U], rg[U];
  f32x2 iv[LaneTurns<HALVES, G>::N];
  auto fetch = [&](const RowAt& r, int b) {
    const int h0 = b * kPer * U;
    const char *ip = in.at(A.seqs, r, h0), *gp = gr.at(A.seqs, r, h0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ld = on && h0 + u * kPer + grp < in.heads;
      rx[u].load(ip + u * kPer * in.head_step, half, ld);
      rg[u].load(gp + u * kPer * gr.head_step, half, ld);
    }
  };
  auto begin_row = [&]() {
    if (nx.live()) {
      fetch(nx, 0);
      turns.load(A.pos, nx.sr, nx.i, iv);
    }
  };
  if (b0 < b1) {
    nx.seek(A.seqs, A.blocks, b0, wave);
    begin_row();
  }
  for (uint32_t blk = b0; blk < b1; ++blk) {
    const RowAt at = nx;
    if (!at.live()) {
      if (at.owned()) out.zero(A.seqs, at, half, grp, on);
      if (blk + 1 < b1) {
        nx.next(A.seqs, A.blocks, wave);
        begin_row();
      }
      continue;
    }
    wave_lds_fence();
    turns.fill(iv, A.rope.point == TDP_POINT_MIDDLE, -1.0f, &ang[wave]);
    wave_lds_fence();
    LaneAngles<T, HALVES> la;
    la.read(A.rope.D, chunk, on, ang[wave].c, ang[wave].s);
    for (int b = 0; b < nb; ++b) {
      const int hb = b * kPer * U;
      const int n = (in.heads - hb + kPer - 1) / kPer;
      float x[U][8], g[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        rx[u].unpack(x[u]);
        rg[u].unpack(g[u]);
      }
      if (b + 1 < nb) {
        fetch(at, b + 1);
      } else if (blk + 1 < b1) {
        nx.next(A.seqs, A.blocks, wave);
        begin_row();
      }
      rotate<T, HALVES, PART, U>(pt, la, exch[HALVES ? wave : 0], lane, n, g);
      char* op = out.at(A.seqs, at, hb);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= n) break;
        float ss = 0.0f, gx = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[u][e], x[u][e], ss);
          gx = fmaf(g[u][e] * w[e], x[u][e], gx);
        }
        // lanes without a head hold zeros, whose r is infinite when eps is 0: they stay out of dw
        const bool has = hb + u * kPer + grp < in.heads;
        const float r = has ? __builtin_amdgcn_rsqf(fmaf(group_sum<G>(ss), inv_d, A.eps)) : 0.0f;
        const float m = group_sum<G>(gx) * inv_d * r * r;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[e] = fmaf(g[u][e], x[u][e] * r, dw[e]);
          y[e] = r * fmaf(g[u][e], w[e], -x[u][e] * m);
        }
        if (on && has) Raw<T>::store(op + u * kPer * out.head_step, half, y);
      }
    }
  }
  // the wave's groups, then its four waves
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = G; o < 64; o <<= 1) dw[e] += __shfl_xor(dw[e], o);
    if (grp == 0 && on) red[wave][lane_dim<T>(A.rope.D, chunk, e)] = dw[e];
  }
  __syncthreads();
  for (int d = threadIdx.x; d < A.rope.D; d += kTok)
    A.parts[(int64_t)blockIdx.x * A.rope.D + d] = (red[0][d] + red[1][d]) + (red[2][d] + red[3][d]);
}

// Sum the workgroups' partial rows: 16 columns per workgroup, 16 strided row
// sums per column joined in order; the first workgroups take queries.
__global__ __launch_bounds__(kTok) void norm_weights_kernel(const float* parts, int nq, int n, int D, float* dwq,
                                                            float* dwk) {
  __shared__ float red[16][17];
  const int per = (D + 15) / 16;
  const bool keys = (int)blockIdx.x >= per;
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int c = (keys ? blockIdx.x - per : blockIdx.x) * 16 + col;
  float* out = keys ? dwk : dwq;
  float v = 0.0f;
  if (c < D)
    for (int r = (keys ? nq : 0) + row; r < (keys ? n : nq); r += 16) v += parts[(int64_t)r * D + c];
  red[row][col] = v;
  __syncthreads();
  if (row == 0 && c < D && out) {
    float sum = 0.0f;
    for (int r = 0; r < 16; ++r) sum += red[r][col];
    out[c] = sum;
  }
}

// Four passes of the wave ahead where a tensor's heads fill them, two where
// they would not: on 16 bf16 heads of 128 dims (4 passes) four took 329 us for
// 2.0 GB against 354, on 8 and 4 fp32 heads of 64 dims (one pass each) two took
// 182 us for 0.8 GB against 208, registers and exchange buffers being smaller.
template <int T, int G, bool NORM, bool HALVES, bool PART>
void launch_forward(const RopeArgs& a, uint32_t grid, hipStream_t st) {
  if (a.rows > 1)
    hipLaunchKernelGGL((rope_few_kernel<T, G, HALVES, PART, NORM>), dim3(grid), dim3(kTok), 0, st, a);
  else if (a.in[0].heads >= 4 * (64 / G))
    hipLaunchKernelGGL((rope_kernel<T, G, HALVES, PART, NORM, 4>), dim3(grid), dim3(kTok), 0, st, a);
  else
    hipLaunchKernelGGL((rope_kernel<T, G, HALVES, PART, NORM, 2>), dim3(grid), dim3(kTok), 0, st, a);
}
template <int T, int G, bool HALVES, bool PART>
void launch_backward(const RopeArgs& a, uint32_t grid, hipStream_t st) {
  hipLaunchKernelGGL((norm_backward_kernel<T, G, HALVES, PART>), dim3(grid), dim3(kTok), 0, st, a);
}

enum class Mode { kRope, kNorm, kBackward };

template <int T, int G, bool HALVES, bool PART>
void launch_mode(Mode m, const RopeArgs& a, uint32_t grid, hipStream_t st) {
  if (m == Mode::kRope) launch_forward<T, G, false, HALVES, PART>(a, grid, st);
  if (m == Mode::kNorm) launch_forward<T, G, true, HALVES, PART>(a, grid, st);
  if (m == Mode::kBackward) launch_backward<T, G, HALVES, PART>(a, grid, st);
}
template <int T, int G>
void launch_mode(Mode m, const RopeArgs& a, uint32_t grid, hipStream_t st) {
  const bool halves = a.rope.pairing == TDP_PAIR_HALVES, part = 2 * a.rope.pairs < a.rope.D;
  if (halves && part) launch_mode<T, G, true, true>(m, a, grid, st);
  else if (halves) launch_mode<T, G, true, false>(m, a, grid, st);
  else if (part) launch_mode<T, G, false, true>(m, a, grid, st);
  else launch_mode<T, G, false, false>(m, a, grid, st);
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

// Rows side by side, and row blocks per workgroup of a forward launch: rows of
// fewer than 4 passes of 64 lanes are taken 32 passes at a time, so that the
// wave's setup is shared, as long as 4096 workgroups (16 per CU) remain (8 and 4
// fp32 heads of 64: 180 us for 0.8 GB against 251 with 4 passes); longer rows are
// taken one by one (16 bf16 heads of 128: 318 us for 2.0 GB against 354 with 16).
uint32_t forward_grid(const tdp_seqs& s, RopeArgs* a) {
  int lanes = 1;  // of a head
  while (lanes * 8 < a->rope.D) lanes *= 2;
  int slots = 1;  // heads of a row
  while (slots < a->in[0].heads || slots < a->in[1].heads) slots *= 2;
  a->rows = slots * lanes * 2 <= 64 ? 64 / (slots * lanes) : 1;
  a->blocks = (uint32_t)((s.max_rows + kWaves * a->rows - 1) / (kWaves * a->rows));
  const int64_t nblk = (int64_t)a->blocks * s.num_seqs;
  const int64_t work = (int64_t)(a->in[0].heads + a->in[1].heads) * ((a->rope.D + 7) / 8) * a->rows;
  int64_t per = work < 4 * 64 ? 32 * 64 / work : 1;
  if (per > nblk / 4096) per = nblk / 4096;
  a->per_wg = (uint32_t)(per < 1 ? 1 : per);
  return (uint32_t)((nblk + a->per_wg - 1) / a->per_wg);
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
  const uint32_t grid = forward_grid(*seqs, &a);
  return run(fn, Mode::kRope, a, dtype, grid, stream);
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
  const uint32_t grid = forward_grid(*seqs, &a);
  return run(fn, Mode::kNorm, a, dtype, grid, stream);
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
  const NormParts n = norm_parts(*seqs, q->heads, k->heads);
  a.q_wgs = (uint32_t)n.q;
  st = run(fn, Mode::kBackward, a, dtype, (uint32_t)(n.q + n.k), stream);
  if (st != TDP_OK || (!dq_weight && !dk_weight)) return st;
  hipLaunchKernelGGL(norm_weights_kernel, dim3(2 * ((D + 15) / 16)), dim3(kTok), 0,
                     reinterpret_cast<hipStream_t>(stream), a.parts, n.q, n.q + n.k, D, dq_weight, dk_weight);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

}  // extern "C"

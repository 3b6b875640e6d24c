// Attention of a tile's rows and its gradients (gfx950 matrix instructions).
//
//   s_ij = scale * q_i . k_j + bias_j,  p_ij = exp(s_ij - lse_i),
//   o_i = sum_j p_ij v_j
//   delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// The scores are never stored: the forward keeps a running maximum and sum
// per query while it walks the keys, the backward computes them again from
// lse.  All products run as 32 x 32 tiles of the matrix instructions with
// fp32 accumulators.
//
// Layouts.  A product C = A B of 32 x 32 with a contraction of 16 takes from
// lane l (h = l / 32) the elements A[l % 32][8h .. 8h+7] and B[8h .. 8h+7][l % 32]
// and leaves C[8 (r / 4) + 4h + r % 4][l % 32] in its register r.  The score
// tile is computed so that the axis the next product keeps lies on the
// columns (keys x queries for o and dq, queries x keys for dk and dv): each
// lane then holds one column, the softmax needs one exchange between the two
// halves of the wave, and registers 8s .. 8s+7 are, as they stand, the B
// operand of the next product's step s with its contraction in the order
//   16s + {4h, .., 4h+3, 8+4h, .., 8+4h+3}.
// The A operand of that product is read in the same order, down the columns
// of the LDS tile (bf16: the transposing 64-bit LDS read, four rows of 16
// columns per 16 lanes).
//
// fp32 tensors run the same code on fp32 matrix instructions, eight
// contractions of 2 for one of 16.
//
// Roundings.  Scores, maxima, sums, delta and every accumulator are fp32 for both
// types.  For bf16 the weights p and the ds enter their second products as bf16
// (at most half a step, 2^-8 of each, ties to even), because the bf16 matrix
// instructions take nothing wider; the sum l is of the weights before that.  The
// outputs then lie 0.0023 (rms, relative) from 64 bits, where rounding the output
// alone gives 0.0017: two independent roundings of that size.  Weights in two bf16
// parts would double those products.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "token_device.h"

namespace tdp {
namespace {

constexpr int kTok = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A bias at or below this (-infinity, the lowest values of fp32 and bf16) takes
// the key out.
constexpr float kBiasOut = -1.0e30f;
// The running maximum is moved only when a block exceeds it by this many
// powers of two: weights stay below 2^8, where fp32 sums and bf16 weights lose
// nothing, and most blocks skip the rescaling of the sums.
constexpr float kSlack = 8.0f;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define TDP_LDS __attribute__((address_space(3)))

template <int T>
struct Mat;
template <>
struct Mat<TDP_BF16> {
  typedef bf16x8 Frag;
  static constexpr int kBytes = 2;
  __device__ static inline f32x16 mma(const Frag& a, const Frag& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static inline Frag pack(const float* x) {
    return __builtin_convertvector(f32x8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}, bf16x8);
  }
};
template <>
struct Mat<TDP_F32> {
  typedef f32x8 Frag;
  static constexpr int kBytes = 4;
  __device__ static inline f32x16 mma(const Frag& a, const Frag& b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  __device__ static inline Frag pack(const float* x) { return f32x8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}; }
};

// A tile of rows in LDS: DP elements per row in 16-byte chunks, chunk c of row
// r at c ^ swizzle(r).  LDS has 64 banks: one pass serves 32 lanes of a
// transposing read (four rows at an aligned group of four chunks) or 16 lanes of
// a 16-byte read (16 rows at the same chunk).  The swizzle's upper bits differ
// between four neighbouring rows, so the first meet no bank twice; it repeats
// after eight rows, so the second take two passes.  A swizzle over 16 rows
// removes that too (no conflict counted), but then rows r and r + 8 need an
// address each, whose registers spill: dq took 432 us instead of 283 on
// 4 x 2240 rows, 16 heads of 128.
template <int T, int DP>
struct Tile {
  typedef typename Mat<T>::Frag Frag;
  static constexpr int kRow = DP * Mat<T>::kBytes;  // bytes
  static constexpr int kChunks = kRow / 16;
  __device__ static inline int at(int r, int c) {
    return r * kRow + (chunk_at(r, c) << 4);
  }
  // the chunk held by slot c of row r
  __device__ static inline int chunk_at(int r, int c) {
    if (kChunks == 4) return c ^ (r >> 2 & 1);
    if (kChunks == 8) return c ^ ((r >> 1 & 1) << 2 | (r >> 2 & 1));
    return c ^ ((r & 3) << 2 | (r >> 2 & 1));
  }
  // A[r][16 kk + 8h .. +7]
  __device__ static inline Frag row_frag(const char* lds, int r, int kk, int h) {
    if constexpr (T == TDP_BF16) {
      return *reinterpret_cast<const bf16x8*>(lds + at(r, 2 * kk + h));
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(lds + at(r, 4 * kk + 2 * h));
      const f32x4 b = *reinterpret_cast<const f32x4*>(lds + at(r, 4 * kk + 2 * h + 1));
      return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
  // rows r0 + {4h .. 4h+3, 8+4h .. 8+4h+3} of column c0 + l % 32
  __device__ static inline Frag col_frag(char* lds, int r0, int c0, int lane) {
    const int h = lane >> 5;
    if constexpr (T == TDP_BF16) {
      const int r = r0 + 4 * h + ((lane & 15) >> 2);
      const int c = c0 + (lane & 16) + 4 * (lane & 3);
      const int off = (c & 7) * 2;
      typedef TDP_LDS bf16x4* P;
      const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((P)(TDP_LDS char*)(lds + at(r, c >> 3) + off));
      const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((P)(TDP_LDS char*)(lds + at(r + 8, c >> 3) + off));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      const int c = c0 + (lane & 31);
      f32x8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = r0 + 4 * h + (e & 3) + 8 * (e >> 2);
        v[e] = *reinterpret_cast<const float*>(lds + at(r, c >> 2) + (c & 3) * 4);
      }
      return v;
    }
  }
};

struct AttnArgs {
  SeqsDev qs, ks;
  HeadsDev q, k, v, o, dout, dq, dk, dv;
  const float* bias;
  float* lse;
  f32x2* stats;  // backward, per query head and row: -lse log2(e) and delta
  float* ws;
  float scale;
  int32_t D, group, splits, m_max;  // m_max: query entries of the longest sequence
  FastDiv by_group;
  uint32_t blocks, tiles;  // row blocks per (sequence, key head); all work items
};

// Workgroups are dealt round-robin to the eight XCDs; each gets a contiguous
// range of the work items, which are ordered so that neighbours walk the same
// keys, and these then stay in that XCD's L2.  Where slots are used unequally the
// ranges are unequal work: the fullest XCD of the conditioned plan's gradients (36
// sequences, a quarter to all of 1024 conditioning rows kept) holds 1.08 to 1.21
// times the mean, counted over four sets of inputs.
__device__ inline uint32_t xcd_item(uint32_t tiles) {
  const uint32_t per = (tiles + 7) / 8;
  return (blockIdx.x & 7) * per + (blockIdx.x >> 3);
}
inline uint32_t xcd_grid(uint32_t tiles) { return (tiles + 7) / 8 * 8; }

__device__ inline float other_half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float other_half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Rows [r0, r0 + ROWS) of a head straight into a tile in LDS: a wave's 64 lanes
// fill 64 neighbouring 16-byte slots, each lane fetching the chunk that the
// swizzle puts there.  Rows at and past `len` and chunks past head_dim lie
// outside the buffer descriptor's range, which makes them zero.
// With EXACT a row past the end is zero whatever the strides; without, rows of
// stride 0 repeat the last one there, which the scores' mask takes out.
template <int T, int DP, int ROWS, bool EXACT = false>
struct Direct {
  typedef Tile<T, DP> L;
  static constexpr int kSlots = ROWS * L::kChunks, N = (kSlots + kTok - 1) / kTok;
  uint32_t off[N];
  __device__ static inline int row_of(int n) { return threadIdx.x / L::kChunks + n * (kTok / L::kChunks); }
  __device__ inline void init(uint32_t row_bytes, int d_bytes) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * kTok, r = i / L::kChunks, c = L::chunk_at(r, i % L::kChunks);
      off[n] = c * 16 < d_bytes ? r * row_bytes + c * 16 : 0xfffffff0u;
    }
  }
  __device__ inline void load(const char* head, int64_t row_bytes, int d_bytes, int r0, int len, int wave,
                              char* lds) const {
#ifdef __HIP_DEVICE_COMPILE__  // the descriptor type exists on the device only
    const int left = len - r0 < ROWS ? len - r0 : ROWS;
    const uint32_t span = left > 0 ? (uint32_t)(left - 1) * (uint32_t)row_bytes + d_bytes : 0;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(head + r0 * row_bytes), 0, __builtin_amdgcn_readfirstlane(span), 0x00020000);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (kSlots % kTok == 0 || n * kTok + wave * 64 < kSlots)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (TDP_LDS void*)(lds + (n * kTok + wave * 64) * 16), 16,
                                                 EXACT && row_of(n) >= left ? 0xfffffff0u : off[n], 0, 0, 0);
#endif
  }
  // Clear what this lane has loaded of a block's keys that take no part: their
  // rows may hold anything, and a weight of zero would not remove a NaN.
  __device__ inline void clear(const float* bl, char* lds) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * kTok;
      if (i < kSlots && bl[i / L::kChunks] == -INFINITY) *reinterpret_cast<u32x4*>(lds + i * 16) = u32x4{0, 0, 0, 0};
    }
  }
};
// The biases of blocks of ROWS keys in powers of two, -infinity where a key takes
// no part or lies past the end: four blocks in LDS, a fifth on its way in a
// register, so that no step waits for the load that it issues.
template <int ROWS>
struct Biases {
  const float* bias;
  float* lds;
  int len;
  float next;
  __device__ inline float get(int b) const {
    const int j = b * ROWS + (int)threadIdx.x;
    return threadIdx.x < ROWS && j < len ? bias[j] : -INFINITY;
  }
  __device__ inline void put(int b, float x) const {
    if (threadIdx.x < ROWS) lds[(b & 3) * ROWS + threadIdx.x] = x <= kBiasOut ? -INFINITY : x * kLog2e;
  }
  __device__ inline const float* at(int b) const { return lds + (b & 3) * ROWS; }
  // before the first block: it and the one after it
  __device__ inline void start(int b) {
    put(b, get(b));
    put(b + 1, get(b + 1));
    next = get(b + 2);
  }
  // in block b's step: what comes two blocks later is stored, three blocks later requested
  __device__ inline void advance(int b) {
    put(b + 2, next);
    next = get(b + 3);
  }
};
__device__ inline void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// The B operand of a product over head_dim, from global memory: element
// 16 kk + 8h + e of the lane's row (null: zero).
template <int T, int DP>
__device__ inline void load_frags(const char* row, int h, int D, typename Mat<T>::Frag* f) {
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    const int d = 16 * kk + 8 * h;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (T == TDP_BF16) {
      u32x4 v = {0, 0, 0, 0};
      if (row && d < D) v = *reinterpret_cast<const u32x4*>(row + 2 * d);
      f[kk] = __builtin_bit_cast(bf16x8, v);
    } else {
      if (row && d < D) load8<TDP_F32>(row, d, x);
      f[kk] = Mat<T>::pack(x);
    }
  }
}

// One lane's column of an accumulator (rows = head_dim) times `f`, as the output dtype.
template <int T, int ND>
__device__ inline void store_column(char* row, int h, int D, const f32x16* acc, float f) {
#pragma unroll
  for (int nd = 0; nd < ND; ++nd)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int d = nd * 32 + r4 * 8 + h * 4;
      if (d >= D) continue;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = acc[nd][r4 * 4 + e] * f;
      if constexpr (T == TDP_BF16) {
        uint2 v;
        v.x = pack_bf16x2(x[0], x[1]);
        v.y = pack_bf16x2(x[2], x[3]);
        *reinterpret_cast<uint2*>(row + 2 * d) = v;
      } else {
        *reinterpret_cast<f32x4*>(row + 4 * d) = f32x4{x[0], x[1], x[2], x[3]};
      }
    }
}

__device__ inline f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}

// A work item's place: sequence, key head, block of query entries or keys, split.
struct Place {
  int s, hk, blk, split;
};
__device__ inline Place place(const AttnArgs& A, uint32_t item) {
  Place p;
  const uint32_t sh = item / (A.blocks * A.splits), rest = item - sh * (A.blocks * A.splits);
  p.split = rest / A.blocks;
  p.blk = rest - p.split * A.blocks;
  p.s = sh / A.k.heads;
  p.hk = sh - p.s * A.k.heads;
  return p;
}

// A block's scores as the softmax takes them: with a bias in powers of two
// (scaled and biased, the bias -infinity where a key takes no part), otherwise
// raw, and -infinity for keys past the end.
template <bool BIAS>
__device__ inline void mask_scores(f32x16& st, const float* bl, float c, int j0, int len, int h) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int j = 8 * (r >> 2) + 4 * h + (r & 3);
    if constexpr (BIAS)
      st[r] = fmaf(st[r], c, bl[j]);
    else if (j0 + j >= len)
      st[r] = -INFINITY;
  }
}

// Forward: 128 query entries of one key head per workgroup, 32 per wave.  K and
// V blocks of 64 keys come through two LDS buffers each, loaded one step ahead.
// A step multiplies block b's scores while the softmax and the product with V
// of block b - 1 run, so that matrix and vector instructions of one wave have
// each other to overlap with; two workgroups share a CU (three at head_dim 64).
// On 4 x 15456 rows, 12 heads of 128: 5.11 ms, 1.15 PFLOP/s, 0.89 of a large
// library product's rate; the matrix pipes are busy 68% of the time, at a clock
// that the card lowers to about 1.7 GHz under this load.  Twice the query entries
// per wave need all 512 registers and spill: 13.0 ms.
template <int T, int DP, bool BIAS>
__global__ __launch_bounds__(kTok, T != TDP_BF16 ? 1 : DP == 64 ? 3 : 2) void attn_forward_kernel(const AttnArgs A) {
  typedef Tile<T, DP> L;
  typedef typename Mat<T>::Frag Frag;
  constexpr int KD = DP / 16, ND = DP / 32, KT = kAttnBlockK / 32, kTile = kAttnBlockK * L::kRow;
  // separate arrays, so that reads of one are not held back by loads into another
  __shared__ __align__(16) char k0[kTile];
  __shared__ __align__(16) char k1[kTile];
  __shared__ __align__(16) char v0[kTile];
  __shared__ __align__(16) char v1[kTile];
  __shared__ __align__(16) float bl[BIAS ? 4 * kAttnBlockK : 4];
  const uint32_t item = xcd_item(A.tiles);
  if (item >= A.tiles) return;
  const Place pl = place(A, item);
  const SeqRows qr = seq_rows(A.qs, pl.s), kr = seq_rows(A.ks, pl.s);
  const int M = qr.cap * A.group, mlen = qr.len * A.group;
  const int m0 = pl.blk * kAttnBlockQ;
  if (m0 >= M) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int m = m0 + wave * 32 + (lane & 31);
  const int row = (int)fastdiv((uint32_t)m, A.by_group), head = pl.hk * A.group + (m - row * A.group);
  constexpr int eb = Mat<T>::kBytes;

  Frag qf[KD];
  load_frags<T, DP>(m < mlen ? A.q.data + eb * (seq_base(A.qs, A.q, pl.s, qr) + row * A.q.row_stride +
                                               head * A.q.head_stride)
                             : nullptr,
                    h, A.D, qf);
  f32x16 o[ND], st[KT];
#pragma unroll
  for (int nd = 0; nd < ND; ++nd) o[nd] = zero16();
  float mx = -INFINITY, l = 0.0f;  // mx in the scores' unit
  // Without a bias a weight's exponent is s c - mc in one fma.  The rounding of
  // mc = mx c scales all weights of a row alike, which is harmless until it passes
  // fp32's range (scores past 10^9 would give infinite weights, or none at all);
  // such rows' scores are lowered by mx first, and mc is 0.  fp32 tensors, whose
  // matrix instructions leave time for it, always take (s - mx) c (the branch
  // costs them 3 % at head_dim 64, this 1).
  constexpr bool kFused = !BIAS && T == TDP_BF16;
  float mc = 0.0f;
  bool far = false;  // a row of the wave needs that
  const float c = A.scale * kLog2e, unit = BIAS ? 1.0f : c;

  const char* kb = A.k.data + eb * (seq_base(A.ks, A.k, pl.s, kr) + pl.hk * A.k.head_stride);
  const char* vb = A.v.data + eb * (seq_base(A.ks, A.v, pl.s, kr) + pl.hk * A.v.head_stride);
  const int64_t krow = eb * A.k.row_stride, vrow = eb * A.v.row_stride;
  const int d_bytes = A.D * eb;
  Biases<kAttnBlockK> biases = {BIAS ? A.bias + kr.row0 : nullptr, bl, kr.len, 0.0f};
  const int nb = (kr.len + kAttnBlockK - 1) / kAttnBlockK;
  const int per = (nb + A.splits - 1) / A.splits;
  const int b0 = pl.split * per;
  const int b1 = m0 >= mlen ? b0 : (b0 + per < nb ? b0 + per : nb);

  Direct<T, DP, kAttnBlockK> kd, vd;
  kd.init((uint32_t)krow, d_bytes);
  vd.init((uint32_t)vrow, d_bytes);
  auto scores = [&](const char* kl, f32x16* sn) __attribute__((always_inline)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      sn[kt] = zero16();
#pragma unroll
      for (int kk = 0; kk < KD; ++kk)
        sn[kt] = Mat<T>::mma(L::row_frag(kl, kt * 32 + (lane & 31), kk, h), qf[kk], sn[kt]);
    }
  };
  // weights of the scores in st, their sums, and the product with V
  auto values = [&](char* vl) __attribute__((always_inline)) {
    const float mu = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      float p[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        p[r] = __builtin_amdgcn_exp2f(BIAS ? st[kt][r] - mu : kFused ? fmaf(st[kt][r], c, -mc) : (st[kt][r] - mu) * c);
        l += p[r];
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Frag pf = Mat<T>::pack(p + 8 * s);
#pragma unroll
        for (int nd = 0; nd < ND; ++nd)
          o[nd] = Mat<T>::mma(L::col_frag(vl, kt * 32 + 16 * s, nd * 32, lane), pf, o[nd]);
      }
    }
  };
  // take block b's scores over: mask them, and move the maximum if they exceed it
  auto take = [&](int b, f32x16* sn) __attribute__((always_inline)) {
    if (BIAS || (b + 1) * kAttnBlockK > kr.len) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        mask_scores<BIAS>(sn[kt], biases.at(b) + kt * 32, c, b * kAttnBlockK + kt * 32, kr.len, h);
    }
    float bm = -INFINITY;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      st[kt] = sn[kt];
#pragma unroll
      for (int r = 0; r < 16; ++r) bm = fmaxf(bm, sn[kt][r]);
    }
    bm = other_half_max(bm);
    if (__any((bm - mx) * unit > kSlack)) {
      const float nm = fmaxf(mx, bm);
      const float f = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((mx - nm) * unit);
      mx = nm;
      l *= f;
#pragma unroll
      for (int nd = 0; nd < ND; ++nd) o[nd] *= f;
      if constexpr (kFused) {
        mc = mx == -INFINITY ? 0.0f : mx * c;
        far = __any(fabsf(mc) > 0x1p24f);
        if (far) mc = 0.0f;
      }
    }
    if (kFused && far) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) st[kt] -= mx == -INFINITY ? 0.0f : mx;
    }
  };
  // block b: its K in kc, the block before's V in vp; K of b + 1 goes to kn, V of b to vc
  auto step = [&](int b, const char* kc, char* kn, char* vp, char* vc) __attribute__((always_inline)) {
    if constexpr (BIAS) biases.advance(b);
    if (b + 1 < b1) kd.load(kb, krow, d_bytes, (b + 1) * kAttnBlockK, kr.len, wave, kn);
    vd.load(vb, vrow, d_bytes, b * kAttnBlockK, kr.len, wave, vc);
    f32x16 sn[KT];
    scores(kc, sn);
    if (b > b0) values(vp);
    take(b, sn);
    wait_loads();
    if constexpr (BIAS) {
      vd.clear(biases.at(b), vc);
      if (b + 1 < b1) kd.clear(biases.at(b + 1), kn);
    }
    __syncthreads();
  };
  if (b0 < b1) {
    kd.load(kb, krow, d_bytes, b0 * kAttnBlockK, kr.len, wave, k0);
    if constexpr (BIAS) biases.start(b0);
    wait_loads();
    __syncthreads();
    if constexpr (BIAS) {
      kd.clear(biases.at(b0), k0);
      __syncthreads();
    }
    int b = b0;
    for (; b + 1 < b1; b += 2) {
      step(b, k0, k1, v1, v0);
      step(b + 1, k1, k0, v0, v1);
    }
    if (b < b1) {
      step(b, k0, k1, v1, v0);
      values(v0);
    } else {
      values(v1);
    }
  }
  l = other_half_sum(l);
  if (m >= M) return;
  if (A.splits > 1) {
    const int64_t e = (((int64_t)pl.split * A.qs.S + pl.s) * A.k.heads + pl.hk) * A.m_max + m;
    const int64_t n = (int64_t)A.splits * A.qs.S * A.k.heads * A.m_max;
    store_column<TDP_F32, ND>(reinterpret_cast<char*>(A.ws + e * DP), h, DP, o, 1.0f);
    if (h == 0) *reinterpret_cast<f32x2*>(A.ws + n * DP + 2 * e) = f32x2{mx, l};
    return;
  }
  const bool live = m < mlen && l != 0.0f;
  char* op = A.o.data + eb * (seq_base(A.qs, A.o, pl.s, qr) + row * A.o.row_stride + head * A.o.head_stride);
  if (!live) {
#pragma unroll
    for (int nd = 0; nd < ND; ++nd) o[nd] = zero16();
  }
  store_column<T, ND>(op, h, A.D, o, live ? 1.0f / l : 0.0f);
  if (A.lse && h == 0)
    A.lse[(int64_t)head * A.qs.total + qr.row0 + row] =
        live ? mx * (BIAS ? kLn2 : A.scale) + logf(l) : -INFINITY;
}

// Join the splits of one query entry per workgroup: weights 2^(c (m_i - max)).
// The waves take the splits in turn, two to four of them in flight each.
template <int T, int DP>
__global__ __launch_bounds__(kTok) void attn_join_kernel(const AttnArgs A, float c, float unit) {
  constexpr int E = DP < 64 ? 1 : DP / 64;
  __shared__ float part[4][E * 64];
  __shared__ f32x2 ml[kAttnMaxSplits];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t g = blockIdx.x;  // ((s, hk), m)
  const int64_t n1 = (int64_t)A.qs.S * A.k.heads * A.m_max;
  const int64_t sh = g / A.m_max;
  const int m = (int)(g - sh * A.m_max), s = (int)(sh / A.k.heads), hk = (int)(sh - (int64_t)s * A.k.heads);
  const SeqRows qr = seq_rows(A.qs, s);
  if (m >= qr.cap * A.group) return;
  if ((int)threadIdx.x < A.splits)
    ml[threadIdx.x] = reinterpret_cast<const f32x2*>(A.ws + n1 * A.splits * DP)[threadIdx.x * n1 + g];
  __syncthreads();
  float mx = -INFINITY, l = 0.0f;
  for (int i = 0; i < A.splits; ++i) mx = fmaxf(mx, ml[i].x);
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.0f;
#pragma unroll 4
  for (int i = wave; i < A.splits; i += 4) {
    // a part without a key holds zeros and -infinity; without any maximum all
    // weights are one (scores that are not numbers come through)
    const float f = mx == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((ml[i].x - mx) * c);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = e * 64 + lane;
      if (d < DP) x[e] = fmaf(A.ws[(i * n1 + g) * DP + d], f, x[e]);
    }
  }
  for (int i = 0; i < A.splits; ++i)
    l = fmaf(ml[i].y, mx == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((ml[i].x - mx) * c), l);
#pragma unroll
  for (int e = 0; e < E; ++e) part[wave][e * 64 + lane] = x[e];
  __syncthreads();
  if (wave) return;
  const int row = (int)fastdiv((uint32_t)m, A.by_group), head = hk * A.group + (m - row * A.group);
  const bool live = row < qr.len && l != 0.0f;
  char* op = A.o.data + Mat<T>::kBytes * (seq_base(A.qs, A.o, s, qr) + row * A.o.row_stride + head * A.o.head_stride);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = e * 64 + lane;
    if (d >= A.D) continue;
    const float y = live ? ((part[0][d] + part[1][d]) + (part[2][d] + part[3][d])) / l : 0.0f;
    if constexpr (T == TDP_BF16)
      reinterpret_cast<__bf16*>(op)[d] = (__bf16)y;
    else
      reinterpret_cast<float*>(op)[d] = y;
  }
  if (A.lse && lane == 0)
    A.lse[(int64_t)head * A.qs.total + qr.row0 + row] = live ? mx * unit + logf(l) : -INFINITY;
}

// A weight again from its score: exp(s - lse) in powers of two, nl = -lse log2(e),
// -infinity for rows without keys.  No weight exceeds one, but lse and its change
// of unit are rounded by up to 2^-22 of it altogether, so past |lse| = 10^8 the
// exponent can be too high by tens or hundreds: infinite weights, gradients that
// are not numbers.  With a bias, which takes scores there more easily, the exponent
// is cut at 0 (one instruction per score, 1 to 2 % of the gradients' time: 6144
// tokens, 16 heads of 128, a 512-token prompt 242 -> 246 us; the minimum keeps a
// NaN, unlike fminf).  Without, the cut would cost 1 % at head_dim
// 128 and 5 % at 64; instead nl is lowered by twice its error beyond 2^24, once
// per row, which keeps every weight below 2^4.
template <bool BIAS>
__device__ inline float weight(float s, float c, float bias, float nl) {
  return __builtin_amdgcn_exp2f(BIAS ? __builtin_elementwise_minimum(fmaf(s, c, bias) + nl, 0.0f) : fmaf(s, c, nl));
}
template <bool BIAS>
__device__ inline float neg_lse(float lse) {
  if (lse == -INFINITY) return -INFINITY;
  const float nl = -lse * kLog2e, past = fabsf(nl) - 0x1p24f;
  return !BIAS && past > 0.0f ? fmaf(past, -0x1p-21f, nl) : nl;
}

// dq: the forward's walk over the keys with a third product.  128 query entries
// per workgroup, 32 per wave; blocks of 64 keys pass through two LDS buffers,
// 32 keys at a time.  The operands of the score products are read ahead of them
// (a barrier for the scheduler, as in attn_dkv_kernel); two workgroups share a
// CU and fill each other's waits.  delta = dout . out is made here, by the lanes
// that hold dout, and left with lse for the dk and dv kernel.  On 4 x 2240 rows,
// 16 heads of 128: 280 us, 0.88 PFLOP/s of its three products (324 us when it ran
// its third product one block behind the scores, as the forward does); its 1152
// workgroups are 2.25 rounds of the 512 places, run as three, and at head_dim 128
// it spills three registers.  Its keys are not split: few tiles of few heads leave
// CUs idle (one of 2048 rows, 3 heads of 128: 48 workgroups).
// The form with a bias takes one workgroup per CU at head_dim 128, where it would
// spill in the loop (gradients of 8 x 480 rows on 343 keys, 9 heads of 96: 70 us
// against 81; of 4 x 2240 rows on 512 keys, 16 heads of 128: 247 against 302).
constexpr int kDqKeys = 64;
template <int T, int DP, bool BIAS>
__global__ __launch_bounds__(kTok, T == TDP_BF16 && !(BIAS && DP == 128) ? 2 : 1) void attn_dq_kernel(const AttnArgs A) {
  typedef Tile<T, DP> L;
  typedef typename Mat<T>::Frag Frag;
  constexpr int KD = DP / 16, ND = DP / 32, kTile = kDqKeys * L::kRow;
  __shared__ __align__(16) char k0[kTile];
  __shared__ __align__(16) char k1[kTile];
  __shared__ __align__(16) char v0[kTile];
  __shared__ __align__(16) char v1[kTile];
  __shared__ __align__(16) float bl[BIAS ? 4 * kDqKeys : 4];
  const uint32_t item = xcd_item(A.tiles);
  if (item >= A.tiles) return;
  const Place pl = place(A, item);
  const SeqRows qr = seq_rows(A.qs, pl.s), kr = seq_rows(A.ks, pl.s);
  const int M = qr.cap * A.group, mlen = qr.len * A.group;
  const int m0 = pl.blk * kAttnBlockQ;
  if (m0 >= M) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int m = m0 + wave * 32 + (lane & 31);
  const bool live = m < mlen;
  const int row = (int)fastdiv((uint32_t)m, A.by_group), head = pl.hk * A.group + (m - row * A.group);
  constexpr int eb = Mat<T>::kBytes;

  auto at = [&](const HeadsDev& t) __attribute__((always_inline)) {
    return live ? t.data + eb * (seq_base(A.qs, t, pl.s, qr) + row * t.row_stride + head * t.head_stride) : nullptr;
  };
  Frag qf[KD], gf[KD];
  float delta = 0.0f;
  {
    Frag of[KD];
    load_frags<T, DP>(at(A.dout), h, A.D, gf);
    load_frags<T, DP>(at(A.o), h, A.D, of);
#pragma unroll
    for (int kk = 0; kk < KD; ++kk)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = fmaf((float)gf[kk][e], (float)of[kk][e], delta);
    delta = other_half_sum(delta);
  }
  load_frags<T, DP>(at(A.q), h, A.D, qf);
  const int64_t stat = (int64_t)head * A.qs.total + qr.row0 + row;
  const float nl = live ? neg_lse<BIAS>(A.lse[stat]) : -INFINITY;
  if (live && h == 0) A.stats[stat] = f32x2{nl, delta};
  const float c = A.scale * kLog2e;
  f32x16 dq[ND];
#pragma unroll
  for (int nd = 0; nd < ND; ++nd) dq[nd] = zero16();

  const char* kb = A.k.data + eb * (seq_base(A.ks, A.k, pl.s, kr) + pl.hk * A.k.head_stride);
  const char* vb = A.v.data + eb * (seq_base(A.ks, A.v, pl.s, kr) + pl.hk * A.v.head_stride);
  const int64_t krow = eb * A.k.row_stride, vrow = eb * A.v.row_stride;
  const int d_bytes = A.D * eb;
  Biases<kDqKeys> biases = {BIAS ? A.bias + kr.row0 : nullptr, bl, kr.len, 0.0f};
  const int nb = m0 >= mlen ? 0 : (kr.len + kDqKeys - 1) / kDqKeys;

  Direct<T, DP, kDqKeys> kd, vd;
  kd.init((uint32_t)krow, d_bytes);
  vd.init((uint32_t)vrow, d_bytes);
  auto load = [&](int b, char* kn, char* vn) __attribute__((always_inline)) {
    kd.load(kb, krow, d_bytes, b * kDqKeys, kr.len, wave, kn);
    vd.load(vb, vrow, d_bytes, b * kDqKeys, kr.len, wave, vn);
  };
  // 32 keys from key k0 of the block in kl and vl
  auto part = [&](int b, int r0, char* kl, char* vl) __attribute__((always_inline)) {
    f32x16 st = zero16(), dp = zero16();
    Frag ka[KD], va[KD];
#pragma unroll
    for (int kk = 0; kk < KD; ++kk) ka[kk] = L::row_frag(kl, r0 + (lane & 31), kk, h);
#pragma unroll
    for (int kk = 0; kk < KD; ++kk) va[kk] = L::row_frag(vl, r0 + (lane & 31), kk, h);
    if (T == TDP_BF16) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < KD; ++kk) st = Mat<T>::mma(ka[kk], qf[kk], st);
#pragma unroll
    for (int kk = 0; kk < KD; ++kk) dp = Mat<T>::mma(va[kk], gf[kk], dp);
    if (!BIAS && b * kDqKeys + r0 + 32 > kr.len) mask_scores<false>(st, nullptr, c, b * kDqKeys + r0, kr.len, h);
    float ds[16];
#pragma unroll
    for (int r = 0; r < 16; ++r)
      ds[r] = weight<BIAS>(st[r], c, BIAS ? biases.at(b)[r0 + 8 * (r >> 2) + 4 * h + (r & 3)] : 0.0f, nl) *
              (dp[r] - delta);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Frag f = Mat<T>::pack(ds + 8 * s);
      Frag tk[ND];
#pragma unroll
      for (int nd = 0; nd < ND; ++nd) tk[nd] = L::col_frag(kl, r0 + 16 * s, nd * 32, lane);
#pragma unroll
      for (int nd = 0; nd < ND; ++nd) dq[nd] = Mat<T>::mma(tk[nd], f, dq[nd]);
    }
  };
  auto step = [&](int b, char* kc, char* vc, char* kn, char* vn) __attribute__((always_inline)) {
    if constexpr (BIAS) biases.advance(b);
    if (b + 1 < nb) load(b + 1, kn, vn);
#pragma unroll
    for (int r0 = 0; r0 < kDqKeys; r0 += 32) part(b, r0, kc, vc);
    wait_loads();
    if constexpr (BIAS) {
      if (b + 1 < nb) {
        kd.clear(biases.at(b + 1), kn);
        vd.clear(biases.at(b + 1), vn);
      }
    }
    __syncthreads();
  };
  if (nb) {
    load(0, k0, v0);
    if constexpr (BIAS) biases.start(0);
    wait_loads();
    __syncthreads();
    if constexpr (BIAS) {
      kd.clear(biases.at(0), k0);
      vd.clear(biases.at(0), v0);
      __syncthreads();
    }
    int b = 0;
    for (; b + 1 < nb; b += 2) {
      step(b, k0, v0, k1, v1);
      step(b + 1, k1, v1, k0, v0);
    }
    if (b < nb) step(b, k0, v0, k1, v1);
  }
  if (m >= M) return;
  char* op = A.dq.data + eb * (seq_base(A.qs, A.dq, pl.s, qr) + row * A.dq.row_stride + head * A.dq.head_stride);
  if (!live) {
#pragma unroll
    for (int nd = 0; nd < ND; ++nd) dq[nd] = zero16();
  }
  store_column<T, ND>(op, h, A.D, dq, A.scale);
}

// The (-lse log2(e), delta) pairs of up to 64 rows into LDS, by the first wave.
__device__ inline void load_stats(const f32x2* from, int left, int wave, int lane, float* lds) {
#ifdef __HIP_DEVICE_COMPILE__
  if (wave) return;
  const uint32_t span = left < 64 ? left * 8 : 512;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<f32x2*>(from), 0, __builtin_amdgcn_readfirstlane(span), 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (TDP_LDS void*)lds, 4, lane * 4, 0, 0, 0);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (TDP_LDS void*)(lds + 64), 4, 256 + lane * 4, 0, 0, 0);
#endif
}

// dk and dv: 128 keys of one key head per workgroup, 32 per wave, their K and V
// in registers.  Blocks of 64 rows of Q and dout, one query head of the group
// after another, pass through three LDS buffers with their lse and delta, one
// being loaded.  They are taken by halves: while one half's scores are
// multiplied, the half before it becomes weights and meets dout and Q again.
// That is the bf16 form at head_dim 128, where only one wave fits a SIMD; smaller
// heads, of which two do (2256 us either way on the conditioned slots), and fp32
// tiles, twice the size under matrix instructions of a sixteenth the rate, take
// two buffers and one half after the other.  Where few key blocks meet many
// rows, the blocks are split over workgroups, whose sums are joined by
// attn_sum_kernel.  On 4 x 2240 rows, 16 heads of 128: 443 us, 0.74 PFLOP/s of its
// four products; K, V and the sums fill all 512 registers (11 spill, 22 with a
// bias), so one wave per SIMD has nothing but its own instructions to cover its
// waits, and the 1152 workgroups are 4.5 rounds of the 256 places, run as five.
constexpr int kDkvRows = 64;
template <int T, int DP, bool BIAS>
__global__ __launch_bounds__(kTok, T == TDP_BF16 && DP <= 64 ? 2 : 1) void attn_dkv_kernel(const AttnArgs A) {
  typedef Tile<T, DP> L;
  typedef typename Mat<T>::Frag Frag;
  constexpr int KD = DP / 16, ND = DP / 32, kTile = kDkvRows * L::kRow;
  __shared__ __align__(16) char q0[kTile];
  __shared__ __align__(16) char q1[kTile];
  __shared__ __align__(16) char g0[kTile];
  __shared__ __align__(16) char g1[kTile];
  constexpr bool kAhead = T == TDP_BF16 && DP == 128;
  __shared__ __align__(16) char q2[kAhead ? kTile : 16];
  __shared__ __align__(16) char g2[kAhead ? kTile : 16];
  __shared__ __align__(16) float s0[2 * kDkvRows];
  __shared__ __align__(16) float s1[2 * kDkvRows];
  __shared__ __align__(16) float s2[2 * kDkvRows];
  const uint32_t item = xcd_item(A.tiles);
  if (item >= A.tiles) return;
  const Place pl = place(A, item);
  const SeqRows qr = seq_rows(A.qs, pl.s), kr = seq_rows(A.ks, pl.s);
  const int j0 = pl.blk * kAttnBlockQ;
  if (j0 >= kr.cap) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int j = j0 + wave * 32 + (lane & 31);
  constexpr int eb = Mat<T>::kBytes;
  float bi = 0.0f;
  bool live = j < kr.len;
  if constexpr (BIAS) {
    bi = live ? A.bias[kr.row0 + j] : -INFINITY;
    bi = bi <= kBiasOut ? -INFINITY : bi * kLog2e;
    live = live && bi != -INFINITY;
  }
  Frag kf[KD], vf[KD];
  load_frags<T, DP>(live ? A.k.data + eb * (seq_base(A.ks, A.k, pl.s, kr) + j * A.k.row_stride +
                                            pl.hk * A.k.head_stride) : nullptr, h, A.D, kf);
  load_frags<T, DP>(live ? A.v.data + eb * (seq_base(A.ks, A.v, pl.s, kr) + j * A.v.row_stride +
                                            pl.hk * A.v.head_stride) : nullptr, h, A.D, vf);
  f32x16 dk[ND], dv[ND], sa, da, sb, db;  // scores and dout . v of first and second halves
#pragma unroll
  for (int nd = 0; nd < ND; ++nd) dk[nd] = dv[nd] = zero16();
  const float c = A.scale * kLog2e;
  const int d_bytes = A.D * eb;
  const int64_t qrow = eb * A.q.row_stride, grow = eb * A.dout.row_stride;

  // blocks of all heads of the group in a row: block b is rows
  // (b mod per_head) * 64 of head b / per_head
  const int per_head = (qr.len + kDkvRows - 1) / kDkvRows;
  const int all = j0 < kr.len ? per_head * A.group : 0;
  const int per = (all + A.splits - 1) / A.splits;
  const int b0 = pl.split * per, b1 = b0 + per < all ? b0 + per : all;

  Direct<T, DP, kDkvRows, true> qd, gd;
  qd.init((uint32_t)qrow, d_bytes);
  gd.init((uint32_t)grow, d_bytes);
  const char* qhead = A.q.data + eb * seq_base(A.qs, A.q, pl.s, qr);
  const char* ghead = A.dout.data + eb * seq_base(A.qs, A.dout, pl.s, qr);
  const f32x2* shead = A.stats + qr.row0;
  int gr = 0;  // row of the next block to load
  // the buffers' rows from the block's first to the end of its head
  int left = 0, left_next = 0;
  auto seek = [&](int head, int row) __attribute__((always_inline)) {
    qhead += eb * head * A.q.head_stride;
    ghead += eb * head * A.dout.head_stride;
    shead += head * A.qs.total;
    gr = row;
  };
  auto load = [&](char* qn, char* gn, float* sn) __attribute__((always_inline)) {
    left_next = qr.len - gr;
    qd.load(qhead, qrow, d_bytes, gr, qr.len, wave, qn);
    gd.load(ghead, grow, d_bytes, gr, qr.len, wave, gn);
    load_stats(shead + gr, left_next, wave, lane, sn);
    gr += kDkvRows;
    if (gr >= qr.len) seek(1, 0);
  };
  // What a half needs from LDS is read ahead of its products, behind barriers
  // for the compiler's scheduler: left to itself it reads each operand right
  // before its product, which with one wave per SIMD exposes every read
  // (4 x 2240 rows, 16 heads of 128: 582 us without, 469 with).
  auto scores = [&](char* ql, char* gl, int r0, f32x16& st, f32x16& dp) __attribute__((always_inline)) {
    st = dp = zero16();
    Frag a[KD], b[KD];
#pragma unroll
    for (int kk = 0; kk < KD; ++kk) {
      a[kk] = L::row_frag(ql, r0 + (lane & 31), kk, h);
      b[kk] = L::row_frag(gl, r0 + (lane & 31), kk, h);
    }
    if (T == TDP_BF16) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < KD; ++kk) {
      st = Mat<T>::mma(a[kk], kf[kk], st);
      dp = Mat<T>::mma(b[kk], vf[kk], dp);
    }
  };
  auto statistics = [&](const float* sl, int r0, f32x4* x) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = *reinterpret_cast<const f32x4*>(sl + 2 * (r0 + 8 * (i >> 1) + 4 * h + 2 * (i & 1)));
  };
  auto values = [&](char* ql, char* gl, const f32x4* x, int r0, int rows, const f32x16& st,
                    const f32x16& dp) __attribute__((always_inline)) {
    float p[16], ds[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 2 * i, row = r0 + 8 * (i >> 1) + 4 * h + 2 * (i & 1);
      float n0 = x[i][0], n1 = x[i][2];
      if constexpr (BIAS) {
        // rows past the end have zeros for Q, dout and their statistics, which
        // a weight of one leaves at zero, but not one that a bias makes infinite
        n0 = row < rows ? n0 : -INFINITY;
        n1 = row + 1 < rows ? n1 : -INFINITY;
      }
      p[r] = weight<BIAS>(st[r], c, bi, n0);
      p[r + 1] = weight<BIAS>(st[r + 1], c, bi, n1);
      ds[r] = p[r] * (dp[r] - x[i][1]);
      ds[r + 1] = p[r + 1] * (dp[r + 1] - x[i][3]);
    }
    const Frag pf[2] = {Mat<T>::pack(p), Mat<T>::pack(p + 8)}, df[2] = {Mat<T>::pack(ds), Mat<T>::pack(ds + 8)};
    if constexpr (kAhead) {
      Frag tv[ND], tk[ND];
#pragma unroll
      for (int nd = 0; nd < ND; ++nd) {
        tv[nd] = L::col_frag(gl, r0, nd * 32, lane);
        tk[nd] = L::col_frag(ql, r0, nd * 32, lane);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int nd = 0; nd < ND; ++nd) {
        dv[nd] = Mat<T>::mma(tv[nd], pf[0], dv[nd]);
        tv[nd] = L::col_frag(gl, r0 + 16, nd * 32, lane);
        dk[nd] = Mat<T>::mma(tk[nd], df[0], dk[nd]);
        tk[nd] = L::col_frag(ql, r0 + 16, nd * 32, lane);
      }
#pragma unroll
      for (int nd = 0; nd < ND; ++nd) {
        dv[nd] = Mat<T>::mma(tv[nd], pf[1], dv[nd]);
        dk[nd] = Mat<T>::mma(tk[nd], df[1], dk[nd]);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int nd = 0; nd < ND; ++nd) {
          dv[nd] = Mat<T>::mma(L::col_frag(gl, r0 + 16 * s, nd * 32, lane), pf[s], dv[nd]);
          dk[nd] = Mat<T>::mma(L::col_frag(ql, r0 + 16 * s, nd * 32, lane), df[s], dk[nd]);
        }
    }
  };
  auto step = [&](int b, char* qc, char* gc, float* sc, char* qp, char* gp, float* sp, char* qn, char* gn,
                  float* sn) __attribute__((always_inline)) {
    const int rows = left_next;
    if (b + 1 < b1) load(qn, gn, sn);
    f32x4 x[8];
    statistics(sp, 32, x);
    scores(qc, gc, 0, sa, da);
    values(qp, gp, x, 32, left, sb, db);
    statistics(sc, 0, x);
    scores(qc, gc, 32, sb, db);
    values(qc, gc, x, 0, rows, sa, da);
    left = rows;
    wait_loads();
    __syncthreads();
  };
  auto step_in_order = [&](int b, char* qc, char* gc, float* sc, char* qn, char* gn,
                           float* sn) __attribute__((always_inline)) {
    const int rows = left_next;
    if (b + 1 < b1) load(qn, gn, sn);
#pragma unroll
    for (int r0 = 0; r0 < kDkvRows; r0 += 32) {
      f32x4 x[8];
      statistics(sc, r0, x);
      scores(qc, gc, r0, sa, da);
      values(qc, gc, x, r0, rows, sa, da);
    }
    wait_loads();
    __syncthreads();
  };
  if (b0 < b1) {
    const int head0 = b0 / per_head;
    seek(pl.hk * A.group + head0, (b0 - head0 * per_head) * kDkvRows);
    load(q0, g0, s0);
    wait_loads();
    __syncthreads();
    if constexpr (!kAhead) {
      int b = b0;
      for (; b + 1 < b1; b += 2) {
        step_in_order(b, q0, g0, s0, q1, g1, s1);
        step_in_order(b + 1, q1, g1, s1, q0, g0, s0);
      }
      if (b < b1) step_in_order(b, q0, g0, s0, q1, g1, s1);
    } else {
      left = left_next;
      if (b0 + 1 < b1) load(q1, g1, s1);
      f32x4 x[8];
      statistics(s0, 0, x);
      scores(q0, g0, 0, sa, da);
      scores(q0, g0, 32, sb, db);
      values(q0, g0, x, 0, left, sa, da);
      wait_loads();
      __syncthreads();
      int b = b0 + 1;
      for (; b + 2 < b1; b += 3) {
        step(b, q1, g1, s1, q0, g0, s0, q2, g2, s2);
        step(b + 1, q2, g2, s2, q1, g1, s1, q0, g0, s0);
        step(b + 2, q0, g0, s0, q2, g2, s2, q1, g1, s1);
      }
      if (b < b1) step(b, q1, g1, s1, q0, g0, s0, q2, g2, s2);
      if (b + 1 < b1) step(b + 1, q2, g2, s2, q1, g1, s1, q0, g0, s0);
      if (b1 == b) {
        statistics(s0, 32, x);
        values(q0, g0, x, 32, left, sb, db);
      } else if (b1 == b + 1) {
        statistics(s1, 32, x);
        values(q1, g1, x, 32, left, sb, db);
      } else {
        statistics(s2, 32, x);
        values(q2, g2, x, 32, left, sb, db);
      }
    }
  }
  if (j >= kr.cap) return;
  if (!live) {
#pragma unroll
    for (int nd = 0; nd < ND; ++nd) dk[nd] = dv[nd] = zero16();
  }
  if (A.splits > 1) {
    const int64_t e = (((int64_t)pl.split * A.ks.S + pl.s) * A.k.heads + pl.hk) * A.ks.max_rows + j;
    const int64_t n = (int64_t)A.splits * A.ks.S * A.k.heads * A.ks.max_rows;
    store_column<TDP_F32, ND>(reinterpret_cast<char*>(A.ws + e * DP), h, DP, dk, A.scale);
    store_column<TDP_F32, ND>(reinterpret_cast<char*>(A.ws + (n + e) * DP), h, DP, dv, 1.0f);
    return;
  }
  store_column<T, ND>(A.dk.data + eb * (seq_base(A.ks, A.dk, pl.s, kr) + j * A.dk.row_stride +
                                        pl.hk * A.dk.head_stride), h, A.D, dk, A.scale);
  store_column<T, ND>(A.dv.data + eb * (seq_base(A.ks, A.dv, pl.s, kr) + j * A.dv.row_stride +
                                        pl.hk * A.dv.head_stride), h, A.D, dv, 1.0f);
}

// Sum the parts of dk and dv in order: a thread per eight elements of a key.
template <int T, int DP>
__global__ __launch_bounds__(kTok) void attn_sum_kernel(const AttnArgs A) {
  constexpr int kPer = DP / 8;
  const int64_t n1 = (int64_t)A.ks.S * A.k.heads * A.ks.max_rows;
  const int64_t t = (int64_t)blockIdx.x * kTok + threadIdx.x;
  const int64_t which = t / (n1 * kPer);  // dk, then dv
  if (which > 1) return;
  const int64_t e = t / kPer - which * n1;
  const int d = (int)(t % kPer) * 8;
  const int64_t sh = e / A.ks.max_rows;
  const int j = (int)(e - sh * A.ks.max_rows), s = (int)(sh / A.k.heads), hk = (int)(sh - (int64_t)s * A.k.heads);
  const SeqRows kr = seq_rows(A.ks, s);
  if (j >= kr.cap || d >= A.D) return;
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int i = 0; i < A.splits; ++i) {
    float y[8];
    load8<TDP_F32>(reinterpret_cast<const char*>(A.ws), ((which * A.splits + i) * n1 + e) * DP + d, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] += y[k];
  }
  const HeadsDev& out = which ? A.dv : A.dk;
  store8<T>(out.data, seq_base(A.ks, out, s, kr) + j * out.row_stride + hk * out.head_stride + d, x);
}

template <int T, int DP, bool BIAS>
void launch_forward(const AttnArgs& A, hipStream_t st) {
  hipLaunchKernelGGL((attn_forward_kernel<T, DP, BIAS>), dim3(xcd_grid(A.tiles)), dim3(kTok), 0, st, A);
  if (A.splits > 1)
    hipLaunchKernelGGL((attn_join_kernel<T, DP>), dim3((unsigned)(A.qs.S * A.k.heads * A.m_max)), dim3(kTok), 0, st, A,
                       BIAS ? 1.0f : A.scale * kLog2e, BIAS ? kLn2 : A.scale);
}

template <int T, int DP, bool BIAS>
void launch_backward(AttnArgs A, int splits, hipStream_t st) {
  hipLaunchKernelGGL((attn_dq_kernel<T, DP, BIAS>), dim3(xcd_grid(A.tiles)), dim3(kTok), 0, st, A);
  A.blocks = (uint32_t)((A.ks.max_rows + kAttnBlockQ - 1) / kAttnBlockQ);
  A.splits = splits;
  A.tiles = A.blocks * (uint32_t)A.ks.S * (uint32_t)A.k.heads * splits;
  hipLaunchKernelGGL((attn_dkv_kernel<T, DP, BIAS>), dim3(xcd_grid(A.tiles)), dim3(kTok), 0, st, A);
  if (splits > 1) {
    const int64_t n = (int64_t)A.ks.S * A.k.heads * A.ks.max_rows * 2 * (DP / 8);
    hipLaunchKernelGGL((attn_sum_kernel<T, DP>), dim3((unsigned)((n + kTok - 1) / kTok)), dim3(kTok), 0, st, A);
  }
}

// The direct loads address a block of 64 rows with 32 bits.
int check_row_strides(const char* fn, int32_t dtype, std::initializer_list<const tdp_heads*> ts) {
  for (const tdp_heads* t : ts)
    if (t->row_stride * dtype_bytes(dtype) > (1 << 25))
      return fail(TDP_ESHAPE, "%s: a row stride of %lld elements exceeds 2^25 bytes", fn, (long long)t->row_stride);
  return TDP_OK;
}

// Checks shared by both calls.
int begin(const char* fn, const tdp_seqs* q_seqs, const tdp_seqs* k_seqs, const tdp_heads* q, const tdp_heads* k,
          const tdp_heads* v, const float* bias, const tdp_heads* out, const float* lse, float scale,
          int32_t head_dim, int32_t dtype, AttnArgs* A) {
  if (!dtype_bytes(dtype)) return fail(TDP_EINVAL, "%s: dtype must be TDP_F32 or TDP_BF16 (got %d)", fn, dtype);
  if (head_dim < 8 || head_dim % 8 != 0 || head_dim > TDP_MAX_ATTENTION_DIM)
    return fail(TDP_ESHAPE, "%s: head_dim must be a multiple of 8 in [8, %d] (got %d)", fn, TDP_MAX_ATTENTION_DIM,
                head_dim);
  if (!(scale > 0.0f) || scale > 3.0e38f) return fail(TDP_EINVAL, "%s: scale must be finite and > 0", fn);
  int st = check_seqs(fn, "q_seqs", q_seqs, &A->qs);
  if (st == TDP_OK) st = check_seqs(fn, "k_seqs", k_seqs, &A->ks);
  if (st != TDP_OK) return st;
  if (q_seqs->num_seqs != k_seqs->num_seqs)
    return fail(TDP_EINVAL, "%s: %d query sequences meet %d key sequences", fn, q_seqs->num_seqs, k_seqs->num_seqs);
  st = check_heads(fn, "q", q, q_seqs, head_dim, dtype, &A->q);
  if (st == TDP_OK) st = check_heads(fn, "k", k, k_seqs, head_dim, dtype, &A->k);
  if (st == TDP_OK) st = check_heads(fn, "v", v, k_seqs, head_dim, dtype, &A->v);
  if (st == TDP_OK) st = check_heads(fn, "out", out, q_seqs, head_dim, dtype, &A->o);
  if (st != TDP_OK) return st;
  if (k->heads != v->heads || q->heads != out->heads || q->heads % k->heads != 0)
    return fail(TDP_EINVAL, "%s: out needs q's heads, v k's, and q's must be a multiple of k's (q %d, k %d, v %d, out %d)",
                fn, q->heads, k->heads, v->heads, out->heads);
  if ((reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(lse)) & 3)
    return fail(TDP_EINVAL, "%s: key_bias and lse must be 4-byte aligned", fn);
  st = check_row_strides(fn, dtype, {q, k, v});
  if (st != TDP_OK) return st;
  A->bias = bias;
  A->lse = const_cast<float*>(lse);
  A->scale = scale;
  A->D = head_dim;
  A->group = q->heads / k->heads;
  A->by_group = make_fastdiv((uint32_t)A->group);
  const int64_t m = (int64_t)q_seqs->max_rows * A->group;
  if (m > (1 << 30)) return fail(TDP_ESHAPE, "%s: %lld rows times heads of one key head exceed 2^30", fn, (long long)m);
  A->m_max = (int32_t)m;
  A->blocks = (uint32_t)((m + kAttnBlockQ - 1) / kAttnBlockQ);
  A->splits = 1;
  return TDP_OK;
}

int check_items(const char* fn, int64_t workgroups) {
  if (workgroups * kTok > 0xffffffffLL - 8 * kTok)
    return fail(TDP_ESHAPE, "%s: %lld workgroups, more work-items than one HIP launch holds", fn, (long long)workgroups);
  return TDP_OK;
}

}  // namespace
}  // namespace tdp

using namespace tdp;

#define TDP_ATTN_DIMS(call, T)                    \
  do {                                            \
    const int dp = attention_padded_dim(head_dim); \
    if (dp == 32) {                               \
      if (key_bias) call(T, 32, true);            \
      else call(T, 32, false);                    \
    } else if (dp == 64) {                        \
      if (key_bias) call(T, 64, true);            \
      else call(T, 64, false);                    \
    } else {                                      \
      if (key_bias) call(T, 128, true);           \
      else call(T, 128, false);                   \
    }                                             \
  } while (0)
#define TDP_ATTN_DISPATCH(call)                    \
  do {                                             \
    if (dtype == TDP_BF16) TDP_ATTN_DIMS(call, TDP_BF16); \
    else TDP_ATTN_DIMS(call, TDP_F32);             \
  } while (0)

extern "C" {

int tdp_attention(const tdp_seqs* q_seqs, const tdp_seqs* k_seqs, const tdp_heads* q, const tdp_heads* k,
                  const tdp_heads* v, const float* key_bias, const tdp_heads* out, float* lse, float scale,
                  int32_t head_dim, int32_t dtype, void* workspace, void* stream) {
  const char* fn = "tdp_attention";
  AttnArgs A = {};
  int st = begin(fn, q_seqs, k_seqs, q, k, v, key_bias, out, lse, scale, head_dim, dtype, &A);
  if (st != TDP_OK) return st;
  A.splits = attention_splits(*q_seqs, *k_seqs, q->heads, k->heads);
  if (A.splits > 1 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return fail(TDP_EINVAL, "%s: workspace must be a 16-byte aligned device pointer (tdp_attention_workspace)", fn);
  A.ws = static_cast<float*>(workspace);
  const int64_t tiles = (int64_t)A.blocks * q_seqs->num_seqs * k->heads * A.splits;
  const int64_t join = A.splits > 1 ? (int64_t)q_seqs->num_seqs * k->heads * A.m_max : 0;
  st = check_items(fn, tiles > join ? tiles : join);
  if (st != TDP_OK) return st;
  A.tiles = (uint32_t)tiles;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
#define CALL(T, DP, B) launch_forward<T, DP, B>(A, hs)
  TDP_ATTN_DISPATCH(CALL);
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

int tdp_attention_backward(const tdp_seqs* q_seqs, const tdp_seqs* k_seqs, const tdp_heads* q, const tdp_heads* k,
                           const tdp_heads* v, const float* key_bias, const tdp_heads* out, const float* lse,
                           const tdp_heads* dout, const tdp_heads* dq, const tdp_heads* dk, const tdp_heads* dv,
                           float scale, int32_t head_dim, int32_t dtype, void* workspace, void* stream) {
  const char* fn = "tdp_attention_backward";
  AttnArgs A = {};
  int st = begin(fn, q_seqs, k_seqs, q, k, v, key_bias, out, lse, scale, head_dim, dtype, &A);
  if (st == TDP_OK) st = check_heads(fn, "dout", dout, q_seqs, head_dim, dtype, &A.dout);
  if (st == TDP_OK) st = check_heads(fn, "dq", dq, q_seqs, head_dim, dtype, &A.dq);
  if (st == TDP_OK) st = check_heads(fn, "dk", dk, k_seqs, head_dim, dtype, &A.dk);
  if (st == TDP_OK) st = check_heads(fn, "dv", dv, k_seqs, head_dim, dtype, &A.dv);
  if (st != TDP_OK) return st;
  if (dout->heads != q->heads || dq->heads != q->heads || dk->heads != k->heads || dv->heads != k->heads)
    return fail(TDP_EINVAL, "%s: dout and dq need q's heads, dk and dv k's", fn);
  if (!lse) return fail(TDP_EINVAL, "%s: null lse", fn);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return fail(TDP_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
  st = check_row_strides(fn, dtype, {dout});
  if (st != TDP_OK) return st;
  A.stats = static_cast<f32x2*>(workspace);
  A.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(*q_seqs, q->heads));
  const int splits = dkv_splits(*q_seqs, *k_seqs, q->heads, k->heads);
  const int64_t qt = A.blocks * ((int64_t)q_seqs->num_seqs * k->heads);
  const int64_t kt = dkv_blocks(*k_seqs, k->heads) * splits;
  const int64_t sum = splits > 1 ? ((int64_t)k_seqs->num_seqs * k->heads * k_seqs->max_rows * 32 + kTok - 1) / kTok : 0;
  st = check_items(fn, qt > kt ? (qt > sum ? qt : sum) : (kt > sum ? kt : sum));
  if (st != TDP_OK) return st;
  A.tiles = (uint32_t)qt;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
#define CALL(T, DP, B) launch_backward<T, DP, B>(A, splits, hs)
  TDP_ATTN_DISPATCH(CALL);
#undef CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

}  // extern "C"

// Products of groups of rows with weights of their own, and their gradients
// (gfx950 matrix instructions).
//
//   y_i = W_e x_i,  dx_i = W_e^T dy_i,  dW_e = sum_i dy_i x_i^T
//
// for the used rows i of the sequences that take weight e.  All three are tiles
// of out[q][p] = sum_r P[p][r] Q[q][r] (p: output features, q: rows, or W's rows
// for dW) in 32 x 32 tiles of the matrix instructions with fp32 accumulators.
// Operands come in two layouts: the contraction along memory rows (x and W of
// y, dy of dx) or across them (W of dx, both of dW); the second kind is read
// from LDS by transposing reads (bf16) or column by column (fp32).
//
// Which rows a sequence has is known on the device only.  Every workgroup counts
// the blocks of rows of all sequences (64 at a time, a lane each) and finds its
// own, so the launch has one workgroup per possible block and those past the
// count leave at once.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

#include "layer_internal.h"
#include "token_device.h"

namespace tdp {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define TDP_LDS __attribute__((address_space(3)))

enum Kind { kForward, kInput, kWeight };  // y, dx, dW
enum Pass { kAll, kRounds, kRest };

// Tiles of 256 by 256 run one to a CU, and a last round of few of them takes as
// long as a full one.  Up to kRestTiles tiles beyond whole rounds of 256 are left to
// a second launch, in quarters of 128 by 128 that have a CU each (gradients of
// 24576 rows for 8 weights of 2048 x 2048, about 800 tiles of dx: 415 us against
// 427).  With twice as many it gains nothing.
constexpr uint32_t kRestTiles = 64;
__host__ __device__ inline uint32_t rest_tiles(uint32_t tiles) {
  const uint32_t rest = tiles % 256;
  return rest <= kRestTiles ? rest : 0;
}

template <int T>
struct Mat;
template <>
struct Mat<TDP_BF16> {
  typedef bf16x8 Frag;
  static constexpr int kBytes = 2;
  __device__ static inline f32x16 mma(const Frag& a, const Frag& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
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
};

struct ProductArgs {
  SeqsDev seqs;
  HeadsDev x, y;      // y: its gradient for dx and dW
  HeadsDev dx;
  const char* w;      // (weights, N, K)
  float *dw, *ws;
  int32_t E, N, K;    // weights, output and input features
  int32_t splits;     // y, dx: of the contraction; dW: weight_places
  uint32_t np;        // tiles of output features
  uint32_t nq;        // dW: tiles of W's rows
  int32_t pass;       // y, dx: kAll, kRounds or kRest
  bool flat;          // y, dx: one weight for all, blocks of the tensors' rows
};

// 16 bytes per lane from a buffer straight into 1 KB of LDS.  Written out because
// the compiler, which cannot tell the stages of a ring of buffers apart around a
// loop, makes reads of one wait for loads into the others; wait_barrier says what
// has to be there.  Nothing is returned in registers.  `lds` and the descriptor
// are the same in all lanes.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // that m0 is not kept, which nothing here relies on
__device__ inline void load_lds(const u32x4& buffer, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(off), "s"(buffer)
               : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ inline uint32_t lds_address(const char* p) { return (uint32_t)(uintptr_t)(TDP_LDS const char*)p; }
// Bytes past `span` read as zeros.
__device__ inline u32x4 buffer_of(const char* base, uint32_t span) {
  const uint64_t a = reinterpret_cast<uintptr_t>(base);
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) & 0xffffu,
               (uint32_t)__builtin_amdgcn_readfirstlane((int)span), 0x00020000u};
}

// A stage is 128 bytes of the contraction: whole cache lines where it runs along
// the operand's rows.  Half of that makes every line cross from L2 twice (256 by
// 256 tiles of 8192 x 8192 x 8192: 906 us against 867).
constexpr int kStageBytes = 128;

// An operand whose contraction runs along its rows: ROWS rows in LDS, chunk c of
// row r at c ^ swizzle(r), so that 16 lanes reading one chunk of 16 rows meet
// every bank once.
template <int T, int ROWS, int THREADS>
struct Along {
  typedef typename Mat<T>::Frag Frag;
  static constexpr int kChunks = kStageBytes / 16, kBytes = ROWS * kStageBytes, kLoads = kBytes / 16 / THREADS;
  static_assert(kBytes % (16 * THREADS) == 0 && THREADS / kChunks % 16 == 0, "whole loads");
  uint32_t off[kLoads];
  int chunk16;  // bytes from the row's first to this lane's chunk
  u32x4 buffer;
  bool in;
  __device__ static inline int swizzle(int r) { return r >> 1 & 7; }
  __device__ inline void init(uint32_t row_bytes) {
    const int r = threadIdx.x / kChunks;
    chunk16 = ((threadIdx.x % kChunks) ^ swizzle(r)) * 16;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) off[n] = (r + n * (THREADS / kChunks)) * row_bytes + chunk16;
  }
  // the next loads: `rows` rows from `base` on, of which `left` bytes remain
  __device__ inline void seek(const char* base, uint32_t row_bytes, int rows, int left) {
    buffer = buffer_of(base, rows > 0 && left > 0 ? (uint32_t)((rows < ROWS ? rows : ROWS) - 1) * row_bytes + left : 0);
    in = chunk16 < left;
  }
  __device__ inline void load(int n, uint32_t lds, int wave) const {
    load_lds(buffer, lds + (n * THREADS + wave * 64) * 16, in ? off[n] : 0xfffffff0u);
  }
  // rows r0 + lane % 32, contractions 16 kk + 8h ..
  __device__ static inline Frag frag(const char* lds, int r0, int kk, int lane) {
    const int r = r0 + (lane & 31), h = lane >> 5, s = swizzle(r);
    const char* row = lds + r * kStageBytes;
    if constexpr (T == TDP_BF16) {
      return *reinterpret_cast<const bf16x8*>(row + ((2 * kk + h) ^ s) * 16);
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(row + ((4 * kk + 2 * h) ^ s) * 16);
      const f32x4 b = *reinterpret_cast<const f32x4*>(row + ((4 * kk + 2 * h + 1) ^ s) * 16);
      return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
};

// An operand whose contraction runs across its rows, which hold COLS elements,
// chunk c of row r at c ^ 4 (r % 4): the four rows that a transposing read touches
// lie in different quarters of the banks.  ANEW: fp32 columns' places are made anew
// for each fragment.  Kept over the loop, those of both operands of dW take the
// registers of two waves per SIMD and more, and reading them back from memory waits
// for the operands' loads too (4096 x 4096 x 4096: 1214 us, 1083 anew).
template <int T, int COLS, int THREADS, bool ANEW>
struct Across {
  typedef typename Mat<T>::Frag Frag;
  static constexpr int kRow = COLS * Mat<T>::kBytes, kChunks = kRow / 16, kRows = kStageBytes / Mat<T>::kBytes;
  static constexpr int kBytes = kRows * kRow, kLoads = kBytes / 16 / THREADS;
  static_assert(kChunks % 16 == 0, "room for the swizzle");
  static_assert(kBytes % (16 * THREADS) == 0 && THREADS % kChunks == 0 && THREADS / kChunks % 4 == 0, "whole rows");
  uint32_t off[kLoads];
  int row, rows_left;
  u32x4 buffer;
  __device__ inline void init(uint32_t row_bytes) {
    row = threadIdx.x / kChunks;
    const int c = (threadIdx.x % kChunks) ^ ((row & 3) << 2);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) off[n] = (row + n * (THREADS / kChunks)) * row_bytes + c * 16;
  }
  // the next loads: `rows` rows from `base` on, each with `left` bytes from there
  __device__ inline void seek(const char* base, uint32_t row_bytes, int rows, int left) {
    buffer = buffer_of(base, rows > 0 ? (uint32_t)((rows < kRows ? rows : kRows) - 1) * row_bytes + left : 0);
    rows_left = rows;
  }
  __device__ inline void load(int n, uint32_t lds, int wave) const {
    load_lds(buffer, lds + (n * THREADS + wave * 64) * 16,
             row + n * (THREADS / kChunks) < rows_left ? off[n] : 0xfffffff0u);
  }
  __device__ static inline Frag frag(char* lds, int c0, int kk, int lane) {
    const int h = lane >> 5;
    if constexpr (T == TDP_BF16) {
      const int r = 16 * kk + 8 * h + ((lane & 15) >> 2), c = c0 + (lane & 16) + 4 * (lane & 3);
      const int at = r * kRow + (((c >> 3) ^ ((r & 3) << 2)) << 4) + (c & 7) * 2;
      typedef TDP_LDS bf16x4* P;
      const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((P)(TDP_LDS char*)(lds + at));
      const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((P)(TDP_LDS char*)(lds + at + 4 * kRow));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      int at = 8 * h * kRow + 4 * (c0 + (lane & 31));
      if (ANEW) asm volatile("" : "+v"(at));
      f32x8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = *reinterpret_cast<const float*>(lds + (16 * kk + e) * kRow + (at ^ ((e & 3) << 6)));
      return v;
    }
  }
};

// Wait for this wave's loads into LDS, all but the last N of them (63: none), and
// for its reads of LDS, then for the other waves.  The compiler moves no access of memory
// across.
template <int N>
__device__ inline void wait_barrier() {
  static_assert(N < 64, "six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x0070 | (N >> 4) << 14);  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The same where only some waves wait for loads.
template <int N>
__device__ inline void wait_barrier_if(bool loads) {
  asm volatile("" ::: "memory");
  if (loads) __builtin_amdgcn_s_waitcnt((N & 15) | 0x0f70 | (N >> 4) << 14);
  wait_barrier<63>();
}

__device__ inline int wave_prefix(int v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(v, d);
    if (lane >= d) v += t;
  }
  return v;
}

__device__ inline int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }

// Blocks of `rows` rows of every sequence in order, found by whole waves; of
// the tensors' rows, whatever sequences they are, if flat.
struct RowBlocks {
  const SeqsDev& q;
  int rows, lane;
  bool flat;
  __device__ inline int count(int s) const {
    if (s >= q.S) return 0;
    return (seq_rows(q, s).cap + rows - 1) / rows;
  }
  __device__ inline int total() const {
    if (flat) return (int)((q.total + rows - 1) / rows);
    if (!q.range) return q.S * ((q.max_rows + rows - 1) / rows);
    int n = 0;
    for (int s = 0; s < q.S; s += 64) n += last_lane(wave_prefix(count(s + lane), lane));
    return n;
  }
  // the sequence of block t, which becomes the block's number in it
  __device__ inline int find(int& t) const {
    if (flat) return 0;
    if (!q.range) {
      const int per = (q.max_rows + rows - 1) / rows, s = t / per;
      t -= s * per;
      return s;
    }
    for (int s = 0; s < q.S; s += 64) {
      const int n = count(s + lane), end = wave_prefix(n, lane);
      const uint64_t past = __ballot(end > t);
      if (past) {
        const int l = __builtin_ctzll(past);
        t -= __builtin_amdgcn_readlane(end - n, l);
        return s + l;
      }
      t -= last_lane(end);
    }
    return 0;  // not reached: t is below the total
  }
};

// Which rows of a block of the tensors' rows some sequence owns and uses: the
// sequences that reach into it are listed in LDS (as many as the block has rows at
// most, since written ranges do not overlap), and each lane looks its rows up.
template <int BQ, int THREADS>
struct BlockRows {
  static constexpr int kBytes = (1 + 3 * BQ) * 4;
  int n;
  const int* list;
  __device__ inline void find(const SeqsDev& q, int r0, int* lds) {
    if (threadIdx.x == 0) lds[0] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < q.S; s += THREADS) {
      const SeqRows r = seq_rows(q, s);
      const int a = (int)(r.row0 - r0);
      if (r.cap > 0 && a < BQ && a + r.cap > 0) {
        const int i = atomicAdd(lds, 1);  // any order: the entries exclude each other
        if (i < BQ) {
          lds[1 + 3 * i] = a;
          lds[2 + 3 * i] = a + r.len;
          lds[3 + 3 * i] = a + r.cap;
        }
      }
    }
    __syncthreads();
    n = lds[0] < BQ ? lds[0] : BQ;
    list = lds + 1;
  }
  __device__ inline bool any_used() const {
    bool any = false;
    for (int i = 0; i < n; ++i) any |= list[3 * i + 1] > 0 && list[3 * i + 1] > list[3 * i];
    return any;
  }
  __device__ inline void look_up(int row, bool& used, bool& owned) const {
    used = owned = false;
    for (int i = 0; i < n; ++i) {
      const bool in = row >= list[3 * i];
      used |= in && row < list[3 * i + 1];
      owned |= in && row < list[3 * i + 2];
    }
  }
};

// Workgroups are dealt round-robin to the eight XCDs, each of which takes a
// contiguous range of the tiles.  Runs of eight tiles along q share one of p, and
// the tiles that an XCD's 32 CUs hold at a time are eight by four: they read
// twelve panels of operands through its L2 instead of 64.
// xcd_item: the workgroup's item of `count`, or false.
__device__ inline bool xcd_item(uint32_t count, uint32_t b, uint32_t& item) {
  const uint32_t per = (count + 7) / 8, slot = b >> 3;
  item = (b & 7) * per + slot;
  return slot < per && item < count;
}
__device__ inline void tile_at(uint32_t nq, uint32_t np, uint32_t item, uint32_t& q, uint32_t& p) {
  const uint32_t group = item / (8 * np), first = group * 8, rest = item - first * np;
  const uint32_t n = nq - first < 8 ? nq - first : 8;
  p = rest / n;
  q = first + (rest - p * n);
}

__device__ inline f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}

// The wave's 32 rows of TP tiles of features, through 4 KB of LDS of its own so
// that whole runs of features leave at once.  OUT: type written.  Row lane % 32
// becomes zero unless `used`, and is written if `owned`; features past `left` are not.
template <int OUT, int TP>
__device__ inline void store_tile(char* out, int64_t row_bytes, bool used, bool owned, int left, const f32x16* acc,
                                  int lane, char* lds) {
  constexpr int eb = OUT == TDP_BF16 ? 2 : 4;
  constexpr int U = OUT == TDP_BF16 && TP > 1 ? 2 : 1;  // tiles side by side in a row of 128 bytes at most
  constexpr int kChunks = U * 32 * eb / 16, kRowsAtOnce = 64 / kChunks;
  const int r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int u0 = 0; u0 < TP; u0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = used ? acc[u0 + u][r4 * 4 + e] : 0.0f;
        const int f = u * 32 + r4 * 8 + h * 4, c = f * eb / 16;
        char* at = lds + r * 128 + ((c ^ (r >> 1 & (kChunks - 1))) << 4) + f * eb % 16;
        if constexpr (OUT == TDP_BF16) {
          uint2 v;
          v.x = pack_bf16x2(x[0], x[1]);
          v.y = pack_bf16x2(x[2], x[3]);
          *reinterpret_cast<uint2*>(at) = v;
        } else {
          *reinterpret_cast<f32x4*>(at) = f32x4{x[0], x[1], x[2], x[3]};
        }
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 32; i += kRowsAtOnce) {
      const int row = i + lane / kChunks, c = lane % kChunks;
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * 128 + ((c ^ (row >> 1 & (kChunks - 1))) << 4));
      const int f = u0 * 32 + c * (16 / eb);
      const bool write = __shfl((int)owned, row);
      if (write && f < left) *reinterpret_cast<u32x4*>(out + row * row_bytes + f * eb) = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// dW's work: the steps of each weight's rows, in parts of at most about a
// `places`-th of all steps, so that a weight with many rows does not outlast the
// others; the longest parts first, which leaves the short ones to fill the gaps.
// Weights of one part are written directly, the others' parts go to slots of
// the workspace: fewer than 2 places, as a weight of n > 1 parts has more than n - 1
// and so at least n / 2 times a part's steps.  More than 64 weights are taken
// whole, in order.  All lanes of all waves call it, `lds` has room for 64 numbers.
struct WeightParts {
  int steps, n, from, slot;  // a lane's weight: its steps, parts, place among all parts, slot of its first (n > 1)
  int total;                 // parts of all weights
  __device__ inline void count(const ProductArgs& A, int step_rows, int lane, int* lds) {
    if (threadIdx.x < 64) lds[threadIdx.x] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < A.seqs.S; s += blockDim.x)
      atomicAdd(lds + s % A.E, (seq_rows(A.seqs, s).len + step_rows - 1) / step_rows);  // whole numbers: any order
    __syncthreads();
    steps = lane < A.E ? lds[lane] : 0;
    __syncthreads();
    const int all = last_lane(wave_prefix(steps, lane)), even = (all + A.splits - 1) / A.splits;
    const int most = even < kWeightSteps ? kWeightSteps : even;
    n = lane < A.E ? (steps <= most ? 1 : (steps + most - 1) / most) : 0;
    const int length = n ? (steps + n - 1) / n : 0;
    from = 0;
    for (int j = 0; j < A.E; ++j) {
      const int lj = __builtin_amdgcn_readlane(length, j), nj = __builtin_amdgcn_readlane(n, j);
      if (lj > length || (lj == length && j < lane)) from += nj;
    }
    const int slots = n > 1 ? n : 0;
    slot = wave_prefix(slots, lane) - slots;
    total = last_lane(wave_prefix(n, lane));
  }
};

// Where an operand of dW reads next: rows of the sequences e, e + step, ... that
// share a weight, one sequence after another.
struct RowCursor {
  int seq, left;  // rows not yet read of the sequence
  const char* at;
  __device__ inline void begin(const SeqsDev& q, const HeadsDev& t, int s, int skip, int eb, int64_t offset) {
    const SeqRows r = seq_rows(q, s);
    seq = s;
    left = r.len - skip;
    at = t.data + eb * (seq_base(q, t, s, r) + skip * t.row_stride) + offset;
  }
  // to a sequence with rows left, if there is one
  __device__ inline void settle(const SeqsDev& q, const HeadsDev& t, int step, int eb, int64_t offset) {
    while (left <= 0 && seq + step < q.S) begin(q, t, seq + step, 0, eb, offset);
  }
};

// BP x BQ output tile per workgroup of WP x WQ waves, in one of two ways.
//
// Eight waves, 256 by 256 (bf16): two waves share a SIMD and take turns, one
// multiplying 32 of the contraction (16 matrix instructions back to back) while
// the other reads its next operands from LDS and sends loads out; a barrier ends
// each turn.  P has three buffers of a stage and Q two, all of the 160 KB: loads
// have a whole stage's products to arrive behind.
//
// Four waves: STAGES buffers of both, each 16 of the contraction read while the
// 16 before are multiplied; two workgroups or more share a CU and fill each
// other's waits, so the 128 by 128 tile is held to the registers of two waves per
// SIMD (against one, 4096 x 4096 x 4096 fp32: y 1015 us and 1211, dW 1083 and 1338;
// 8 x 1000 rows, 1024 -> 2048 bf16: dx 38 and 58).
template <int T, int KIND, int BP, int BQ, int WP, int WQ, int STAGES>
__global__ __launch_bounds__(64 * WP * WQ, BQ == 128 && STAGES == 2 ? 2 : 1) void product_kernel(const ProductArgs A) {
  constexpr int THREADS = 64 * WP * WQ, eb = Mat<T>::kBytes, kStep = kStageBytes / eb, KK = kStep / 16;
  constexpr int TP = BP / WP / 32, TQ = BQ / WQ / 32;
  constexpr bool kTurns = WP * WQ == 8;
  typedef typename Mat<T>::Frag Frag;
  typedef std::conditional_t<KIND == kForward, Along<T, BP, THREADS>, Across<T, BP, THREADS, KIND == kWeight>> OpP;
  typedef std::conditional_t<KIND == kWeight, Across<T, BQ, THREADS, true>, Along<T, BQ, THREADS>> OpQ;
  constexpr int kP = kTurns ? 3 : STAGES, kQ = kTurns ? 2 : STAGES;  // buffers
  __shared__ __align__(1024) char lds_p[kP * OpP::kBytes];
  __shared__ __align__(1024) char lds_q[kQ * OpQ::kBytes];
  static_assert(kP * OpP::kBytes >= 4096 * WP * WQ, "the epilogue's place");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wp = wave % WP, wq = wave / WP;

  // the tile: its block of rows, or of W's rows, and its features
  uint32_t tq, tp;
  int s = 0, blk = 0, e = 0;
  SeqRows sr = {};
  const int split = KIND == kWeight ? 0 : blockIdx.y;
  int w_part = 0, w_parts = 1, w_steps = 0, w_slot = -1;  // dW
  int f0, r0;
  bool some = false, used[TQ], owned[TQ];  // some row of the tile; the lane's
  if constexpr (KIND != kWeight) {
    const bool quarters = BQ == 128 && A.pass == kRest;  // of the tiles of 256 that are left
    const RowBlocks rb = {A.seqs, quarters ? 256 : BQ, lane, A.flat};
    const uint32_t nq = (uint32_t)rb.total(), all = nq * A.np, rest = A.pass == kAll ? 0 : rest_tiles(all);
    uint32_t item;
    if (!xcd_item(quarters ? 4 * rest : all - rest, blockIdx.x, item)) return;
    tile_at(nq, A.np, quarters ? all - rest + item / 4 : item, tq, tp);
    blk = (int)tq;
    s = rb.find(blk);
    if (A.flat) {
      sr.span = sr.cap = sr.len = (int)A.seqs.total;
    } else {
      sr = seq_rows(A.seqs, s);
    }
    e = s % A.E;
    f0 = (int)tp * (quarters ? 256 : BP);
    r0 = blk * (quarters ? 256 : BQ);
    if (quarters) {
      r0 += (item & 1) * 128;
      f0 += (item >> 1 & 1) * 128;
      if (r0 >= sr.cap || f0 >= (KIND == kForward ? A.N : A.K)) return;
    }
    some = r0 < sr.len;
    if (A.flat) {
      static_assert(kP * OpP::kBytes >= BlockRows<BQ, THREADS>::kBytes, "room for the list");
      BlockRows<BQ, THREADS> br;
      br.find(A.seqs, r0, reinterpret_cast<int*>(lds_p));
      some = br.any_used();
#pragma unroll
      for (int j = 0; j < TQ; ++j) br.look_up((wq * TQ + j) * 32 + (lane & 31), used[j], owned[j]);
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < TQ; ++j) {
        const int row = r0 + (wq * TQ + j) * 32 + (lane & 31);
        used[j] = row < sr.len;
        owned[j] = row < sr.cap;
      }
    }
  } else {
    const uint32_t grid = (A.nq * A.np + 7) / 8 * 8;
    const int part = blockIdx.x / grid;
    uint32_t item;
    if (!xcd_item(A.nq * A.np, blockIdx.x - part * grid, item)) return;
    tile_at(A.nq, A.np, item, tq, tp);
    f0 = (int)tp * BP;
    r0 = (int)tq * BQ;
#pragma unroll
    for (int j = 0; j < TQ; ++j) used[j] = owned[j] = r0 + (wq * TQ + j) * 32 + (lane & 31) < A.N;
    if (A.E <= 64) {
      WeightParts wp;
      wp.count(A, kStep, lane, reinterpret_cast<int*>(lds_p));
      if (part >= wp.total) return;
      const int l = __builtin_ctzll(__ballot(part >= wp.from && part < wp.from + wp.n));
      e = l;
      w_part = part - __builtin_amdgcn_readlane(wp.from, l);
      w_parts = __builtin_amdgcn_readlane(wp.n, l);
      w_steps = __builtin_amdgcn_readlane(wp.steps, l);
      if (w_parts > 1) w_slot = __builtin_amdgcn_readlane(wp.slot, l) + w_part;
    } else {
      e = part;
      for (int i = e; i < A.seqs.S; i += 64 * A.E) {
        const int sq = i + lane * A.E;
        const int n = sq < A.seqs.S ? (seq_rows(A.seqs, sq).len + kStep - 1) / kStep : 0;
        w_steps += last_lane(wave_prefix(n, lane));
      }
    }
  }
  const char* w = A.w + (int64_t)e * A.N * A.K * eb;
  const int features = KIND == kForward ? A.N : A.K;   // of the output
  const int inner = KIND == kForward ? A.K : A.N;      // y and dx: the contraction's length
  const int64_t xrow = A.x.row_stride * eb, yrow = A.y.row_stride * eb;

  OpP P;
  OpQ Q;
  f32x16 acc[TQ][TP];
#pragma unroll
  for (int j = 0; j < TQ; ++j)
#pragma unroll
    for (int i = 0; i < TP; ++i) acc[j][i] = zero16();

  // where the next loads begin
  uint32_t prow, qrow;
  int t0, t1;  // steps
  RowCursor pc, qc;  // dW; y and dx use `at` alone
  if constexpr (KIND != kWeight) {
    const int steps = some ? (inner + kStep - 1) / kStep : 0, per = (steps + A.splits - 1) / A.splits;
    t0 = split * per;
    t1 = t0 + per < steps ? t0 + per : steps;
    const HeadsDev& in = KIND == kForward ? A.x : A.y;
    qrow = (uint32_t)(in.row_stride * eb);
    qc.at = in.data + eb * ((A.flat ? 0 : seq_base(A.seqs, in, s, sr)) + r0 * in.row_stride) +
            (int64_t)t0 * kStageBytes;
    prow = (uint32_t)A.K * eb;
    pc.at = KIND == kForward ? w + (int64_t)f0 * prow + (int64_t)t0 * kStageBytes
                             : w + (int64_t)t0 * kStep * prow + f0 * eb;
  } else {
    prow = (uint32_t)xrow;
    qrow = (uint32_t)yrow;
    // the sequence that this part begins in
    auto steps_of = [&](int sq) { return sq < A.seqs.S ? (seq_rows(A.seqs, sq).len + kStep - 1) / kStep : 0; };
    const int per = (w_steps + w_parts - 1) / w_parts;
    t0 = w_part * per;
    t1 = t0 + per < w_steps ? t0 + per : w_steps;
    int skip = t0, seq = e;
    if (t0 < t1)
      for (int i = e; i < A.seqs.S; i += 64 * A.E) {
        const int n = steps_of(i + lane * A.E), end = wave_prefix(n, lane);
        const uint64_t past = __ballot(end > skip);
        if (past) {
          const int l = __builtin_ctzll(past);
          skip -= __builtin_amdgcn_readlane(end - n, l);
          seq = i + l * A.E;
          break;
        }
        skip -= last_lane(end);
      }
    pc.begin(A.seqs, A.x, seq, skip * kStep, eb, f0 * eb);
    qc.begin(A.seqs, A.y, seq, skip * kStep, eb, r0 * eb);
  }
  P.init(prow);
  Q.init(qrow);
  int p_at = t0 * kStep, q_at = p_at;  // y and dx: the contraction's place
  // Set an operand's next stage up.  Past the last step it holds zeros, or rows of
  // the next part.
  auto seek_p = [&]() __attribute__((always_inline)) {
    if constexpr (KIND == kForward) {
      P.seek(pc.at, prow, A.N - f0, (inner - p_at) * eb);
      pc.at += kStageBytes;
    } else if constexpr (KIND == kInput) {
      P.seek(pc.at, prow, inner - p_at, (A.K - f0) * eb);
      pc.at += (int64_t)kStep * prow;
    } else {
      pc.settle(A.seqs, A.x, A.E, eb, f0 * eb);
      P.seek(pc.at, prow, pc.left, (A.K - f0) * eb);
      pc.at += (int64_t)kStep * xrow;
      pc.left -= kStep;
    }
    p_at += kStep;
  };
  auto seek_q = [&]() __attribute__((always_inline)) {
    if constexpr (KIND != kWeight) {
      Q.seek(qc.at, qrow, sr.len - r0, (inner - q_at) * eb);
      qc.at += kStageBytes;
    } else {
      qc.settle(A.seqs, A.y, A.E, eb, r0 * eb);
      Q.seek(qc.at, qrow, qc.left, (A.N - r0) * eb);
      qc.at += (int64_t)kStep * yrow;
      qc.left -= kStep;
    }
    q_at += kStep;
  };
  const uint32_t p0 = lds_address(lds_p), q0 = lds_address(lds_q);
  auto load_p = [&](int buf, int n) __attribute__((always_inline)) { P.load(n, p0 + buf * OpP::kBytes, wave); };
  auto load_q = [&](int buf, int n) __attribute__((always_inline)) { Q.load(n, q0 + buf * OpQ::kBytes, wave); };
  auto fill_p = [&](int buf) __attribute__((always_inline)) {
    seek_p();
#pragma unroll
    for (int n = 0; n < OpP::kLoads; ++n) load_p(buf, n);
  };
  auto fill_q = [&](int buf) __attribute__((always_inline)) {
    seek_q();
#pragma unroll
    for (int n = 0; n < OpQ::kLoads; ++n) load_q(buf, n);
  };
  Frag a[2][TP], b[2][TQ];
  auto read = [&](int pbuf, int qbuf, int kk, int set) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TP; ++i) a[set][i] = OpP::frag(lds_p + pbuf * OpP::kBytes, (wp * TP + i) * 32, kk, lane);
#pragma unroll
    for (int j = 0; j < TQ; ++j) b[set][j] = OpQ::frag(lds_q + qbuf * OpQ::kBytes, (wq * TQ + j) * 32, kk, lane);
  };
  if constexpr (kTurns) {
    static_assert(KK == 4, "two turns of 32");
    // The first four waves run a turn ahead of the others, whose SIMDs they share.
    // A buffer is free once the second four have read it, one turn behind the first;
    // these fill Q's in the reading turn after that, the second four already while
    // they multiply in that time.  What a stage needs of a wave has arrived when the
    // turn before its first reading ends: the first four wait as they end their
    // multiplying turn, the others as they end their reading one.
    const bool ahead = wave < 4;
    auto products = [&](int buf) __attribute__((always_inline)) {  // buf >= 0: fill Q's meanwhile
      if (buf >= 0 && !ahead) seek_q();
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < TQ; ++j) {
#pragma unroll
          for (int i = 0; i < TP; ++i) acc[j][i] = Mat<T>::mma(a[k][i], b[k][j], acc[j][i]);
          if (buf >= 0 && k == 0 && j < OpQ::kLoads) {
            __builtin_amdgcn_sched_barrier(0);
            if (!ahead) load_q(buf, j);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
    };
    static_assert(OpQ::kLoads <= TQ, "a load after each row of products");
    auto stage = [&](int pbuf, int qbuf) __attribute__((always_inline)) {
      read(pbuf, qbuf, 0, 0);
      read(pbuf, qbuf, 1, 1);
      if (ahead) fill_q(qbuf ^ 1);
      wait_barrier<63>();
      products(-1);
      wait_barrier<63>();
      read(pbuf, qbuf, 2, 0);
      read(pbuf, qbuf, 3, 1);
      fill_p((pbuf + 2) % 3);
      wait_barrier_if<OpP::kLoads>(!ahead);
      products(qbuf);
      wait_barrier_if<OpP::kLoads>(ahead);
    };
    if (t0 < t1) {
      fill_p(0);
      fill_q(0);
      fill_p(1);
      if (ahead) {
        wait_barrier<OpP::kLoads>();
      } else {
        fill_q(1);
        wait_barrier<OpP::kLoads + OpQ::kLoads>();
        wait_barrier<63>();
      }
      for (int t = t0;;) {
        stage(0, 0);
        if (++t >= t1) break;
        stage(1, 1);
        if (++t >= t1) break;
        stage(2, 0);
        if (++t >= t1) break;
        stage(0, 1);
        if (++t >= t1) break;
        stage(1, 0);
        if (++t >= t1) break;
        stage(2, 1);
        if (++t >= t1) break;
      }
      if (ahead) wait_barrier<63>();
    }
  } else {
    // Ahead of a stage's last 16 its buffers are read whole and the next stage is
    // there: the waves meet with products still to do, then the buffers are filled
    // again.  Loads go out one by one between the products, as fast as they are
    // taken (back to back they hold the wave up).
    constexpr int kLoads = OpP::kLoads + OpQ::kLoads;
    static_assert(KK % 2 == 0, "the sets take turns");
    auto stage = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const bool last = kk == KK - 1, first = kk == 0;
        if (last) wait_barrier<(STAGES - 2) * kLoads>();
        const int next = (buf + 1) % STAGES, before = (buf + STAGES - 1) % STAGES;
        read(last ? next : buf, last ? next : buf, last ? 0 : kk + 1, ~kk & 1);
        if (first) seek_q();
        if (last) seek_p();
#pragma unroll
        for (int j = 0; j < TQ; ++j) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < TP; ++i) acc[j][i] = Mat<T>::mma(a[kk & 1][i], b[kk & 1][j], acc[j][i]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = 0; n < OpP::kLoads; ++n)
            if (last && n * TQ / OpP::kLoads == j) load_p(buf, n);
#pragma unroll
          for (int n = 0; n < OpQ::kLoads; ++n)
            if (first && n * TQ / OpQ::kLoads == j) load_q(before, n);
        }
      }
    };
    if (t0 < t1) {
#pragma unroll
      for (int i = 0; i < STAGES; ++i) {
        fill_p(i);
        if (i < STAGES - 1) fill_q(i);
      }
      wait_barrier<(STAGES - 1) * kLoads - OpQ::kLoads>();
      read(0, 0, 0, 0);
      for (int t = t0;;) {
        stage(0);
        if (++t >= t1) break;
        stage(1);
        if (++t >= t1) break;
        if constexpr (STAGES == 4) {
          stage(2);
          if (++t >= t1) break;
          stage(3);
          if (++t >= t1) break;
        }
      }
    }
  }
  wait_barrier<0>();
  // out
  char* lds = lds_p + wave * 4096;
  const int wf = f0 + wp * TP * 32;
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    const int row = r0 + (wq * TQ + j) * 32;
    if constexpr (KIND == kWeight) {
      float* out = (w_slot >= 0 ? A.ws + (int64_t)w_slot * A.N * A.K : A.dw + (int64_t)e * A.N * A.K) +
                   (int64_t)row * A.K + wf;
      store_tile<TDP_F32, TP>(reinterpret_cast<char*>(out), (int64_t)A.K * 4, used[j], owned[j], A.K - wf, acc[j], lane,
                              lds);
    } else if (A.splits > 1) {
      // parts lie by the tensor's rows: (splits, total rows, features)
      float* out = A.ws + ((int64_t)split * A.seqs.total + sr.row0 + row) * features + wf;
      store_tile<TDP_F32, TP>(reinterpret_cast<char*>(out), (int64_t)features * 4, used[j], owned[j], features - wf,
                              acc[j], lane, lds);
    } else {
      const HeadsDev& o = KIND == kForward ? A.y : A.dx;
      char* out = o.data + eb * ((A.flat ? 0 : seq_base(A.seqs, o, s, sr)) + row * o.row_stride + wf);
      store_tile<T, TP>(out, o.row_stride * eb, used[j], owned[j], features - wf, acc[j], lane, lds);
    }
  }
}

constexpr int kJoin = 256;

// Sum the parts of y or dx in order: a workgroup per block of rows and columns.
template <int T>
__global__ __launch_bounds__(kJoin) void product_join_kernel(const ProductArgs A, HeadsDev o, int features, int rows) {
  const int lane = threadIdx.x & 63;
  const RowBlocks rb = {A.seqs, rows, lane, false};
  int blk = blockIdx.x;
  if (blk >= rb.total()) return;
  const int s = rb.find(blk);
  const SeqRows sr = seq_rows(A.seqs, s);
  const int per = features / 4, c = (blockIdx.y * kJoin + threadIdx.x) % per, r = (blockIdx.y * kJoin + threadIdx.x) / per;
  const int row = blk * rows + r;
  if (r >= rows || row >= sr.cap) return;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* from = A.ws + (sr.row0 + row) * features + c * 4;
#pragma unroll 4
  for (int i = 0; i < A.splits; ++i) v += *reinterpret_cast<const f32x4*>(from + (int64_t)i * A.seqs.total * features);
  char* to = o.data + Mat<T>::kBytes * (seq_base(A.seqs, o, s, sr) + row * o.row_stride + c * 4);
  if constexpr (T == TDP_BF16) {
    uint2 b;
    b.x = pack_bf16x2(v[0], v[1]);
    b.y = pack_bf16x2(v[2], v[3]);
    *reinterpret_cast<uint2*>(to) = b;
  } else {
    *reinterpret_cast<f32x4*>(to) = v;
  }
}

// dW of the weights of several parts, summed in order with eight parts' loads under
// way.  A thread takes one quad, and up to 16 where that fills the CUs, since each
// workgroup counts the sequences first: for one weight of 512 x 384 in 42 parts
// 7 us, against 158 with 16 quads each and a part's load at a time.
constexpr int kJoinQuads = 16;
__global__ __launch_bounds__(kJoin) void weight_join_kernel(const ProductArgs A, int step_rows, int each) {
  __shared__ int counts[64];
  const int lane = threadIdx.x & 63, e = blockIdx.y;
  WeightParts wp;
  wp.count(A, step_rows, lane, counts);
  const int n = __builtin_amdgcn_readlane(wp.n, e);
  if (n == 1) return;
  const int64_t quads = (int64_t)A.N * A.K / 4;
  const f32x4* parts = reinterpret_cast<const f32x4*>(A.ws) + __builtin_amdgcn_readlane(wp.slot, e) * quads;
  f32x4* out = reinterpret_cast<f32x4*>(A.dw) + e * quads;
  for (int k = 0; k < each; ++k) {
    const int64_t i = ((int64_t)blockIdx.x * each + k) * kJoin + threadIdx.x;
    if (i >= quads) return;
    f32x4 v = parts[i];
    int j = 1;
    for (; j + 8 <= n; j += 8) {
      f32x4 p[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) p[u] = parts[(j + u) * quads + i];
#pragma unroll
      for (int u = 0; u < 8; ++u) v += p[u];
    }
    for (; j < n; ++j) v += parts[j * quads + i];
    out[i] = v;
  }
}

int check_items(const char* fn, int64_t workgroups, int threads) {
  if (workgroups * threads > 0xffffffffLL - 8 * threads)
    return fail(TDP_ESHAPE, "%s: %lld workgroups, more work-items than one HIP launch holds", fn, (long long)workgroups);
  return TDP_OK;
}

int begin(const char* fn, const tdp_seqs* seqs, const tdp_rows* x, const void* weight, int32_t num_weights,
          const tdp_rows* y, int32_t in_features, int32_t out_features, int32_t dtype, ProductArgs* A) {
  if (!dtype_bytes(dtype)) return fail(TDP_EINVAL, "%s: dtype must be TDP_F32 or TDP_BF16 (got %d)", fn, dtype);
  int st = check_product(fn, seqs, num_weights, in_features, out_features);
  if (st == TDP_OK) st = check_seqs(fn, "seqs", seqs, &A->seqs);
  if (st == TDP_OK) st = check_rows(fn, "x", x, dtype, &A->x);
  if (st == TDP_OK) st = check_rows(fn, "y", y, dtype, &A->y);
  if (st != TDP_OK) return st;
  if (!weight || (reinterpret_cast<uintptr_t>(weight) & 15))
    return fail(TDP_EINVAL, "%s: weight must be a 16-byte aligned device pointer", fn);
  for (const tdp_rows* t : {x, y})
    if (t->row_stride * dtype_bytes(dtype) > (1 << 23))
      return fail(TDP_ESHAPE, "%s: a row stride of %lld elements exceeds 2^23 bytes", fn, (long long)t->row_stride);
  A->w = static_cast<const char*>(weight);
  A->E = num_weights;
  A->N = out_features;
  A->K = in_features;
  return TDP_OK;
}

// A launch over blocks of rows: y or dx.  Without `enqueue` only its checks.
template <int T, int KIND, int BP, int BQ, int WP, int WQ, int STAGES>
int launch_rows(const char* fn, ProductArgs A, const tdp_seqs& seqs, const ProductShape& sh, bool enqueue,
                hipStream_t st) {
  const int features = KIND == kForward ? A.N : A.K;
  A.np = (uint32_t)((features + BP - 1) / BP);
  A.splits = sh.splits;
  const HeadsDev &in = KIND == kForward ? A.x : A.y, &out = KIND == kForward ? A.y : A.dx;
  auto one_matrix = [&](const HeadsDev& t) { return seqs.row_range || t.seq_stride == seqs.max_rows * t.row_stride; };
  A.flat = flat_rows(seqs, A.E) && one_matrix(in) && one_matrix(out);
  const int64_t blocks = row_blocks(seqs, BQ, A.flat), tiles = (blocks * A.np + 7) / 8 * 8;
  const int64_t join_y = ((int64_t)kJoinRows * (features / 4) + kJoin - 1) / kJoin, join_x = row_blocks(seqs, kJoinRows);
  int rc = check_items(fn, tiles * sh.splits, 64 * WP * WQ);
  if (rc == TDP_OK && sh.splits > 1) rc = check_items(fn, join_x * join_y, kJoin);
  if (rc != TDP_OK || !enqueue) return rc;
  if constexpr (BQ == 256) {
    // except for ragged sequences the tiles are known here
    if (sh.splits == 1 && ((seqs.row_range && !A.flat) || rest_tiles((uint32_t)(blocks * A.np)))) A.pass = kRounds;
  }
  hipLaunchKernelGGL((product_kernel<T, KIND, BP, BQ, WP, WQ, STAGES>), dim3((unsigned)tiles, (unsigned)sh.splits),
                     dim3(64 * WP * WQ), 0, st, A);
  if constexpr (BQ == 256) {
    if (A.pass == kRounds) {
      A.pass = kRest;
      hipLaunchKernelGGL((product_kernel<T, KIND, 128, 128, 2, 2, 4>), dim3(4 * kRestTiles), dim3(256), 0, st, A);
    }
  }
  if (sh.splits > 1)
    hipLaunchKernelGGL((product_join_kernel<T>), dim3((unsigned)join_x, (unsigned)join_y), dim3(kJoin), 0, st, A, out,
                       features, kJoinRows);
  return TDP_OK;
}

template <int T, int BP, int BQ, int WP, int WQ>
int launch_weight(const char* fn, ProductArgs A, const ProductShape& sh, bool enqueue, hipStream_t st) {
  A.np = (uint32_t)((A.K + BP - 1) / BP);
  A.nq = (uint32_t)((A.N + BQ - 1) / BQ);
  A.splits = sh.splits;
  // of weights split at `places`: at most one part more each than `places` in all
  const int64_t parts = A.E + (sh.splits > 1 ? sh.splits : 0), quads = (int64_t)A.N * A.K / 4;
  const int64_t tiles = ((int64_t)A.np * A.nq + 7) / 8 * 8 * parts;
  int64_t each = quads * A.E / (kJoin * 2048);
  each = each < 1 ? 1 : (each > kJoinQuads ? kJoinQuads : each);
  const int64_t join = (quads + kJoin * each - 1) / (kJoin * each);
  int rc = check_items(fn, tiles, 64 * WP * WQ);
  if (rc == TDP_OK && sh.splits > 1) rc = check_items(fn, join * A.E, kJoin);
  if (rc != TDP_OK || !enqueue) return rc;
  hipLaunchKernelGGL((product_kernel<T, kWeight, BP, BQ, WP, WQ, 2>), dim3((unsigned)tiles), dim3(64 * WP * WQ), 0, st,
                     A);
  if (sh.splits > 1)
    hipLaunchKernelGGL(weight_join_kernel, dim3((unsigned)join, (unsigned)A.E), dim3(kJoin), 0, st, A,
                       kStageBytes / Mat<T>::kBytes, (int)each);
  return TDP_OK;
}

template <int KIND>
int run_rows(const char* fn, const ProductArgs& A, const tdp_seqs& seqs, const ProductShape& sh, int32_t dtype,
             bool enqueue, hipStream_t st) {
  constexpr int NB = KIND == kForward ? kNarrowY : kNarrowDx;
  if (dtype == TDP_BF16) {
    if (sh.rows == 256) return launch_rows<TDP_BF16, KIND, 256, 256, 4, 2, 2>(fn, A, seqs, sh, enqueue, st);
    if (sh.rows == 128 && sh.deep) return launch_rows<TDP_BF16, KIND, 128, 128, 2, 2, 4>(fn, A, seqs, sh, enqueue, st);
    if (sh.rows == 128) return launch_rows<TDP_BF16, KIND, 128, 128, 2, 2, 2>(fn, A, seqs, sh, enqueue, st);
    return launch_rows<TDP_BF16, KIND, NB, 32, NB / 32, 1, 2>(fn, A, seqs, sh, enqueue, st);
  }
  if (sh.rows == 128 && sh.deep) return launch_rows<TDP_F32, KIND, 128, 128, 2, 2, 4>(fn, A, seqs, sh, enqueue, st);
  if (sh.rows == 128) return launch_rows<TDP_F32, KIND, 128, 128, 2, 2, 2>(fn, A, seqs, sh, enqueue, st);
  return launch_rows<TDP_F32, KIND, NB, 32, NB / 32, 1, 2>(fn, A, seqs, sh, enqueue, st);
}

int run_weight(const char* fn, const ProductArgs& A, const ProductShape& sh, int32_t dtype, bool enqueue,
               hipStream_t st) {
  if (dtype == TDP_F32) return launch_weight<TDP_F32, 128, 128, 2, 2>(fn, A, sh, enqueue, st);
  if (sh.rows == 256) return launch_weight<TDP_BF16, 256, 256, 4, 2>(fn, A, sh, enqueue, st);
  return launch_weight<TDP_BF16, 128, 128, 2, 2>(fn, A, sh, enqueue, st);
}

int check_workspace(const char* fn, const ProductShape& sh, const void* ws) {
  if (sh.splits > 1 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15)))
    return fail(TDP_EINVAL, "%s: workspace must be a 16-byte aligned device pointer (%s_workspace)", fn, fn);
  return TDP_OK;
}

}  // namespace
}  // namespace tdp

using namespace tdp;

extern "C" {

int tdp_grouped_product(const tdp_seqs* seqs, const tdp_rows* x, const void* weight, int32_t num_weights,
                        const tdp_rows* y, int32_t in_features, int32_t out_features, int32_t dtype, void* workspace,
                        void* stream) {
  const char* fn = "tdp_grouped_product";
  ProductArgs A = {};
  int st = begin(fn, seqs, x, weight, num_weights, y, in_features, out_features, dtype, &A);
  if (st != TDP_OK) return st;
  const ProductShape sh = rows_shape(*seqs, out_features, in_features, dtype, kNarrowY, flat_rows(*seqs, num_weights));
  st = check_workspace(fn, sh, workspace);
  if (st != TDP_OK) return st;
  A.ws = static_cast<float*>(workspace);
  st = run_rows<kForward>(fn, A, *seqs, sh, dtype, true, reinterpret_cast<hipStream_t>(stream));
  if (st != TDP_OK) return st;
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

int tdp_grouped_product_backward(const tdp_seqs* seqs, const tdp_rows* x, const void* weight, int32_t num_weights,
                                 const tdp_rows* dy, const tdp_rows* dx, float* dweight, int32_t in_features,
                                 int32_t out_features, int32_t dtype, void* workspace, void* stream) {
  const char* fn = "tdp_grouped_product_backward";
  ProductArgs A = {};
  int st = begin(fn, seqs, x, weight, num_weights, dy, in_features, out_features, dtype, &A);
  if (st == TDP_OK && dx) st = check_rows(fn, "dx", dx, dtype, &A.dx);
  if (st != TDP_OK) return st;
  if (reinterpret_cast<uintptr_t>(dweight) & 15)
    return fail(TDP_EINVAL, "%s: dweight must be 16-byte aligned", fn);
  const ProductShape si = rows_shape(*seqs, in_features, out_features, dtype, kNarrowDx, flat_rows(*seqs, num_weights));
  const ProductShape sw = weight_shape(*seqs, num_weights, in_features, out_features, dtype);
  if (dx) st = check_workspace(fn, si, workspace);
  if (st == TDP_OK && dweight) st = check_workspace(fn, sw, workspace);
  if (st != TDP_OK) return st;
  A.ws = static_cast<float*>(workspace);
  A.dw = dweight;
  hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  for (const bool enqueue : {false, true}) {
    if (st == TDP_OK && dx) st = run_rows<kInput>(fn, A, *seqs, si, dtype, enqueue, hs);
    if (st == TDP_OK && dweight) st = run_weight(fn, A, sw, dtype, enqueue, hs);
  }
  if (st != TDP_OK) return st;
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TDP_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TDP_OK;
}

}  // extern "C"

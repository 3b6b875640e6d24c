// Launch shapes and workspace sizes of the layer operators (layer norm, grouped
// products), shared by the host side (tokens.cpp) and the kernels.
#pragma once

#include "token_internal.h"

namespace tdp {

// Layer norm: lanes per row (the power of two that holds it in eight elements
// each, up to a wave; wider rows take four passes of a wave, then the workgroup).
inline int norm_rows_per_block(int32_t channels) {
  const int chunks = channels / 8;
  return chunks <= 8 ? 32 : chunks <= 16 ? 16 : chunks <= 32 ? 8 : chunks <= 256 ? 4 : 1;
}
inline int64_t norm_blocks(int32_t max_rows, int32_t channels) {
  const int r = norm_rows_per_block(channels);
  return ((int64_t)max_rows + r - 1) / r;
}
// Workgroups per set of weights in the backward launch; each leaves two partial
// rows of sums, so more of them cost the join and fewer leave CUs idle (35840 rows
// of 2048 bf16: 81 us with 512, 86 with 384, 84 with 256).
constexpr int kLayerNormParts = 512;
inline int64_t layer_norm_parts(const tdp_seqs& s, int32_t channels, int32_t sets) {
  const int64_t blocks = norm_blocks(s.max_rows, channels) * ((s.num_seqs + sets - 1) / sets);
  int64_t n = (kLayerNormParts + sets - 1) / sets;
  return n < blocks ? n : blocks;
}

// Grouped products.  With one weight for all sequences the rows need not be told
// apart before they are stored, so tiles may be of the tensors' rows, across the
// ends of sequences.  Taken where these are short and their last tiles are a large
// part of all (bf16, y and dx: 24 x 46 rows of 1632 -> 5696 34 and 41 us against 76
// and 74 with tiles of their own, 48 x 100 of 2048 -> 2048 50 and 49 against 58 and
// 60, but 48 x 200 95 and 99 against 92 and 88); looking the rows up costs long
// sequences 3 %.
inline bool flat_rows(const tdp_seqs& s, int32_t weights) {
  return weights == 1 && s.num_seqs > 1 && s.total_rows < (int64_t)s.num_seqs * 192;
}
// Blocks of `rows` rows of the tensors if flat, else of the sequences: exactly
// where these are uniform, else at most one unfinished block each.
inline int64_t row_blocks(const tdp_seqs& s, int rows, bool flat = false) {
  if (flat) return (s.total_rows + rows - 1) / rows;
  if (!s.row_range) return seq_blocks(s, rows);
  return s.total_rows / rows + (s.num_seqs < s.total_rows ? s.num_seqs : s.total_rows);
}
struct ProductShape {
  int rows;    // of the output tile: 256 (by 256 features), 128 (by 128) or 32 (by kNarrowY or kNarrowDx)
  int splits;  // of the contraction
  bool deep;   // 128 rows: four stages on their way instead of two, one workgroup per CU
};
constexpr int kNarrowY = 64, kNarrowDx = 128;
constexpr int kJoinRows = 8;
constexpr int kProductMaxSplits = 16;
inline int64_t tiles_across(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }
// y (features = N, inner = K) and dx (the other way round): the tile and the
// splits of the contraction that a model of the time expects to be fastest.  A
// step of 128 bytes of the contraction takes a tile `wait` ns on its own and `busy`
// of a CU that is full of them; splitting costs a launch and the parts' traffic.
// Where all tiles of 128 have a CU to themselves, they keep four stages on their
// way instead of two (8 x 100 x 2048 -> 2048: 19 us against 27).  Measured, bf16, with
// tiles of 32, 128 and 256 rows: 64 x 2048 -> 2048 12, 18 and 39 us (128 in 8 splits
// 14); 8 x 256 x 1024 -> 1024 12, 12 and 24; 4 x 2240 x 512 -> 512 14, 13 and 17; 32 x
// 150 x 2048 -> 4096 270, 180 and 149; 200 x 4096 -> 4096 35, 30 and 71 (128 in 4 splits
// 20).  fp32, 32 and 128 rows: 64 x 2048 -> 2048 48 and 132 (32 in splits 18); 4 x 2240
// x 512 -> 512 54 and 69.
inline ProductShape rows_shape(const tdp_seqs& s, int32_t features, int32_t inner, int32_t dtype, int narrow,
                               bool flat) {
  struct Tile {
    int rows;
    int64_t wait, busy;
  };
  const bool bf16 = dtype == TDP_BF16;
  const Tile tiles[3] = {{32, bf16 ? 300 : 750, (bf16 ? 210 : 280) * narrow / 64},
                         {128, bf16 ? 430 : 1900, bf16 ? 580 : 2000},
                         {256, 1100, 1700}};
  const int64_t all = inner * dtype_bytes(dtype), total = (all + 127) / 128;
  ProductShape best = {32, 1, false};
  int64_t least = INT64_MAX;
  for (int i = 0; i < (bf16 ? 3 : 2); ++i) {
    const int width = i == 0 ? narrow : tiles[i].rows;
    const int64_t n = row_blocks(s, tiles[i].rows, flat) * tiles_across(features, width);
    for (int sp = 1; sp <= kProductMaxSplits && (sp == 1 || total >= 4 * sp); sp *= 2) {
      const int64_t steps = (total + sp - 1) / sp, rounds = (n * sp + 255) / 256;
      int64_t ns = rounds * tiles[i].busy > tiles[i].wait ? rounds * tiles[i].busy : tiles[i].wait;
      ns = ns * steps + (sp == 1 ? 0 : 9000 + sp * s.total_rows * features / 500);  // 8 bytes at 4 TB/s
      if (ns < least) {
        least = ns;
        best = {tiles[i].rows, sp, i == 1 && n * sp <= 256};
      }
    }
  }
  return best;
}
// dW: its tile of W's rows is `rows` too, the contraction the rows of a weight's
// sequences.  How many rows a weight has is known on the device only, so `splits`
// says in how many parts the rows of all weights are cut where one has them all
// (parts of less than kWeightSteps steps are not worth a slot).  A step does not
// reach across the end of a sequence, so many short ones are many steps of few rows.
constexpr int kWeightSteps = 8;
constexpr int kWeightMaxPlaces = 64;
inline ProductShape weight_shape(const tdp_seqs& s, int32_t weights, int32_t in_features, int32_t out_features,
                                 int32_t dtype) {
  const int64_t big = weights * tiles_across(in_features, 256) * tiles_across(out_features, 256);
  ProductShape sh = {dtype == TDP_BF16 && big >= 192 ? 256 : 128, 1, false};
  if (weights > 64) return sh;
  const int64_t tiles = tiles_across(in_features, sh.rows) * tiles_across(out_features, sh.rows);
  int64_t n = (sh.rows == 256 ? 256 : 512) / tiles;
  const int64_t steps = row_blocks(s, 128 / dtype_bytes(dtype));
  if (n > steps / kWeightSteps) n = steps / kWeightSteps;
  if (n > kWeightMaxPlaces) n = kWeightMaxPlaces;
  sh.splits = n < 2 ? 1 : (int)n;
  return sh;
}
inline int64_t rows_workspace(const tdp_seqs& s, int32_t features, int32_t inner, int32_t dtype, int narrow,
                              bool flat) {
  const ProductShape sh = rows_shape(s, features, inner, dtype, narrow, flat);
  return sh.splits == 1 ? 0 : align256(sh.splits * s.total_rows * features * 4);
}
inline int64_t weight_workspace(const tdp_seqs& s, int32_t weights, int32_t in_features, int32_t out_features,
                                int32_t dtype) {
  const ProductShape sh = weight_shape(s, weights, in_features, out_features, dtype);
  return sh.splits == 1 ? 0 : align256((int64_t)2 * sh.splits * in_features * out_features * 4);
}
// Sequences and the weights that they share: at most 2^30, so that sums of two such
// numbers stay in 32 bits, here and in the kernels.
int check_weights(const char* fn, const tdp_seqs* seqs, int32_t num_weights);
int check_product(const char* fn, const tdp_seqs* seqs, int32_t num_weights, int32_t in_features,
                  int32_t out_features);

}  // namespace tdp

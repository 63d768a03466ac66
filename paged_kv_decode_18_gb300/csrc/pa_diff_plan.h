// pa_diff_plan.h -- sizes of differential attention's launches; plain
// arithmetic, for the library and for a test on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

constexpr int kMapRows = 8;    // rows of one map in a warp tile
constexpr int kDFixWarps = 8;  // of a CTA of the warp tiles' merge, at most

// Most (sequence, query tile) pairs of S windows of at most `longest` tokens, T tokens in
// all, in tiles of `unit` tokens.
inline int64_t diff_pairs(int64_t S, int64_t T, int64_t longest, int unit) {
  const int64_t by_window = S * ((longest + unit - 1) / unit), by_token = (T + unit - 1) / unit + S;
  return by_window < by_token ? by_window : by_token;
}

// The longest window that the warp tiles take beside tcgen05 tiles of min_lq tokens and more.
inline int64_t diff_warp_longest(int64_t max_q_len, int min_lq) {
  return max_q_len < min_lq ? max_q_len : min_lq - 1;
}

// Whether a plan's flat tiles, `heads` segments of up to `tiles` each to a pair, are counted in
// 32 bits, and (the cuts' arithmetic inside a pair) their costs in quarters of a tile too.
inline bool diff_tiles_fit(int64_t pairs, int64_t heads, int64_t tiles, int start_cost4) {
  const int64_t most = 0x7fffffff;
  if (heads <= 0 || tiles <= 0) return true;
  return tiles <= most / heads && pairs <= most / (heads * tiles) &&
         4 * tiles + start_cost4 <= most / heads;
}

// The merge of warp tiles: a CTA has `warps` warps for `chunk` rows of a segment, and
// `chunks` CTAs a segment's rows. A row has a warp at least, whatever number of rows the
// device finds in a window: chunk <= warps.
struct DiffMerge {
  int warps, chunk, chunks;
};

// by_row: few segments in many pieces. longest: the longest window that the call
// announces; QT query tokens and G heads make a tile.
inline DiffMerge diff_merge(bool by_row, int64_t longest, int QT, int G) {
  const int rows = (int)(longest < QT ? longest : QT) * G;
  DiffMerge m;
  m.warps = by_row || rows > kDFixWarps / 2 ? kDFixWarps : kDFixWarps / 2;
  m.chunk = by_row ? 1 : m.warps;
  m.chunks = by_row ? rows : 1;
  return m;
}

// Which row of its CTA's a warp merges, and which of the row's `per_row` warps it is
// (a row is `nrows` or more: none).
struct DiffDeal {
  int row, group, per_row;
};
PA_HD DiffDeal diff_deal(int warps, int nrows, int warp) {
  DiffDeal d;
  d.per_row = warps / nrows;
  d.row = warp / d.per_row;
  d.group = warp - d.row * d.per_row;
  return d;
}

}  // namespace pa

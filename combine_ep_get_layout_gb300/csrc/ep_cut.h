// How the experts' rows are cut into tiles of columns of a product: every
// warp of a call (and the host that sizes it) has to find the same cut, so
// the rules are here once.  Host and device; no CUDA header.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define EP_BOTH __host__ __device__ __forceinline__
#else
#define EP_BOTH inline
#endif

namespace ep {

constexpr int kColumnStep = 32;  // columns of a pair's product come in these

EP_BOTH int ceil_over(int a, int b) { return a / b + (a % b != 0); }

// Where a call's rows end: `cap` of them are there, an expert has at most
// `most_rows`, a tile at most `max_cols` (a multiple of kColumnStep).
struct RowLimits {
  int cap, most_rows, max_cols;
};

// The rows of an expert that are computed, of `count` from `first` on.
EP_BOTH int rows_within(const RowLimits &l, int first, int count) {
  if (first < 0 || first >= l.cap || count < 0) return 0;
  const int left = l.cap - first < l.most_rows ? l.cap - first : l.most_rows;
  return count < left ? count : left;
}

// As few tiles as hold the rows, of about equal size.
EP_BOTH int tiles_of(const RowLimits &l, int rows) { return ceil_over(rows, l.max_cols); }

// Columns of a tile of these rows, the last one perhaps excepted, which takes
// no more than it needs.  Not monotone: 260 rows by at most 256 are two tiles
// of 160 columns, 256 are one of 256.
EP_BOTH int tile_cols(const RowLimits &l, int rows) {
  if (rows == 0) return 0;
  return ceil_over(ceil_over(rows, tiles_of(l, rows)), kColumnStep) * kColumnStep;
}

// The rows of tile `part` of an expert's, from *from on.
EP_BOTH int tile_rows(const RowLimits &l, int rows, int part, int *from) {
  const int cols = tile_cols(l, rows);
  *from = part * cols;
  return rows - *from < cols ? rows - *from : cols;
}

// The most columns that a tile of any such call has.
EP_BOTH int most_cols_of(const RowLimits &l) {
  const int n = ceil_over(l.most_rows, kColumnStep) * kColumnStep;
  return n < kColumnStep ? kColumnStep : n < l.max_cols ? n : l.max_cols;
}

// The most columns that a tile of experts from, from + step, ... has: of the
// rows that are computed, since an expert that the capacity cuts may be a
// single, wider tile.
EP_BOTH int widest_tile(const RowLimits &l, const int32_t *offset, const int32_t *count, int experts, int from, int step) {
  int most = 0;
#pragma unroll 8
  for (int e = from; e < experts; e += step) {
    const int cols = tile_cols(l, rows_within(l, offset[e], count[e]));
    most = cols > most ? cols : most;
  }
  return most;
}

}  // namespace ep

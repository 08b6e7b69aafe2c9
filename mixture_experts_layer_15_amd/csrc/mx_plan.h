// How the 4-bit calls count their rows: host code without a GPU header (the
// kernels use it too), so that a test without a GPU can try it.
#pragma once

namespace moe {

// ---- expert network: rows in groups of 32, none of two experts

// Groups of an expert's `rows` rows, counted up to a multiple of `unit`.
constexpr int mx_groups(int rows, int unit) {
  return rows / (32 * unit) * unit + (rows % (32 * unit) ? unit : 0);
}

// Most groups that El segments of S rows in all have if none overlap (each
// segment of r rows at most r / 32 + unit - 1 / 32).
constexpr long long mx_max_groups(long long S, int El, int unit) { return S / 32 + (S < El ? S : El) * unit; }

// A running number of groups, held to what the workspace has room for: bounds
// that do not ascend make segments that overlap, with more groups in all.
constexpr int mx_add_groups(int before, int n, int limit) { return before + n < limit ? before + n : limit; }

// ---- conversion: tiles of 256 columns and 8 or 64 rows

constexpr int kMxTileCols = 256;

struct MxConvertPlan {
  int rt;         // rows of a tile
  int row_tiles;  // of one matrix
  int col_tiles;
  long long tiles;
};

constexpr int mx_row_tiles(int rows, int rt) { return rows / rt + (rows % rt != 0); }

// Block-major scales are written in runs of 64 bytes where that leaves work for
// the chip (128 matrices of 768 x 2048 quantized: 82 us, in runs of 8 bytes 104; 4
// of them, 384 tiles of 64 rows: equal).
constexpr MxConvertPlan mx_convert_plan(int batch, int rows, int cols, bool block_major) {
  const int col_tiles = cols / kMxTileCols + (cols % kMxTileCols != 0);
  const int rt = block_major && (long long)batch * mx_row_tiles(rows, 64) * col_tiles >= 1024 ? 64 : 8;
  const int row_tiles = mx_row_tiles(rows, rt);
  return MxConvertPlan{rt, row_tiles, col_tiles, (long long)batch * row_tiles * col_tiles};
}

}  // namespace moe

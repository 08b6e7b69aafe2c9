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

}  // namespace moe

// Which kernels the router-training calls run, as rules on sizes and types:
// host code without a GPU header, so that a test without a GPU can ask it
// which variants a list of cases reaches.
#pragma once
#include <algorithm>
#include <cmath>

namespace moe {

// ---- row kernels (balance.hip)

// A row of E logits on L lanes: lane g holds elements (c L + g) V + v,
// c < C, v < V (V = 4: 16-byte loads, E a multiple of 4).
struct RowGeom {
  int V, L, C;
};
constexpr int kRowWave = 64;            // lanes of a wave
constexpr int kBalanceThreads = 512;    // workgroup of the balance loss
constexpr int kGateThreads = 256;       // and of the gradient
constexpr int kMaxRowBlocks = 512;
constexpr int kMaxGradBlocks = 512;
constexpr int kSoloPasses = 4;

constexpr RowGeom row_geom(int E) {
  if (E % 4 == 0)
    return E <= 4     ? RowGeom{4, 1, 1}
           : E <= 8   ? RowGeom{4, 2, 1}
           : E <= 16  ? RowGeom{4, 4, 1}
           : E <= 32  ? RowGeom{4, 4, 2}
           : E <= 64  ? RowGeom{4, 4, 4}
           : E <= 128 ? RowGeom{4, 8, 4}
           : E <= 256 ? RowGeom{4, 16, 4}
                      : RowGeom{4, 32, 4};
  return E <= 4     ? RowGeom{1, 4, 1}
         : E <= 16  ? RowGeom{1, 16, 1}
         : E <= 32  ? RowGeom{1, 16, 2}
         : E <= 64  ? RowGeom{1, 16, 4}
         : E <= 128 ? RowGeom{1, 16, 8}
         : E <= 256 ? RowGeom{1, 16, 16}
                    : RowGeom{1, 32, 16};
}

// The row shapes for few rows: more lanes a row, so that the rows spread over
// more compute units and a lane stores less.
constexpr RowGeom wide_row_geom(int E) {
  if (E <= 16) return row_geom(E);
  if (E % 4 == 0)
    return E <= 32    ? RowGeom{4, 8, 1}
           : E <= 64  ? RowGeom{4, 16, 1}
           : E <= 128 ? RowGeom{4, 32, 1}
           : E <= 256 ? RowGeom{4, 64, 1}
                      : RowGeom{4, 64, 2};
  return E <= 32    ? RowGeom{1, 32, 1}
         : E <= 64  ? RowGeom{1, 64, 1}
         : E <= 128 ? RowGeom{1, 64, 2}
         : E <= 256 ? RowGeom{1, 64, 4}
                    : RowGeom{1, 64, 8};
}

// Rows that a workgroup passes over at a time.
constexpr long long pass_rows(RowGeom g, int threads) { return threads / g.L; }

// Workgroups of a row kernel that passes over `pass` rows at a time: whole
// passes, as many workgroups as there are passes up to `most`.
inline int row_blocks(long long T, long long pass, int most, long long* rows_per_block) {
  const long long passes = std::max<long long>((T + pass - 1) / pass, 1);
  const long long each = (passes + most - 1) / most;
  *rows_per_block = each * pass;
  return (int)((passes + each - 1) / each);
}

// The balance loss: up to four passes one workgroup makes them all, in one
// launch (256 tokens of 128, a call among others: 8.4 us, in two kernels
// 11.5 us; at eight passes, 1000 tokens of 64, 12.8 against 11.6 us).  Below
// 64 passes the wide shape spreads the rows (the two kernels together: 1000
// tokens of 64, 10.5 us, wide 7.8 us; 2048 of 128, 10.3 and 8.9 us; 8192 of
// 128, which are 128 passes, 10.8 and 11.1 us).
constexpr RowGeom balance_geom(long long T, int E) {
  const long long pass = pass_rows(row_geom(E), kBalanceThreads);
  return T > kSoloPasses * pass && T < 64 * pass ? wide_row_geom(E) : row_geom(E);
}
inline int balance_blocks(long long T, int E, long long* rows) {
  long long pass = pass_rows(row_geom(E), kBalanceThreads);
  if (T <= kSoloPasses * pass) {
    *rows = kSoloPasses * pass;
    return 1;
  }
  pass = pass_rows(balance_geom(T, E), kBalanceThreads);
  // Rows of 16-byte loads: one workgroup a compute unit, with half the partial
  // sums to add (32768 tokens of 128: both kernels 13.4 us, 16.5 us with 512
  // workgroups; 131072 of 256: 34.8 and 35.4 us); of 4-byte loads two (65536
  // tokens of 511: 35.6 us, 39.2 us with 256).
  return row_blocks(T, pass, E % 4 == 0 ? 256 : kMaxRowBlocks, rows);
}

// The gradient's row shape: the wide one up to 512 passes of the other (2048
// tokens, E = 64: 7.6 us, wide 4.8 us; 8192, E = 128: 10.7 and 9.6 us; 16384,
// E = 256, 1024 passes: 16.8 and 21.2 us).
constexpr RowGeom gate_geom(long long T, int E) {
  return T < 512 * pass_rows(row_geom(E), kGateThreads) ? wide_row_geom(E) : row_geom(E);
}
inline int gate_blocks(long long T, int E, long long* rows) {
  return row_blocks(T, pass_rows(gate_geom(T, E), kGateThreads), kMaxGradBlocks, rows);
}

// ---- products of the router's backward pass (route_grad.hip)

// Experts in a row of dL as the products read it: the steps that the kernels
// of dx are made for.
constexpr int padded_experts(int E) { return E <= 32 ? 32 : (E + 63) / 64 * 64; }

// Tokens of a part of dW_r whose mask bits are held in LDS at a time.
constexpr int kSegment = 16384;

// Plan of the dW_r kernel: its tile of bc columns by be experts, and the parts
// of the token range.
struct DwPlan {
  int bc, be;
  int splits;
};

// One workgroup fits a compute unit.  A part costs the rounds of workgroups
// over the 256 compute units times (start and end of a workgroup, 4 us, plus
// its tokens at the measured time each), plus its partial sums, written and
// read at 4 TB/s.  The tall tiles have the better rate on many tokens of wide
// rows but need that many more parts to fill the chip.  Measured, 24 launches
// over 12 sets of tokens, twice: 16384 tokens of 7168, E = 256, 256 x 128 tiles
// 177 and 214 us, 128 x 128 200 and 222 us; E = 64, 256 x 64 60 us, 128 x 64 73
// to 75 us; E = 8, 256 x 32 43 us, 128 x 32 48 us (5.4 TB/s of x).  8192 tokens
// of 2048, E = 128: 256 x 128 23.5 us with 32 parts, 128 x 128 21 us with 16.
inline double dw_cost(long long T, int d, int E, int bc, int be, double ns_token, int splits) {
  const double tiles = (double)((d + bc - 1) / bc) * ((E + be - 1) / be);
  const double rounds = std::ceil(tiles * splits / 256.0);
  const double tokens = std::ceil((double)T / splits / 64.0) * 64.0;
  return rounds * (4000.0 + tokens * ns_token) +
         (splits > 1 ? 2.0 * splits * d * E * 4 / 4000.0 : 0.0);
}

inline DwPlan dw_plan(long long T, int d, int E, bool bf16) {
  DwPlan best{128, 32, 1};
  double cost = -1.0;
  auto offer = [&](int bc, int be, double ns_token) {
    // (the plan is made several times a call: few candidates)
    for (const int n : {1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 14, 16, 18, 20, 24, 28, 32, 40, 48, 64}) {
      if (n > 1 && (long long)n * 64 > T + 63) break;
      const double c = dw_cost(T, d, E, bc, be, ns_token, n);
      if (cost < 0 || c < cost) {
        cost = c;
        best = DwPlan{bc, be, n};
      }
    }
  };
  if (E <= 32) {
    offer(128, 32, bf16 ? 12.0 : 22.0);
    if (bf16) offer(256, 32, 22.0);
  } else if (E <= 64) {
    offer(128, 64, bf16 ? 17.0 : 30.0);
    if (bf16) offer(256, 64, 30.0);
  } else {
    offer(128, 128, bf16 ? 25.0 : 60.0);
    if (bf16) offer(256, 128, 44.0);
  }
  return best;
}
constexpr long long dw_tokens_per_split(long long T, int splits) {
  return ((T + splits - 1) / splits + 63) / 64 * 64;
}

// Few tokens for dx: workgroups of 512 columns and 64 tokens for less than
// half of the compute units.
constexpr bool few_tokens(long long T, int d) {
  return (long long)((d + 511) / 512) * ((T + 63) / 64) < 128;
}

// dW_r and dx of few tokens in one launch (a launch less, and the narrow grids
// side by side; float32 rows of more than 256 experts leave eight waves no
// registers).
inline bool products_in_one_launch(long long T, int d, int E, bool bf16) {
  return few_tokens(T, d) && dw_plan(T, d, E, bf16).bc == 128 &&
         (bf16 || padded_experts(E) <= 256);
}

}  // namespace moe

// Microscaled 4-bit floating point (OCP MX, MXFP4): conversion, and the expert
// network with activations and weights in 4 bits.
//
// "Serving MoE models with expert parallelism on 8xH200" (reviosa), section
// "Quantization choices", weighs 4-bit expert weights; here the activations
// are held in 4 bits too, so that the products run on the scaled matrix
// instruction (v_mfma_scale_f32_32x32x64_f8f6f4, four times the bf16 rate).
//
//   conversion:  block of 32:  X = floor(log2 max|v|) - 2 (clamped to -127..125),
//                code = the E2M1 value nearest to v / 2^X (ties to even, at most 6)
//   gate/up:     h[p] = Q(silu(A_p Wg_j) * (A_p Wu_j)),  A_p = x[sorted_slot[p] / k]
//   down:        y[p] = (h[p] Wd_j) * gate(p)
//
// Operand layout: lane l of an MFMA operand holds the 32 codes (16 bytes) of
// row l % 32 and 32-value block l / 32 of a 64-deep step, and that block's
// scale.  A step of 32 rows is therefore 1 KB of consecutive 16-byte pieces:
// the unit of the blocked weight layout and of the intermediate h, which lies
// in the workspace as [group of 32 rows][F / 64] units with scales
// [group][32 rows][F / 32].  Groups are counted per expert (a group never holds
// rows of two), so h needs no gather.  Weights
// are the A operand in the permuted row order (feature 16 (l / 32) + q in
// register q), so a lane's 16 results are 16 consecutive features of a token.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe_device.h"
#include "moe_internal.h"
#include "mx_plan.h"

namespace moe {
namespace {

constexpr int kNumXcd = 8;
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---- conversion

// The scale byte of a block whose largest magnitude has these float32 bits:
// X + 127 = exponent field - 2, at least 0; 127 for a block of zeros; 255
// (NaN) where the block holds an infinity or a NaN.  (The field of the largest
// finite magnitude, 254, gives 252.)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (amax_bits == 0) return 127;
  return e == 255 ? 255 : e < 2 ? 0 : e - 2;
}

// 2^(127 - byte): v times it is exact, or far below half of the smallest code.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == 255 ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 8 values -> 8 codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t mx_codes8(const float* v, float inv) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] * inv, v[1] * inv, 1.0f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] * inv, v[3] * inv, 1.0f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] * inv, v[5] * inv, 1.0f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] * inv, v[7] * inv, 1.0f, 3);
  return q;
}

// Tiles of kTileCols columns and `rt` rows (a multiple of 8): 32 threads of 8
// values for a row, 8 rows a pass.  Block-major scales pass through LDS, so
// that they are written and read in runs of rt bytes.
constexpr int kTileCols = kMxTileCols;

struct ConvertArgs {
  const void* src;
  void* dst;
  uint8_t* codes;
  uint8_t* scales;
  int rows, cols, rt;
  int row_tiles, col_tiles;
  long long tiles;
};

struct ConvertTile {
  long long row0;  // first row of the batch element, in rows of the whole array
  int r0, c0;      // first row and column of the tile
};

__device__ __forceinline__ ConvertTile convert_tile(const ConvertArgs& a, long long i) {
  const long long rt = i / a.col_tiles;
  return ConvertTile{rt / a.row_tiles * a.rows, (int)(rt % a.row_tiles) * a.rt,
                     (int)(i % a.col_tiles) * kTileCols};
}

// A tile of kPass passes is loaded whole before its first values are converted.
// Arrays of many tiles (kPass 8) are more than a cache holds: their values pass
// by it.  402 MB of bfloat16 with block-major scales, 509 MB in all, quantized:
// pass by pass 122 us, all loads first 121, and past the cache 84 (6.1 TB/s);
// dequantized 97, stores past the cache 74 (6.9 TB/s).
template <bool kBF16, bool kBlockMajor, int kPass>
__global__ __launch_bounds__(256) void mx_quantize_kernel(ConvertArgs a) {
  constexpr int kRows = 8 * kPass;
  __shared__ uint8_t lds[kBlockMajor ? (kTileCols / 32) * kRows : 1];
  const int cq = threadIdx.x % 32, rr = threadIdx.x / 32;
  for (long long i = blockIdx.x; i < a.tiles; i += gridDim.x) {
    const ConvertTile t = convert_tile(a, i);
    const int c = t.c0 + cq * 8;
    const long long at0 = (t.row0 + t.r0 + rr) * a.cols + c;
    u32x4_t raw[kPass][kBF16 ? 1 : 2];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int r = t.r0 + rr + 8 * p;
#pragma unroll
      for (int h = 0; h < (kBF16 ? 1 : 2); ++h) raw[p][h] = u32x4_t{0, 0, 0, 0};
      if (r < a.rows && c < a.cols) {
        const u32x4_t* from = reinterpret_cast<const u32x4_t*>(
            static_cast<const unsigned char*>(a.src) + (at0 + (long long)(8 * p) * a.cols) * (kBF16 ? 2 : 4));
#pragma unroll
        for (int h = 0; h < (kBF16 ? 1 : 2); ++h) raw[p][h] = kPass > 1 ? __builtin_nontemporal_load(from + h) : from[h];
      }
    }
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int r = rr + 8 * p;
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if constexpr (kBF16) v[q] = __uint_as_float(q & 1 ? raw[p][0][q >> 1] & 0xffff0000u : raw[p][0][q >> 1] << 16);
        else v[q] = __uint_as_float(raw[p][q >> 2][q & 3]);
      }
      uint32_t top = 0;  // (as integers: a NaN is above an infinity, which is above the rest)
#pragma unroll
      for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[q]) & 0x7fffffffu);
      top = max(top, (uint32_t)__shfl_xor((int)top, 1, kWave));
      top = max(top, (uint32_t)__shfl_xor((int)top, 2, kWave));
      const uint32_t byte = mx_scale_byte(top);
      if (t.r0 + r < a.rows && c < a.cols) {
        const long long at = at0 + (long long)(8 * p) * a.cols;
        const uint32_t q = byte == 255 ? 0 : mx_codes8(v, mx_inverse(byte));
        *reinterpret_cast<uint32_t*>(a.codes + at / 2) = q;
        if (cq % 4 == 0) {
          if constexpr (kBlockMajor) lds[(cq / 4) * kRows + r] = (uint8_t)byte;
          else a.scales[at / 32] = (uint8_t)byte;
        }
      }
    }
    if constexpr (kBlockMajor) {
      __syncthreads();
      const int n = min(kRows, a.rows - t.r0), kb0 = t.c0 / 32;
      const int kbs = min(kTileCols / 32, a.cols / 32 - kb0);
      for (int j = threadIdx.x; j < kbs * kRows; j += 256) {
        const int kb = j / kRows, r = j % kRows;
        if (r < n)
          a.scales[t.row0 * (a.cols / 32) + (long long)(kb0 + kb) * a.rows + t.r0 + r] =
              lds[kb * kRows + r];
      }
      __syncthreads();
    }
  }
}

template <bool kBF16, bool kBlockMajor, int kPass>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(ConvertArgs a) {
  constexpr int kRows = 8 * kPass;
  __shared__ uint8_t lds[kBlockMajor ? (kTileCols / 32) * kRows : 1];
  const int cq = threadIdx.x % 32, rr = threadIdx.x / 32;
  for (long long i = blockIdx.x; i < a.tiles; i += gridDim.x) {
    const ConvertTile t = convert_tile(a, i);
    const int c = t.c0 + cq * 8;
    const long long at0 = (t.row0 + t.r0 + rr) * a.cols + c;
    uint32_t codes[kPass];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      codes[p] = 0;
      if (t.r0 + rr + 8 * p < a.rows && c < a.cols)
        codes[p] = *reinterpret_cast<const uint32_t*>(a.codes + (at0 + (long long)(8 * p) * a.cols) / 2);
    }
    if constexpr (kBlockMajor) {
      const int n = min(kRows, a.rows - t.r0), kb0 = t.c0 / 32;
      const int kbs = min(kTileCols / 32, a.cols / 32 - kb0);
      for (int j = threadIdx.x; j < kbs * kRows; j += 256) {
        const int kb = j / kRows, r = j % kRows;
        if (r < n)
          lds[kb * kRows + r] =
              a.scales[t.row0 * (a.cols / 32) + (long long)(kb0 + kb) * a.rows + t.r0 + r];
      }
      __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int r = rr + 8 * p;
      if (t.r0 + r >= a.rows || c >= a.cols) continue;
      const long long at = at0 + (long long)(8 * p) * a.cols;
      uint32_t byte;
      if constexpr (kBlockMajor) byte = lds[(cq / 4) * kRows + r];
      else byte = a.scales[at / 32];
      u32x4_t w = __builtin_bit_cast(u32x4_t, e2m1x8_to_bf16x8(codes[p], e8m0_to_f32(byte)));
      if (byte == 255) w = u32x4_t{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
      if constexpr (kBF16) {
        u32x4_t* to = reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.dst) + at);
        if constexpr (kPass > 1) __builtin_nontemporal_store(w, to);
        else *to = w;
      } else {
        u32x4_t* to = reinterpret_cast<u32x4_t*>(static_cast<float*>(a.dst) + at);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t f = {w[2 * h] << 16, w[2 * h] & 0xffff0000u, w[2 * h + 1] << 16, w[2 * h + 1] & 0xffff0000u};
          if constexpr (kPass > 1) __builtin_nontemporal_store(f, to + h);
          else to[h] = f;
        }
      }
    }
    if constexpr (kBlockMajor) __syncthreads();
  }
}

// ---- the expert network

struct MxArgs {
  const uint8_t* A;            // gate/up: x codes [T][K / 2]; down: h units
  const uint8_t* AS;           // gate/up: x scales [T][K / 32]; down: h scales
  uint32_t a_bytes, as_bytes;  // gate/up
  const int32_t* sorted_slot;
  const int32_t* offsets;      // [El + 1]
  int k;
  const uint8_t* W0;           // gate or down codes
  const uint8_t* W1;           // up codes
  const uint8_t* S0;           // their scales [K / 32][Nout] per expert
  const uint8_t* S1;
  const float* topk_w;         // down: gates or null
  uint16_t* y;                 // down: [S][Nout]
  uint8_t* h;                  // gate/up: h units
  uint8_t* hs;                 // gate/up: h scales
  int El, S;
  int max_groups;              // that h has room for
  int K, Nout;
  int blocked;
};

// Raw buffer resource over `bytes` bytes at `base` (wave-uniform): loads at or
// past `bytes` read zeros instead of faulting.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// Segment bounds as the caller gives them, held inside [0, S], so that rows of y
// are in bounds whatever they are (bounds that do not ascend: group_table).
__device__ __forceinline__ int bound(const MxArgs& a, int e) {
  return max(0, min(a.offsets[e], a.S));
}

// The same for a wave-uniform e, by a scalar load: one through the vector
// pipe would be waited for behind every load in flight.
__device__ __forceinline__ int uniform_bound(const MxArgs& a, int e) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto* p = (const __attribute__((address_space(4))) int32_t*)(a.offsets + __builtin_amdgcn_readfirstlane(e));
  return max(0, min((int)*p, a.S));
#else
  return bound(a, e);
#endif
}

// groups[e] = number of groups of 32 rows of experts before e (groups[El]: of
// all), each expert's counted up to a multiple of kUnit, by one workgroup of
// kThreads threads.  Never more than the workspace holds (as long as the segments
// do not overlap, it holds all; the sums stop there, so they cannot overflow).
template <int kThreads, int kUnit>
__device__ __forceinline__ void group_table(const MxArgs& a, int* groups) {
  constexpr int kPer = kMaxExperts / kThreads;
  __shared__ int waves[kThreads / kWave];
  const int limit = a.max_groups / kUnit * kUnit;
  int n[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    n[i] = e < a.El ? mx_groups(max(0, bound(a, e + 1) - bound(a, e)), kUnit) : 0;
    sum = mx_add_groups(sum, n[i], limit);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(incl, o, kWave);
    if (lane_id() >= o) incl = mx_add_groups(incl, v, limit);
  }
  if (lane_id() == kWave - 1) waves[threadIdx.x / kWave] = incl;
  int before = __shfl_up(incl, 1, kWave);
  if (lane_id() == 0) before = 0;
  __syncthreads();
  for (int w = 0; w < (int)threadIdx.x / kWave; ++w) before = mx_add_groups(before, waves[w], limit);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e <= a.El) groups[e] = before;
    before = mx_add_groups(before, n[i], limit);
  }
  if (a.El == kMaxExperts && threadIdx.x == kThreads - 1) groups[kMaxExperts] = before;
  __syncthreads();
}

// The expert that holds group `g` (the last e with groups[e] <= g).
__device__ __forceinline__ int expert_of(const int* groups, int El, int g) {
  int lo = 0, hi = El - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (groups[mid] <= g) lo = mid;
    else hi = mid - 1;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// permuted weight row of MFMA row r of a 32-row block
__device__ __forceinline__ int feat(int r) {
  return (((r >> 2) & 1) << 4) | (((r >> 3) & 3) << 2) | (r & 3);
}

// The product of 32 x 64 by 64 x 32; byte kByte of sb is b's scale, byte 0 of sa a's.
template <int kByte>
__device__ __forceinline__ f32x16_t mfma_mx(u32x4_t a, u32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
#if defined(__HIP_DEVICE_COMPILE__)
  const i32x8_t av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, kByte, (int)sb);
#else
  (void)a;
  (void)b;
  (void)sa;
  (void)sb;
  return c;
#endif
}

// How a block of 32 rows of a stage (128 K values: 64 bytes, 4 chunks of 16)
// lies in LDS, and what lane l moves there as half block h.  Consecutive lanes
// write consecutive places, and four of them have to read 64 consecutive bytes:
// 16 rows' first chunks, then their second ones and so on pass the cache at
// 9.7 TB/s on all compute units, 64 bytes of one row after the other at 34.
// From units: lane l takes row 16 h + l % 16, chunk l / 16 (half chunk % 2 of
// unit chunk / 2); offset in the two units of the stage, and a chunk's place.
__device__ __forceinline__ uint32_t unit_offset(int h, int l) {
  const int c = l >> 4;
  return (c >> 1) * 1024 + ((c & 1) * 32 + 16 * h + (l & 15)) * 16;
}

__device__ __forceinline__ int unit_place(int row, int chunk) {
  return (row >> 4) * 1024 + chunk * 256 + (row & 15) * 16;
}

// From rows: lane l takes row 16 h + l / 4.  The chunks of a row change places,
// so that any 8 or 16 consecutive rows' places of one chunk are in different banks.
__device__ __forceinline__ int row_turn(int row) {
  return ((row >> 1) & 2) | (((row >> 1) ^ (row >> 3)) & 1);
}

__device__ __forceinline__ uint32_t row_chunk(int l) { return 16u * ((l & 3) ^ row_turn(l >> 2)); }

__device__ __forceinline__ int row_place(int row, int chunk) {
  return row * 64 + ((chunk ^ row_turn(row & 15)) << 4);
}

// Epilogue of a gate/up pair: 16 consecutive features of token row r of group
// `grp` (lane half g), feature block fb: silu(gate) * up in float32, converted
// to MXFP4 with the other half's 16 features.  Returns the scale byte.
__device__ __forceinline__ uint32_t store_h(const MxArgs& a, const f32x16_t& gate, const f32x16_t& up,
                                            int grp, int fb, int l) {
  float h[16];
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    h[q] = silu_f32(gate[q]) * up[q];
    top = max(top, __float_as_uint(h[q]) & 0x7fffffffu);
  }
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
  const uint32_t byte = mx_scale_byte(top);
  const float inv = mx_inverse(byte);
  u32x2_t q = {mx_codes8(h, inv), mx_codes8(h + 8, inv)};
  if (byte == 255) q = u32x2_t{0, 0};
  const int r = l & 31, g = l >> 5;
  *reinterpret_cast<u32x2_t*>(a.h + ((long long)grp * (a.Nout / 64) + (fb >> 1)) * 1024 +
                              ((fb & 1) * 32 + r) * 16 + 8 * g) = q;
  return byte;
}

__device__ __forceinline__ uint8_t* h_scale(const MxArgs& a, int grp, int r, int fb) {
  return a.hs + ((long long)grp * 32 + r) * (a.Nout / 32) + fb;
}

// Epilogue of a down block: 16 consecutive columns of row p.
__device__ __forceinline__ void store_y(const MxArgs& a, const f32x16_t& v, int p, int col, float gw) {
  uint16_t* o = a.y + (long long)p * a.Nout + col;
  float h[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) h[q] = v[q] * gw;
  *reinterpret_cast<u32x4_t*>(o) = u32x4_t{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3]),
                                           bf16_pair(h[4], h[5]), bf16_pair(h[6], h[7])};
  *reinterpret_cast<u32x4_t*>(o + 8) = u32x4_t{bf16_pair(h[8], h[9]), bf16_pair(h[10], h[11]),
                                               bf16_pair(h[12], h[13]), bf16_pair(h[14], h[15])};
}

// -- few rows per expert, blocked weights: streamed by each wave into registers.
// An item is a group of 32 rows and kNB weight blocks of 32 rows (gate/up: two
// gate blocks and the up blocks of the same features); the four waves of a
// workgroup take a quarter of K each and add their results through LDS, so
// that a handful of experts still fills the chip.  64 tokens of the Qwen3 shape:
// gate/up 38.5 us for 214 MB (5.6 TB/s), down 24.8 us for 107 MB, of which 6 us
// are the joining of the quarters (three steps of K each).  Not bound by loads in flight: two, three or
// four steps a wave take the same, six more (43 and 32 us).  A wave keeps kD steps of
// 64 K values in flight; nothing passes LDS before the results.
constexpr int kNB = 4;
constexpr int kD = 3;

template <bool kGateUp>
__global__ __launch_bounds__(256, 2) void mx_stream_kernel(MxArgs a) {
  constexpr int H = kGateUp ? 2 : 4;  // output blocks of an item
  __shared__ int groups[kMaxExperts + 1];
  __shared__ f32x4_t red[4][kNB][4][kWave];  // [wave][block][registers 4q ..][lane]
  group_table<256, 1>(a, groups);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l = lane_id(), g = l >> 5, r = l & 31;
  const int nS = a.K / 64, ngrp = a.Nout / (32 * H);
  const int n_items = groups[a.El] * ngrp;
  const int per_xcd = (n_items + kNumXcd - 1) / kNumXcd;
  const int xcd = blockIdx.x % kNumXcd, slots = gridDim.x / kNumXcd;
  const int end = min(n_items, (xcd + 1) * per_xcd);
  const int s0 = nS * wave / 4, s1 = nS * (wave + 1) / 4;
  const uint32_t wrow = (uint32_t)a.K / 2, wmat = (uint32_t)a.Nout * wrow;
  const uint32_t smat = (uint32_t)(a.K / 32) * a.Nout;
  // Scales of a step: a lane loads four columns of a K block (down: 128 columns in
  // a load, gate/up: 64 a matrix), and each block's are fetched from the lane that
  // holds them.
  const uint32_t voffS = kGateUp ? (uint32_t)((l >> 4) & 1) * a.Nout + 4u * (l & 15)
                                 : (uint32_t)g * a.Nout + 4u * r;
  const int from = 4 * (g * (8 * H) + feat(r) / 4), shift = 8 * (r & 3);
  struct Item {
    int e, nb, grp, row0, rend, slot;  // feature group, row group, rows; slot of the lane's row
  };
  auto decode = [&](int it) {
    Item i;
    i.e = expert_of(groups, a.El, it / ngrp);
    const int m_tiles = __builtin_amdgcn_readfirstlane(groups[i.e + 1] - groups[i.e]);
    const int in = it - groups[i.e] * ngrp;
    i.nb = __builtin_amdgcn_readfirstlane(in / m_tiles);
    const int mt = __builtin_amdgcn_readfirstlane(in % m_tiles);
    i.grp = __builtin_amdgcn_readfirstlane(groups[i.e]) + mt;
    i.row0 = uniform_bound(a, i.e) + mt * 32;
    i.rend = uniform_bound(a, i.e + 1);
    i.slot = a.sorted_slot[min(i.row0 + r, i.rend - 1)];
    return i;
  };
  u32x4_t wb[kD][kNB], tb[kD];
  uint32_t ws[kD][kGateUp ? 2 : 1];
  uint8_t ts[kD];
  // Step s of item i into place d.  A step that the wave does not have (or an
  // item that is not there) reads zeros, without a branch: the number of loads
  // in flight is then the same on every path, and the waits for them are exact.
  auto issue = [&](const Item& i, bool there, int s, int d) {
    const bool on = there && s < s1;
    const uint32_t wn = on ? wmat : 0, sn = on ? smat : 0;
    const __amdgpu_buffer_rsrc_t rW0 = rsrc(a.W0 + (size_t)i.e * wmat, wn);
    const __amdgpu_buffer_rsrc_t rW1 = kGateUp ? rsrc(a.W1 + (size_t)i.e * wmat, wn) : rW0;
    const __amdgpu_buffer_rsrc_t rS0 = rsrc(a.S0 + (size_t)i.e * smat, sn);
    const __amdgpu_buffer_rsrc_t rS1 = kGateUp ? rsrc(a.S1 + (size_t)i.e * smat, sn) : rS0;
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
      const int fb = i.nb * H + n % H;
      wb[d][n] = __builtin_amdgcn_raw_buffer_load_b128(n >= H ? rW1 : rW0, 16u * l,
                                                       (uint32_t)fb * 32u * wrow + s * 1024u, 2);
    }
    const uint32_t at = (uint32_t)(2 * s) * a.Nout + i.nb * (32u * H);
    ws[d][0] = __builtin_amdgcn_raw_buffer_load_b32(rS0, voffS, at, 0);
    if constexpr (kGateUp) ws[d][1] = __builtin_amdgcn_raw_buffer_load_b32(rS1, voffS, at, 0);
    if constexpr (kGateUp) {
      const uint32_t t = (uint32_t)i.slot / (uint32_t)a.k;
      tb[d] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(a.A, on ? a.a_bytes : 0), t * wrow + 16u * g, s * 32u, 0);
      ts[d] = __builtin_amdgcn_raw_buffer_load_b8(rsrc(a.AS, on ? a.as_bytes : 0), t * (uint32_t)(a.K / 32) + g,
                                                  2u * s, 0);
    } else {
      tb[d] = __builtin_amdgcn_raw_buffer_load_b128(
          rsrc(a.A + (long long)i.grp * nS * 1024, on ? (uint32_t)nS * 1024u : 0), 16u * l, s * 1024u, 0);
      ts[d] = __builtin_amdgcn_raw_buffer_load_b8(
          rsrc(a.AS + (long long)i.grp * nS * 64, on ? (uint32_t)nS * 64u : 0), (uint32_t)(r * 2 * nS) + g, 2u * s, 0);
    }
  };
  auto multiply = [&](f32x16_t(&acc)[kNB], int d) {
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
      const int v = __builtin_amdgcn_ds_bpermute(from + 32 * (n % H), (int)ws[d][n / H]);
      acc[n] = mfma_mx<0>(wb[d][n], tb[d], acc[n], (uint32_t)v >> shift, ts[d]);
    }
  };
  const __amdgpu_buffer_rsrc_t rG = rsrc(a.topk_w, !kGateUp && a.topk_w ? (uint32_t)a.S * 4u : 0);
  auto gate_of = [&](const Item& i) { return __builtin_amdgcn_raw_buffer_load_b32(rG, 4u * i.slot, 0, 0); };
  int it = xcd * per_xcd + (int)blockIdx.x / kNumXcd;
  if (it >= end) return;
  auto at_most = [&](int i) { return i < end ? i : it; };
  Item cur = decode(it), next = decode(at_most(it + slots));
  uint32_t gw = gate_of(cur);
#pragma unroll
  for (int d = 0; d < kD; ++d) {
    issue(cur, true, s0 + d, d);
    __builtin_amdgcn_sched_barrier(0);
  }
  while (true) {
    const bool more = it + slots < end;
    // (two items ahead: a wait for its slots waits for nothing later)
    const Item third = decode(at_most(it + 2 * slots));
    f32x16_t acc[kNB];
#pragma unroll
    for (int n = 0; n < kNB; ++n) acc[n] = f32x16_t{};
    int s = s0;
    for (; s + kD < s1; s += kD) {
#pragma unroll
      for (int d = 0; d < kD; ++d) {
        multiply(acc, d);
        __builtin_amdgcn_sched_barrier(0);
        issue(cur, true, s + d + kD, d);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // the next item's first steps fly while this one's results are joined
    const uint32_t next_gw = gate_of(next);
#pragma unroll
    for (int d = 0; d < kD; ++d) {
      multiply(acc, d);
      __builtin_amdgcn_sched_barrier(0);
      issue(next, more, s0 + d, d);
      __builtin_amdgcn_sched_barrier(0);
    }
    const int row0 = cur.row0, rend = cur.rend, nb = cur.nb, grp = cur.grp;
    // results of block n meet in wave n (gate/up: of pair n in wave n)
    __syncthreads();  // the last item's sums have been read
#pragma unroll
    for (int n = 0; n < kNB; ++n) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[wave][n][q][l] = f32x4_t{acc[n][4 * q], acc[n][4 * q + 1], acc[n][4 * q + 2], acc[n][4 * q + 3]};
    }
    __syncthreads();
    if (wave < H) {
      f32x16_t sum[kNB / H];
#pragma unroll
      for (int i = 0; i < kNB / H; ++i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4_t v = red[0][i * H + wave][q][l];
#pragma unroll
          for (int w = 1; w < 4; ++w) v += red[w][i * H + wave][q][l];
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[i][4 * q + j] = v[j];
        }
      }
      const int fb = nb * H + wave;
      if constexpr (kGateUp) {
        const uint32_t byte = store_h(a, sum[0], sum[1], grp, fb, l);
        if (g == 0) *h_scale(a, grp, r, fb) = (uint8_t)byte;
      } else if (row0 + r < rend) {
        store_y(a, sum[0], row0 + r, fb * 32 + 16 * g, a.topk_w ? __uint_as_float(gw) : 1.0f);
      }
    }
    if (!more) break;
    it += slots;
    cur = next;
    next = third;
    gw = next_gw;
  }
}

// -- many rows per expert: tiles of 128 rows x 256 weight rows (gate/up: 128
// gate and the up rows of the same features) through a ring of LDS stages of
// 128 K values, filled by LDS-DMA.  Four waves of 64 x 128; two workgroups a
// CU, so that the conversion of one's results runs beside the other's products.
// A DMA instruction takes 64 bytes of each of 16 rows (the cache counts lines,
// not bytes: 32 bytes of 32 rows made it the bottleneck).  The rows' scales come
// 16 bytes (four stages) at a time, for the same reason, and are read into
// registers.
// 8192 tokens of the Qwen3 shape: gate/up 145 us (2.84 PFLOP/s), down 111 us (1.86,
// beside 268 MB of results).  The matrix instructions alone, nothing else running,
// reach 6.5 PFLOP/s here (the clock falls under them); a wave's stage takes 1800
// cycles or more, 1024 of them the matrix cores', an eighth of the tiles' rows
// are padding, and the results' conversion takes 17 us of gate/up and, with its
// stores, 40 of down.
constexpr int kBM = 4;        // groups of 32 rows of a tile
constexpr int kStages = 3;
constexpr int kBlock = 2048;  // of 32 rows
constexpr int kStageW = kBM * kBlock;              // weight rows behind the tile's rows
constexpr int kStageWS = kStageW + 8 * kBlock;     // their scales [4 K blocks][256]
constexpr int kStage = kStageWS + 4 * 256;
constexpr int kRowScales = kStages * kStage;       // [2][128 rows][16]
constexpr int kTileTable = kRowScales + 2 * kBM * 512;  // groups before each expert, El + 1
// (up to 251 experts two workgroups fit a compute unit, with more of them one)
inline int tile_lds(int El) { return kTileTable + (El + 1) * 4; }

// One LDS-DMA load per active lane: lane i's 16 (4) bytes, from voff + soff in
// the buffer (from), land at lds + 16 i (4 i); lds is wave-uniform.
__device__ __forceinline__ void lds_dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, unsigned char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
#else
  (void)r, (void)voff, (void)soff, (void)lds;
#endif
}

__device__ __forceinline__ void lds_dma4(const uint8_t* from, unsigned char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)const_cast<uint8_t*>(from),
                                   (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
#else
  (void)from, (void)lds;
#endif
}

// At most N vector-memory operations of this wave are outstanding, its LDS
// reads have returned, and then so for the whole workgroup.  (No fence, which
// would wait for every load in flight.)
template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The ring runs on across items: the next item's first stages and addresses are
// under way before the present one's results are converted and stored.  A stage is
// two steps of 64 K values: the operands of one are read while the other's
// products run, across stages and items, so that a wave's matrix instructions
// do not stand behind its reads, and the loads of the stage after next go out
// between them.  (Reads and loads in front of the products: 158 us for the
// Qwen3 prefill gate/up.)
template <bool kGateUp>
__global__ __launch_bounds__(256, 2) void mx_tile_kernel(MxArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  int* groups = reinterpret_cast<int*>(lds + kTileTable);
  group_table<256, kBM>(a, groups);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l = lane_id(), g = l >> 5, r = l & 31;
  const int wm = wave >> 1, wn = wave & 1;
  const int nK = a.K / 128, nS = max(nK, 2);  // (a lone stage is followed by one of zeros)
  const int cols = kGateUp ? 128 : 256;  // output columns of a tile
  const int ntn = (a.Nout + cols - 1) / cols;
  const uint32_t wrow = (uint32_t)a.K / 2, wmat = (uint32_t)a.Nout * wrow;
  const uint32_t smat = (uint32_t)(a.K / 32) * a.Nout;
  const uint32_t stepW = a.blocked ? 2048u : 64u;  // of a stage
  uint32_t voffW[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    voffW[h] = a.blocked ? unit_offset(h, l) : (uint32_t)feat(16 * h + (l >> 2)) * wrow + row_chunk(l);
  const int n_items = groups[a.El] / kBM * ntn;
  const int per_xcd = (n_items + kNumXcd - 1) / kNumXcd;
  const int xcd = blockIdx.x % kNumXcd, slots = gridDim.x / kNumXcd;
  const int end = min(n_items, (xcd + 1) * per_xcd);
  int it = xcd * per_xcd + (int)blockIdx.x / kNumXcd;
  if (it >= end) return;

  // An item: tile nt of the columns, rows row0 .. rend - 1 (up to 128) in groups
  // g0 .. of expert e.  Found from the one before, `in` being its number among
  // its expert's items (M tiles fastest).
  struct Item {
    int e, in, nt, g0, row0, rend;
  };
  auto place = [&](int e, int in) {
    Item t;
    int first = __builtin_amdgcn_readfirstlane(groups[e]);
    int m_tiles = __builtin_amdgcn_readfirstlane(groups[e + 1]) / kBM - first / kBM;
    while (in >= m_tiles * ntn) {
      in -= m_tiles * ntn;
      ++e;
      first = __builtin_amdgcn_readfirstlane(groups[e]);
      m_tiles = __builtin_amdgcn_readfirstlane(groups[e + 1]) / kBM - first / kBM;
    }
    t.e = e;
    t.in = in;
    t.nt = __builtin_amdgcn_readfirstlane(in / m_tiles);
    const int mt = in - t.nt * m_tiles;
    t.g0 = first + mt * kBM;
    t.row0 = uniform_bound(a, e) + mt * kBM * 32;
    t.rend = uniform_bound(a, e + 1);
    return t;
  };
  // This lane's slots of an item: gate/up: of the two rows that it moves, row
  // l / 4 of a half block; down: of the two rows whose results it has.
  auto load_slots = [&](const Item& t, int (&slot)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = kGateUp ? wave * 32 + 16 * h + (l >> 2) : (wm * 2 + h) * 32 + r;
      slot[h] = a.sorted_slot[min(t.row0 + row, t.rend - 1)];
    }
  };

  // This wave's LDS-DMA of an item: A block `wave`, W blocks wave and wave + 4,
  // the scales of A block `wave`, and K block `wave` of the weights' scales.
  __amdgpu_buffer_rsrc_t rA, rAS, rW0, rW1;
  uint32_t voffA[2], voffAS, sW0, sW1;
  const uint8_t* ps;  // this lane's four scales of stage 0
  constexpr uint32_t stepA = kGateUp ? 64 : 2048;
  auto aim = [&](const Item& t, const int (&slot)[2], bool there) {
    const uint32_t on = there ? ~0u : 0u;  // (of the buffers' sizes)
    if constexpr (kGateUp) {
      uint32_t tok[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        tok[h] = (uint32_t)slot[h] / (uint32_t)a.k;
        voffA[h] = tok[h] * wrow + row_chunk(l);
      }
      rA = rsrc(a.A, a.a_bytes & on);
      rAS = rsrc(a.AS, a.as_bytes & on);
      // lanes 0 .. 31: their rows, which other lanes move
      const uint32_t lo = __shfl((int)tok[0], 4 * (l & 15), kWave), hi = __shfl((int)tok[1], 4 * (l & 15), kWave);
      voffAS = (l & 16 ? hi : lo) * (uint32_t)(a.K / 32);
    } else {
      // (all kBM groups of the tile exist; rows behind the segment hold whatever
      // was there and only reach results that are not stored)
      rA = rsrc(a.A + (long long)(t.g0 + wave) * (2 * nK) * 1024, (uint32_t)nK * 2048u & on);
      rAS = rsrc(a.AS + (long long)(t.g0 + wave) * (4 * nK) * 32, (uint32_t)nK * 128u & on);
#pragma unroll
      for (int h = 0; h < 2; ++h) voffA[h] = unit_offset(h, l);
      voffAS = (uint32_t)r * (4 * nK);
    }
    const uint32_t f0 = (uint32_t)t.nt * cols;
    rW0 = rsrc(a.W0 + (size_t)t.e * wmat, wmat & on);
    rW1 = kGateUp ? rsrc(a.W1 + (size_t)t.e * wmat, wmat & on) : rW0;
    // (down, 128 columns left: the second half repeats the first and is not stored)
    sW0 = __builtin_amdgcn_readfirstlane((f0 + 32u * wave) * wrow);
    sW1 = __builtin_amdgcn_readfirstlane(kGateUp || f0 + 128u >= (uint32_t)a.Nout ? sW0 : sW0 + 128u * wrow);
    // scales of one K block: 4 rows a lane (gate/up: 32 lanes for either matrix).
    // These loads have no bounds of their own: columns behind the matrix repeat its
    // last ones, and the zeros behind a lone stage take that stage's (a row that
    // a NaN among them spoils is NaN already).
    const uint32_t f = kGateUp ? f0 + 4u * (l & 31) : min(f0 + 4u * l, (uint32_t)a.Nout - 4u);
    ps = (kGateUp && g ? a.S1 : a.S0) + (size_t)t.e * smat + (uint32_t)wave * a.Nout + f;
  };
  // this lane's operands in a stage
  const int first_w = wn * (kGateUp ? 2 : 4);
  int read_a[2], read_w[2];  // of either step
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    read_a[q] = wm * 2 * kBlock + (kGateUp ? row_place(r, 2 * q + g) : unit_place(r, 2 * q + g));
    read_w[q] = kStageW + first_w * kBlock + (a.blocked ? unit_place(r, 2 * q + g) : row_place(r, 2 * q + g));
  }
  const int read_ws = kStageWS + g * 256 + first_w * 32 + feat(r);
  int put = 0;  // the ring's next place
  // (an aim without memory writes zeros into places that no stage will be read
  // from, and keeps the number of loads in flight what the waits count on)
  constexpr int kIssued = 7;  // LDS-DMA instructions of a stage
  auto issue_one = [&](int s, int i) {
    unsigned char* st = lds + put * kStage;
    const int h = i & 1;
    if (i < 2) {
      lds_dma16(rA, voffA[h], (uint32_t)s * stepA, st + wave * kBlock + h * 1024);
    } else if (i < 4) {
      lds_dma16(rW0, voffW[h], sW0 + (uint32_t)s * stepW, st + kStageW + wave * kBlock + h * 1024);
    } else if (i < 6) {
      lds_dma16(rW1, voffW[h], sW1 + (uint32_t)s * stepW, st + kStageW + (wave + 4) * kBlock + h * 1024);
    } else {
      lds_dma4(ps + (uint32_t)(4 * min(s, nK - 1)) * a.Nout, st + kStageWS + wave * 256);
    }
    if (i == kIssued - 1) put = put == kStages - 1 ? 0 : put + 1;
  };
  // Row scales of stages s .. s + 3 (s a multiple of 4) into the two buffers in
  // turn.  (Behind the row's end come others' or zeros, not used.)
  int put_rs = 0, get_rs = 1;
  auto issue_row_scales = [&](int s) {
    if (g == 0) lds_dma16(rAS, voffAS, 4u * s, lds + kRowScales + put_rs * (kBM * 512) + wave * 512);
    put_rs ^= 1;
  };

  static_assert(kStages == 3, "a place for the stage being read and two ahead");
  const int e0 = expert_of(groups, a.El, it / ntn * kBM);
  Item cur = place(e0, it - groups[e0] / kBM * ntn);
  // (slots and gates are fetched an item ahead, and taken behind a wait that covers
  // them: a wait for their own sake would be one for the whole ring)
  int slot[2] = {0, 0};
  float gw[2] = {1.0f, 1.0f}, gn[2] = {1.0f, 1.0f};
  const bool use_slots = kGateUp || a.topk_w;
  auto load_gates = [&](float (&w)[2]) {
    if (kGateUp || !a.topk_w) return;
    // (slots behind the last kept one may be anything)
    w[0] = a.topk_w[min((uint32_t)slot[0], (uint32_t)a.S - 1)];
    w[1] = a.topk_w[min((uint32_t)slot[1], (uint32_t)a.S - 1)];
  };
  auto after = [&](const Item& t, bool there) { return there ? place(t.e, t.in + slots) : t; };
  if (use_slots) load_slots(cur, slot);
  aim(cur, slot, true);
  load_gates(gw);
  Item next = after(cur, it + slots < end);
  if (use_slots) load_slots(next, slot);
  issue_row_scales(0);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (i == nK) aim(cur, slot, false);
#pragma unroll
    for (int j = 0; j < kIssued; ++j) issue_one(i, j);
  }
  int get = 0;
  uint32_t rs[2];  // row scales of the stage
  uint32_t ws[2][4];
  u32x4_t av[2][2], wv[2][4];
  auto read = [&](int q) {
    const unsigned char* st = lds + get * kStage;
#pragma unroll
    for (int m = 0; m < 2; ++m) av[q][m] = *reinterpret_cast<const u32x4_t*>(st + read_a[q] + m * kBlock);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int b = kGateUp ? (n >> 1) * 4 + (n & 1) : n;  // of the wave's weight blocks
      wv[q][n] = *reinterpret_cast<const u32x4_t*>(st + read_w[q] + b * kBlock);
      ws[q][n] = st[read_ws + q * 512 + b * 32];
    }
  };
  // The next stage is there for every wave, with all that was asked for before the
  // newest stage, and every wave has read the present one; its first operands.
  auto arrive = [&](int s) {
    stage_barrier<kIssued>();
    asm volatile("" : "+v"(slot[0]), "+v"(slot[1]), "+v"(gw[0]), "+v"(gw[1]), "+v"(gn[0]), "+v"(gn[1]));
    if (s % 4 == 0) get_rs ^= 1;
#pragma unroll
    for (int m = 0; m < 2; ++m)
      rs[m] = *reinterpret_cast<const uint32_t*>(lds + kRowScales + get_rs * (kBM * 512) + ((wm * 2 + m) * 32 + r) * 16 + 4 * (s % 4));
    read(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  arrive(0);
  for (;;) {
    const bool more = it + slots < end;
    f32x16_t acc[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[m][n] = f32x16_t{};
    Item third = next;
    for (int s = 0; s < nS; ++s) {
      // Every wave has read the stage before this one, whose place the new one takes.
      int at = s + 2;
      if (at >= nS) at -= nS;
      // Row scales four stages at a time (the next item's in the last stage), so late
      // that every wave has read the last of those whose place they take: a stage
      // back or more.
      if (at == 1 || (s % 4 == 1 && s + 3 < nK)) issue_row_scales(at == 1 ? 0 : s + 3);
      if (at == 0 || at == nK) {  // the next item's first stages follow (or zeros)
        aim(next, slot, more && at == 0);
        if (at == 0) {
          load_gates(gn);
          third = after(next, it + 2 * slots < end);
          if (use_slots) load_slots(third, slot);
        }
      }
      uint32_t as[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) as[m] = s < nK ? rs[m] >> (8 * g) : 0;
      read(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = i >> 1, m = i & 1;
        acc[m][n] = mfma_mx<0>(wv[0][n], av[0][m], acc[m][n], ws[0][n], as[m]);
        if (i < kIssued) {
          issue_one(at, i);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      get = get == kStages - 1 ? 0 : get + 1;
      arrive(s + 1 == nS ? 0 : s + 1);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m) acc[m][n] = mfma_mx<2>(wv[1][n], av[1][m], acc[m][n], ws[1][n], as[m]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int grp = cur.g0 + wm * 2 + m, p0 = cur.row0 + (wm * 2 + m) * 32;
      if (p0 >= cur.rend) continue;
      if constexpr (kGateUp) {
        const int fb = cur.nt * 4 + wn * 2;
        const uint32_t lo = store_h(a, acc[m][0], acc[m][2], grp, fb, l);
        const uint32_t hi = store_h(a, acc[m][1], acc[m][3], grp, fb + 1, l);
        if (g == 0) *reinterpret_cast<uint16_t*>(h_scale(a, grp, r, fb)) = (uint16_t)(lo | hi << 8);
      } else {
        // 32 rows x 64 columns at a time through LDS, so that a store takes whole
        // lines: the place of the stage that was read last, the part of it that
        // this wave alone fills (its weight blocks; 16-byte chunk c of row i at
        // c ^ i % 8).
        unsigned char* tmp = lds + put * kStage + kStageW + wave * kBlock;
#pragma unroll
        for (int n = 0; n < 4; n += 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = acc[m][n + b][q] * gw[m];
            unsigned char* row = tmp + (r >> 4) * (4 * kBlock) + (r & 15) * 128;
            const int c = b * 4 + g * 2;
            *reinterpret_cast<u32x4_t*>(row + ((c ^ (r & 7)) << 4)) =
                u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
            *reinterpret_cast<u32x4_t*>(row + (((c + 1) ^ (r & 7)) << 4)) =
                u32x4_t{bf16_pair(v[8], v[9]), bf16_pair(v[10], v[11]), bf16_pair(v[12], v[13]), bf16_pair(v[14], v[15])};
          }
          const int col = cur.nt * 256 + wn * 128 + n * 32 + (l & 7) * 8;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = q * 8 + (l >> 3);
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(tmp + (i >> 4) * (4 * kBlock) + (i & 15) * 128 +
                                                                (((l & 7) ^ (i & 7)) << 4));
            if (p0 + i < cur.rend && col < a.Nout)
              *reinterpret_cast<u32x4_t*>(a.y + (long long)(p0 + i) * a.Nout + col) = v;
          }
        }
      }
    }
    if (!more) break;
    it += slots;
    cur = next;
    next = third;
    gw[0] = gn[0];
    gw[1] = gn[1];
  }
  __builtin_amdgcn_s_waitcnt((0 & 15) | (7 << 4) | (15 << 8));  // no LDS-DMA outlives the workgroup
}

// Which kernel takes a problem.  Streaming reads an expert's weights once per 32
// rows, and its items are short: it is ahead with less than 24 rows an expert, and
// with more as long as its gate/up items (32 rows x 64 features) do not fill the
// 512 workgroups that are resident.  Measured, streamed / in tiles: 128 experts of
// the Qwen3 shape with 16 rows 68 / 74 us, 24 rows 75 / 74, 32 rows 96 / 76, 64
// rows 138 / 80; 16 experts of 2048 x 1024 with 24 rows (192 items) 21 / 32, 64
// rows (512) 33 / 27; 2 of 1024 x 768 with 512 rows (384) 18 / 20, 1024 rows (768)
// 24 / 21; one of 7168 x 2048 with 128 rows (128) 30 / 49, 512 rows (512) 55 / 51.
// Row-major weights always come in tiles: a lane's pieces of its row, read straight
// into registers, are 32 bytes of each of 32 rows a load (128 experts of the Qwen3
// shape with 4 rows 149 us, in tiles 77; 8 of 4096 x 1536 with 1 row 42 and 35; the
// other way round only for the smallest: 2 of 1024 x 768 16 and 18).
// Rows are counted over all T k slots, as the host knows no more: where a rank holds
// a part of the experts, those named here are all its slots', of which it keeps some.
bool use_tiles(const Shape& s) {
  return !s.blocked || (s.S >= 24LL * s.El && s.S * s.F >= 448LL * (32 * 64));
}

// Groups of 32 rows that the experts' segments can have.
size_t max_groups(const Shape& s) { return (size_t)mx_max_groups(s.S, s.El, use_tiles(s) ? kBM : 1); }

template <bool kGateUp>
hipError_t launch_products(const Shape& s, const MxArgs& a, hipStream_t st) {
  if (!use_tiles(s)) {
    const long long items = (long long)max_groups(s) * (a.Nout / (kGateUp ? 64 : 128));
    const int grid = (int)std::min(512LL, (items + 7) / 8 * 8);
    hipLaunchKernelGGL(mx_stream_kernel<kGateUp>, dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  static std::atomic<uint64_t> done{0};
  const hipError_t e = set_lds_attr(reinterpret_cast<const void*>(mx_tile_kernel<kGateUp>), tile_lds(kMaxExperts), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(mx_tile_kernel<kGateUp>, dim3(512), dim3(256), tile_lds(s.El), st, a);
  return hipGetLastError();
}

template <bool kQuantize>
hipError_t convert(int batch, int rows, int cols, int bf16, const void* src, void* dst, uint8_t* codes,
                   uint8_t* scales, int block_major, hipStream_t st) {
  const MxConvertPlan plan = mx_convert_plan(batch, rows, cols, block_major);
  const ConvertArgs a{src,  dst,     codes,          scales,         rows,
                      cols, plan.rt, plan.row_tiles, plan.col_tiles, plan.tiles};
  const unsigned grid = (unsigned)std::min(a.tiles, 1LL << 20);
  auto go = [&](auto b, auto m, auto p) {
    if constexpr (kQuantize)
      hipLaunchKernelGGL((mx_quantize_kernel<b.value, m.value, p.value>), dim3(grid), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((mx_dequantize_kernel<b.value, m.value, p.value>), dim3(grid), dim3(256), 0, st, a);
  };
  auto with_layout = [&](auto b) {
    using std::integral_constant;
    if (!block_major) go(b, std::false_type{}, integral_constant<int, 1>{});
    else if (a.rt == 8) go(b, std::true_type{}, integral_constant<int, 1>{});
    else go(b, std::true_type{}, integral_constant<int, 8>{});
  };
  if (bf16) with_layout(std::true_type{});
  else with_layout(std::false_type{});
  return hipGetLastError();
}

}  // namespace

hipError_t mx_quantize(int batch, int rows, int cols, int bf16, const void* src, uint8_t* codes,
                       uint8_t* scales, int block_major, hipStream_t st) {
  return convert<true>(batch, rows, cols, bf16, src, nullptr, codes, scales, block_major, st);
}

hipError_t mx_dequantize(int batch, int rows, int cols, int bf16, const uint8_t* codes,
                         const uint8_t* scales, void* dst, int block_major, hipStream_t st) {
  return convert<false>(batch, rows, cols, bf16, nullptr, dst, const_cast<uint8_t*>(codes),
                        const_cast<uint8_t*>(scales), block_major, st);
}

size_t mx_ffn_ws_bytes(const Shape& s) {
  return align_up(max_groups(s) * (s.F / 64) * 1024) + align_up(max_groups(s) * (s.F / 128) * 128 + 256);
}

hipError_t expert_ffn_mx(const Shape& s, const uint8_t* x, const uint8_t* xs, const int32_t* sorted_slot,
                         const int32_t* offsets, const void* w_gate, const void* w_up,
                         const void* w_down, const void* s_gate, const void* s_up,
                         const void* s_down, const float* topk_w, void* y, void* ws, hipStream_t st) {
  uint8_t* h = static_cast<uint8_t*>(ws);
  uint8_t* hs = h + align_up(max_groups(s) * (s.F / 64) * 1024);
  MxArgs a{};
  a.A = x;
  a.AS = xs;
  a.a_bytes = (uint32_t)((long long)s.T * s.d / 2);
  a.as_bytes = (uint32_t)((long long)s.T * s.d / 32);
  a.sorted_slot = sorted_slot;
  a.offsets = offsets;
  a.k = s.k;
  a.W0 = static_cast<const uint8_t*>(w_gate);
  a.W1 = static_cast<const uint8_t*>(w_up);
  a.S0 = static_cast<const uint8_t*>(s_gate);
  a.S1 = static_cast<const uint8_t*>(s_up);
  a.h = h;
  a.hs = hs;
  a.El = s.El;
  a.S = (int)s.S;
  a.max_groups = (int)max_groups(s);
  a.K = s.d;
  a.Nout = s.F;
  a.blocked = s.blocked;
  hipError_t e = launch_products<true>(s, a, st);
  if (e != hipSuccess) return e;
  a.A = h;
  a.AS = hs;
  a.W0 = static_cast<const uint8_t*>(w_down);
  a.W1 = nullptr;
  a.S0 = static_cast<const uint8_t*>(s_down);
  a.S1 = nullptr;
  a.topk_w = topk_w;
  a.y = static_cast<uint16_t*>(y);
  a.K = s.F;
  a.Nout = s.d;
  return launch_products<false>(s, a, st);
}

}  // namespace moe

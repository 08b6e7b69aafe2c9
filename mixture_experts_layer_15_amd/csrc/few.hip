// The whole layer for a handful of tokens, in two kernels.
//
// "Serving MoE models with expert parallelism on 8xH200" (reviosa), section
// "Batching: MoE needs bigger batches than you think": with few tokens every
// expert that is touched sees one or two rows and the layer streams weights.
// At one token the weights take less time than the launches, partial sums and
// drained chips of a kernel per stage, so here one kernel forms the logits and
// a second does the rest:
//
//  router   a workgroup forms the logits of four experts (all of K; no partial
//           sums leave it) and clears the counters of the second kernel.
//  layer    every workgroup selects the top k of every token (a few hundred
//           logits) and lists the touched experts for itself; then workgroups
//           take tickets: first the gate/up items (expert, 32 features), then
//           the down items (64 columns, expert).  An item is two weight blocks
//           of 32 rows that the four waves stream into registers, a quarter of
//           K each, and multiply on the matrix cores (the expert's rows, at
//           most 16, are one operand); the quarters meet in LDS.  A down item
//           starts its weights' loads, then waits for its expert's h.  The
//           last of a column group's down items adds the slots in order.
//
// A waiting workgroup holds a down ticket, so every gate/up ticket is already
// held by a running workgroup, and those never wait: the wait ends whatever
// else runs on the device, also if only some of the workgroups ever become
// resident.  What crosses workgroups (h, the experts' rows, counters) is
// written and read with device-scope accesses, which go past the L2 of the
// XCD; a store is complete (vmcnt) before the counter that announces it moves.
#include <algorithm>
#include <type_traits>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMaxTokens = MOE_FEW_MAX_TOKENS;
constexpr int kMaxSlots = MOE_FEW_MAX_SLOTS;
constexpr int kPad = 16;        // words between counters: a cache line each
constexpr int kRowPad = 36;     // floats of a token's 32 results in LDS
constexpr int kThreads = 256;
constexpr int kRouterThreads = 512;
static_assert(kMaxTokens <= 16, "an item's rows are half of a 32-row operand");
static_assert(kMaxSlots <= kThreads, "a thread per slot");

struct FewArgs {
  const void* x;
  const void* w_router;
  const float* bias;
  float* logits;
  int32_t* topk_idx;   // or null
  float* topk_w;       // or null
  const void* W[3];    // gate, up, down
  const void* S[3];
  void* out;
  uint32_t* ctr;       // ticket, then a counter per listed expert and per column group
  int n_ctr;           // words
  void* h;             // [slots][F] act, rows in the experts' order
  float* y;            // [slots][d], slot order
  int T, d, E, k, F, e0, El;
  int blocked;
};

__device__ __forceinline__ uint32_t* expert_counter(const FewArgs& a, int i) { return a.ctr + (1 + i) * kPad; }
__device__ __forceinline__ uint32_t* column_counter(const FewArgs& a, int i) {
  return a.ctr + (1 + kMaxSlots + i) * kPad;
}

// ---- router

// Sums of the first N of v over the wave; lane l ends with one of them in
// v[0], the one whose number it returns.  A step halves the values: N + 6
// exchanges rather than 6 N.
template <int N, int O = 1, int M>
__device__ __forceinline__ int wave_sums(float (&v)[M]) {
  if constexpr (N > 1) {
    const bool up = lane_id() & O;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float keep = up ? v[i + N / 2] : v[i], send = up ? v[i] : v[i + N / 2];
      v[i] = keep + __shfl_xor(send, O, kWave);
    }
    return (up ? N / 2 : 0) + wave_sums<N / 2, O * 2>(v);
  } else if constexpr (O < kWave) {
    v[0] += __shfl_xor(v[0], O, kWave);
    return wave_sums<1, O * 2>(v);
  } else {
    return 0;
  }
}

template <bool kBF16, int TT>
__global__ __launch_bounds__(kRouterThreads) void few_router_kernel(FewArgs a) {
  __shared__ float part[kRouterThreads / kWave][TT * 4];
  const int tid = threadIdx.x;
  for (int i = blockIdx.x * kRouterThreads + tid; i < a.n_ctr; i += gridDim.x * kRouterThreads) a.ctr[i] = 0;
  if (a.w_router == nullptr) return;
  const int e0 = blockIdx.x * 4;
  const bool whole = a.E % 4 == 0;
  float acc[TT * 4];
#pragma unroll
  for (int i = 0; i < TT * 4; ++i) acc[i] = 0.0f;
  // a thread: four rows of the matrix, four experts
  for (int c = tid * 4; c < a.d; c += kRouterThreads * 4) {
    float w[4][4], x[TT][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const long long at = (long long)(c + r) * a.E + e0;
      if constexpr (kBF16) {
        const uint16_t* p = static_cast<const uint16_t*>(a.w_router) + at;
        if (whole) {
          const u32x2_t u = *reinterpret_cast<const u32x2_t*>(p);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[r][j] = bf16_to_f32(uint16_t(u[j >> 1] >> (16 * (j & 1))));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[r][j] = e0 + j < a.E ? bf16_to_f32(p[j]) : 0.0f;
        }
      } else {
        const float* p = static_cast<const float*>(a.w_router) + at;
        if (whole) {
          const f32x4_t u = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[r][j] = u[j];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[r][j] = e0 + j < a.E ? p[j] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const long long at = (long long)min(t, a.T - 1) * a.d + c;
      if constexpr (kBF16) {
        const u32x2_t u = *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(a.x) + at);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[t][r] = bf16_to_f32(uint16_t(u[r >> 1] >> (16 * (r & 1))));
      } else {
        const f32x4_t u = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.x) + at);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[t][r] = u[r];
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t * 4 + j] = fmaf(x[t][r], w[r][j], acc[t * 4 + j]);
  }
  const int i = wave_sums<TT * 4>(acc);
  if (lane_id() < TT * 4) part[tid / kWave][i] = acc[0];
  __syncthreads();
  if (tid < TT * 4) {
    float s = part[0][tid];
#pragma unroll
    for (int w = 1; w < kRouterThreads / kWave; ++w) s += part[w][tid];
    const int t = tid / 4, e = e0 + tid % 4;
    if (t < a.T && e < a.E) a.logits[t * a.E + e] = a.bias ? s + a.bias[e] : s;
  }
}

// ---- selection

// Logits as integers in their order: NaN and -inf lowest, -0 as 0; 0 is below
// them all.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) v = -__builtin_inff();
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOE_DPP_MAX(ctrl) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false))
  MOE_DPP_MAX(0x111);  // within 16 lanes
  MOE_DPP_MAX(0x112);
  MOE_DPP_MAX(0x114);
  MOE_DPP_MAX(0x118);
  MOE_DPP_MAX(0x142);  // from the 16 lanes before
  MOE_DPP_MAX(0x143);  // from the 32 lanes before
#undef MOE_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// What every workgroup of the layer kernel knows.
struct Plan {
  int idx[kMaxSlots];        // chosen expert of a slot
  float gate[kMaxSlots];
  int first[kMaxSlots];      // first slot of the same expert, -1: not local
  int expert[kMaxSlots];     // listed experts, by first slot: local id
  int row0[kMaxSlots + 1];   // first row of a listed expert
  int list_row0[kMaxSlots];  // the same, by the expert's first slot
  int slot[kMaxSlots];       // slot of a row
  int n, rows;               // listed experts, rows
  int ticket, last;
};

__device__ __forceinline__ void select_top_k(const FewArgs& a, Plan& p) {
  constexpr int kV = kMaxExperts / kWave;
  const int wave = threadIdx.x / kWave, l = lane_id();
  for (int t = wave; t < a.T; t += kThreads / kWave) {
    uint32_t key[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int e = j * kWave + l;
      key[j] = e < a.E ? logit_key(a.logits[t * a.E + e]) : 0;
    }
    float top = 0.0f, sum = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      uint32_t m = key[0];
#pragma unroll
      for (int j = 1; j < kV; ++j) m = max(m, key[j]);
      m = wave_max(m);
      int e = -1;  // the lowest expert with this key
#pragma unroll
      for (int j = kV - 1; j >= 0; --j) {
        const uint64_t b = __ballot(key[j] == m);
        if (b) e = j * kWave + __builtin_ctzll(b);
      }
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (e == j * kWave + l) key[j] = 0;
      const float v = key_logit(m);
      if (i == 0) top = v;
      const float w = expf(v - top);
      sum += w;
      if (l == 0) {
        p.idx[t * a.k + i] = e;
        p.gate[t * a.k + i] = w;
      }
    }
    __builtin_amdgcn_wave_barrier();  // (this wave's own LDS writes, in order)
    for (int i = l; i < a.k; i += kWave) p.gate[t * a.k + i] /= sum;
  }
}

// Lists the touched local experts in the order of their first slots, and
// their slots in increasing order.
__device__ __forceinline__ void make_plan(const FewArgs& a, Plan& p) {
  const int s = threadIdx.x, S = a.T * a.k;
  int first = -1, pos = 0;
  if (s < S) {
    const int e = p.idx[s];
    if (e >= a.e0 && e < a.e0 + a.El) {
      for (int q = S - 1; q >= 0; --q)
        if (p.idx[q] == e) first = q;
      for (int q = first; q < s; ++q) pos += p.idx[q] == e;
    }
    p.first[s] = first;
  }
  __syncthreads();
  if (s < S && first == s) {
    int rank = 0, row0 = 0;
    for (int q = 0; q < S; ++q) {
      const int f = p.first[q];
      rank += q < s && f == q;
      row0 += f >= 0 && f < s;
    }
    p.expert[rank] = p.idx[s] - a.e0;
    p.row0[rank] = row0;
    p.list_row0[s] = row0;
  }
  if (s == 0) {
    int n = 0, rows = 0;
    for (int q = 0; q < S; ++q) {
      n += p.first[q] == q;
      rows += p.first[q] >= 0;
    }
    p.n = n;
    p.rows = rows;
    p.row0[n] = rows;
  }
  __syncthreads();
  if (first >= 0) p.slot[p.list_row0[first] + pos] = s;
  __syncthreads();
}

// ---- the products

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// cache policies of raw buffer loads: weights pass once (nt); what another
// workgroup of this launch wrote is read at device scope (sc1)
constexpr int kOnce = 2, kDevice = 16;

// kV: values of a lane's 16-byte piece; a load covers 32 rows of 2 kV values of
// K: lane l holds row l % 32, values (l / 32) kV ...  In either weight layout
// the loads of a block follow each other at a fixed step.
template <int kFmt>
struct Format {
  static constexpr int kV = kFmt == kF32 ? 4 : kFmt == kBF16 ? 8 : kFmt == kFP8 ? 16 : 32;
  static constexpr int kPieces = kFmt == kF32 ? 1 : kV / 8;  // 16-byte pieces of activations
  // loads a wave keeps in flight per weight block (fp8: whole scale blocks of 4)
  static constexpr int kD = kFmt == kFP4 ? 6 : kFmt == kFP8 ? 8 : 12;
  static constexpr int kSplit = kFmt == kFP8 ? 4 : 1;  // loads that stay in one wave
};

// One item's two weight blocks times the expert's rows: this wave's quarter of
// K, result [block][feature 16 (l / 32) + q][token l % 32].  `ready` is called
// once the first weights are on their way and before any activation is read.
template <int kFmt, bool kDown, typename F>
__device__ __forceinline__ void stream_item(const FewArgs& a, int expert, int fb0, int fb1, const void* x,
                                            uint32_t x_bytes, uint32_t x_row, F&& ready, f32x16_t (&acc)[2]) {
  using C = Format<kFmt>;
  constexpr bool kAct32 = kFmt == kF32;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l = lane_id(), g = l >> 5, r = l & 31;
  const int K = kDown ? a.F : a.d, N = kDown ? a.d : a.F;
  const int n = K / (2 * C::kV) / C::kSplit;  // splittable runs of loads
  const int s0 = n * wave / 4 * C::kSplit, s1 = n * (wave + 1) / 4 * C::kSplit;
  const uint32_t row_bytes = (uint32_t)K / C::kV * 16u;
  const uint32_t mat = (uint32_t)N * row_bytes;
  const int feature = (((r >> 2) & 1) << 4) | (((r >> 3) & 3) << 2) | (r & 3);
  const uint32_t voff = a.blocked ? 16u * l : (uint32_t)feature * row_bytes + 16u * g;
  const uint32_t step = a.blocked ? 1024u : 32u;
  const unsigned char* w0 = static_cast<const unsigned char*>(a.W[kDown ? 2 : 0]) + (size_t)expert * mat;
  const unsigned char* w1 = kDown ? w0 : static_cast<const unsigned char*>(a.W[1]) + (size_t)expert * mat;
  const uint32_t o0 = (uint32_t)fb0 * 32u * row_bytes, o1 = (uint32_t)fb1 * 32u * row_bytes;
  // MXFP4 scales [K / 32][N]
  const uint32_t smat = (uint32_t)(K / 32) * N;
  const unsigned char* m0 = static_cast<const unsigned char*>(a.S[kDown ? 2 : 0]) + (kFmt == kFP4 ? (size_t)expert * smat : 0);
  const unsigned char* m1 = kDown ? m0 : static_cast<const unsigned char*>(a.S[1]) + (kFmt == kFP4 ? (size_t)expert * smat : 0);
  const uint32_t svoff = (uint32_t)g * N + feature;
  // FP8 scales [N / 128][K / 128]
  const float* q0 = static_cast<const float*>(a.S[kDown ? 2 : 0]) + ((size_t)expert * (N / 128) + fb0 / 4) * (K / 128);
  const float* q1 = static_cast<const float*>(a.S[kDown ? 2 : 1]) + ((size_t)expert * (N / 128) + fb1 / 4) * (K / 128);

  u32x4_t wb[C::kD][2], xb[C::kD][C::kPieces];
  uint32_t sb[C::kD][2];
  // Loads behind this wave's part of K read nothing (a buffer of no bytes
  // gives zeros), so that the loop has no branches and its waits are exact.
  auto issue_w = [&](int s, int e) {
    const bool in = s < s1;
    wb[e][0] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(w0, in ? mat : 0), voff, o0 + s * step, kOnce);
    wb[e][1] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(w1, in ? mat : 0), voff, o1 + s * step, kOnce);
    if constexpr (kFmt == kFP4) {
      sb[e][0] = __builtin_amdgcn_raw_buffer_load_b8(rsrc(m0, in ? smat : 0), svoff, (uint32_t)(2 * s) * N + fb0 * 32u, 0);
      sb[e][1] = __builtin_amdgcn_raw_buffer_load_b8(rsrc(m1, in ? smat : 0), svoff, (uint32_t)(2 * s) * N + fb1 * 32u, 0);
    }
  };
  const uint32_t xoff = x_row + (uint32_t)g * C::kV * (kAct32 ? 4u : 2u);
  auto issue_x = [&](int s, int e) {
    const __amdgpu_buffer_rsrc_t rx = rsrc(x, s < s1 ? x_bytes : 0);
#pragma unroll
    for (int q = 0; q < C::kPieces; ++q)
      xb[e][q] = __builtin_amdgcn_raw_buffer_load_b128(rx, xoff + 16u * q, (uint32_t)s * (2 * C::kV) * (kAct32 ? 4u : 2u),
                                                       kDown ? kDevice : 0);
  };
  f32x16_t part[2];
  auto compute = [&](int s, int e) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if constexpr (kFmt == kF32) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(wb[e][b][q]), __uint_as_float(xb[e][0][q]), acc[b], 0, 0, 0);
      } else if constexpr (kFmt == kBF16) {
        acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, wb[e][b]),
                                                         __builtin_bit_cast(bf16x8_t, xb[e][0]), acc[b], 0, 0, 0);
      } else if constexpr (kFmt == kFP8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const u32x2_t lo = e4m3x4_to_bf16x4(wb[e][b][2 * q]), hi = e4m3x4_to_bf16x4(wb[e][b][2 * q + 1]);
          part[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, u32x4_t{lo[0], lo[1], hi[0], hi[1]}),
                                                            __builtin_bit_cast(bf16x8_t, xb[e][q]), part[b], 0, 0, 0);
        }
      } else {
        const float sc = e8m0_to_f32(sb[e][b]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e2m1x8_to_bf16x8(wb[e][b][q], sc),
                                                           __builtin_bit_cast(bf16x8_t, xb[e][q]), acc[b], 0, 0, 0);
      }
    }
    if constexpr (kFmt == kFP8) {
      if (e % 4 == 3) {  // a scale block ends: its sums enter with its scales
        const int kb = min(s / 4, K / 128 - 1);
        const float f0 = q0[kb], f1 = q1[kb];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          acc[0][q] = fmaf(f0, part[0][q], acc[0][q]);
          acc[1][q] = fmaf(f1, part[1][q], acc[1][q]);
        }
        part[0] = f32x16_t{};
        part[1] = f32x16_t{};
      }
    }
  };
#pragma unroll
  for (int b = 0; b < 2; ++b) acc[b] = part[b] = f32x16_t{};
#pragma unroll
  for (int e = 0; e < C::kD; ++e) issue_w(s0 + e, e);
  ready();
#pragma unroll
  for (int e = 0; e < C::kD; ++e) issue_x(s0 + e, e);
  for (int s = s0; s < s1; s += C::kD) {
#pragma unroll
    for (int e = 0; e < C::kD; ++e) {
      compute(s + e, e);
      issue_w(s + e + C::kD, e);
      issue_x(s + e + C::kD, e);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// This wave's results to LDS, tokens 0 .. 15: red[wave][block][token][feature].
__device__ __forceinline__ void to_lds(float (*red)[2][kMaxTokens][kRowPad], const f32x16_t (&acc)[2]) {
  const int l = lane_id(), g = l >> 5, r = l & 31;
  if (r < kMaxTokens) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 16; q += 4)
        *reinterpret_cast<f32x4_t*>(&red[threadIdx.x / kWave][b][r][16 * g + q]) =
            f32x4_t{acc[b][q], acc[b][q + 1], acc[b][q + 2], acc[b][q + 3]};
  }
}

__device__ __forceinline__ float quarters(float (*red)[2][kMaxTokens][kRowPad], int b, int r, int f) {
  return ((red[0][b][r][f] + red[1][b][r][f]) + red[2][b][r][f]) + red[3][b][r][f];
}

// Every device-scope store of this thread is complete.
__device__ __forceinline__ void stores_done() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  asm volatile("" ::: "memory");
}

template <typename T>
__device__ __forceinline__ void device_store(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int kFmt>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
  constexpr bool kAct32 = kFmt == kF32;
  __shared__ Plan p;
  __shared__ __attribute__((aligned(16))) float red[4][2][kMaxTokens][kRowPad];
  const int tid = threadIdx.x;
  uint32_t next = 0;
  if (tid == 0) next = __hip_atomic_fetch_add(a.ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  select_top_k(a, p);
  __syncthreads();
  if (blockIdx.x == 0 && tid < a.T * a.k) {
    if (a.topk_idx) a.topk_idx[tid] = p.idx[tid];
    if (a.topk_w) a.topk_w[tid] = p.gate[tid];
  }
  make_plan(a, p);
  if (p.n == 0) {  // no local expert is touched
    const int size = a.T * a.d * (kAct32 ? 4 : 2) / 16;  // d is a multiple of 128
    for (int i = blockIdx.x * kThreads + tid; i < size; i += gridDim.x * kThreads)
      static_cast<u32x4_t*>(a.out)[i] = u32x4_t{0, 0, 0, 0};
    return;
  }
  const int nf = a.F / 32, nc = a.d / 64;
  const int n_up = p.n * nf, n_items = n_up + nc * p.n;
  const int r = lane_id() & 31;
  for (;;) {
    if (tid == 0) p.ticket = (int)next;
    __syncthreads();
    const int item = __builtin_amdgcn_readfirstlane(p.ticket);
    if (item >= n_items) return;
    if (tid == 0) next = __hip_atomic_fetch_add(a.ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    f32x16_t acc[2];
    if (item < n_up) {
      const int i = item / nf, fb = item % nf;
      const int row0 = __builtin_amdgcn_readfirstlane(p.row0[i]), n = __builtin_amdgcn_readfirstlane(p.row0[i + 1]) - row0;
      const uint32_t t = (uint32_t)p.slot[row0 + min(r, n - 1)] / (uint32_t)a.k;
      const uint32_t xrow = (uint32_t)a.d * (kAct32 ? 4u : 2u);
      stream_item<kFmt, false>(a, __builtin_amdgcn_readfirstlane(p.expert[i]), fb, fb, a.x, (uint32_t)a.T * xrow, t * xrow, [] {}, acc);
      to_lds(red, acc);
      __syncthreads();
      for (int q = tid; q < n * 32; q += kThreads) {
        const int row = q / 32, f = q % 32;
        const float z = quarters(red, 0, row, f), u = quarters(red, 1, row, f);
        const long long at = (long long)(row0 + row) * a.F + fb * 32 + f;
        if constexpr (kAct32) {
          device_store(static_cast<float*>(a.h) + at, z / (1.0f + expf(-z)) * u);
        } else {
          const uint32_t v = f32_to_bf16(silu_f32(z) * u);
          const uint32_t w = (uint32_t)__shfl_xor((int)v, 1, kWave);  // (the neighbour is in the loop too)
          if (f % 2 == 0) device_store(reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.h) + at), v | w << 16);
        }
      }
      stores_done();
      __syncthreads();
      if (tid == 0)
        __hip_atomic_fetch_add(expert_counter(a, i), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else {
      const int c = (item - n_up) / p.n, i = (item - n_up) % p.n;
      const int row0 = __builtin_amdgcn_readfirstlane(p.row0[i]), n = __builtin_amdgcn_readfirstlane(p.row0[i + 1]) - row0;
      const uint32_t hrow = (uint32_t)a.F * (kAct32 ? 4u : 2u);
      stream_item<kFmt, true>(
          a, __builtin_amdgcn_readfirstlane(p.expert[i]), 2 * c, 2 * c + 1, a.h, (uint32_t)p.rows * hrow,
          (uint32_t)(row0 + min(r, n - 1)) * hrow,
          [&] {
            if (tid == 0)
              while (__hip_atomic_load(expert_counter(a, i), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < (uint32_t)nf)
                __builtin_amdgcn_s_sleep(1);
            __syncthreads();
          },
          acc);
      to_lds(red, acc);
      __syncthreads();
      for (int q = tid; q < n * 64; q += kThreads) {
        const int row = q / 64, b = q / 32 % 2, f = q % 32;
        const int slot = p.slot[row0 + row];
        device_store(a.y + (long long)slot * a.d + c * 64 + q % 64, quarters(red, b, row, f) * p.gate[slot]);
      }
      stores_done();
      __syncthreads();
      if (tid == 0)
        p.last = __hip_atomic_fetch_add(column_counter(a, c), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(p.n - 1);
      __syncthreads();
      if (p.last) {
        for (int q = tid; q < a.T * 64; q += kThreads) {
          const int t = q / 64, col = c * 64 + q % 64;
          float sum = 0.0f;
          for (int s = t * a.k; s < (t + 1) * a.k; ++s)
            if (p.first[s] >= 0)
              sum += __hip_atomic_load(a.y + (long long)s * a.d + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          if constexpr (kAct32) static_cast<float*>(a.out)[(long long)t * a.d + col] = sum;
          else static_cast<uint16_t*>(a.out)[(long long)t * a.d + col] = f32_to_bf16(sum);
        }
      }
    }
  }
}

struct FewLayout {
  size_t ctr, logits, h, y, total;
  int n_ctr;
};

FewLayout few_layout(const Shape& s) {
  FewLayout L{};
  L.n_ctr = (1 + kMaxSlots + s.d / 64) * kPad;
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.ctr = take((size_t)L.n_ctr * 4);
  L.logits = take((size_t)s.T * s.E * 4);
  L.h = take((size_t)s.S * s.F * act_bytes(s));
  L.y = take((size_t)s.S * s.d * 4);
  L.total = o;
  return L;
}

}  // namespace

size_t few_ws_bytes(const Shape& s) { return few_layout(s).total; }

hipError_t forward_few(const Shape& s, const moe_forward_args_t& f, void* ws, hipStream_t st) {
  const FewLayout L = few_layout(s);
  unsigned char* base = static_cast<unsigned char*>(ws);
  FewArgs a{};
  a.x = f.x;
  a.w_router = f.w_router;
  a.bias = f.router_bias;
  a.logits = f.logits ? f.logits : reinterpret_cast<float*>(base + L.logits);
  a.topk_idx = f.topk_idx;
  a.topk_w = f.topk_w;
  a.W[0] = f.w_gate;
  a.W[1] = f.w_up;
  a.W[2] = f.w_down;
  a.S[0] = f.s_gate;
  a.S[1] = f.s_up;
  a.S[2] = f.s_down;
  a.out = f.out;
  a.ctr = reinterpret_cast<uint32_t*>(base + L.ctr);
  a.n_ctr = L.n_ctr;
  a.h = base + L.h;
  a.y = reinterpret_cast<float*>(base + L.y);
  a.T = s.T;
  a.d = s.d;
  a.E = s.E;
  a.k = s.k;
  a.F = s.F;
  a.e0 = s.e0;
  a.El = s.El;
  a.blocked = s.blocked;
  auto router = [&](auto bf16, auto tt) {
    hipLaunchKernelGGL((few_router_kernel<bf16.value, tt.value>), dim3((s.E + 3) / 4), dim3(kRouterThreads), 0, st, a);
  };
  using std::integral_constant;
  auto by_tokens = [&](auto bf16) {
    if (s.T == 1) router(bf16, integral_constant<int, 1>{});
    else if (s.T <= 4) router(bf16, integral_constant<int, 4>{});
    else router(bf16, integral_constant<int, kMaxTokens>{});
  };
  if (s.act == kBF16) by_tokens(std::true_type{});
  else by_tokens(std::false_type{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // two workgroups a compute unit; fewer where there are fewer items
  const long long items = std::min<long long>(s.S, s.El) * (s.F / 32 + s.d / 64);
  const dim3 grid((unsigned)std::min(512LL, items)), block(kThreads);
  switch (s.weight) {
    case kF32:
      hipLaunchKernelGGL(few_layer_kernel<kF32>, grid, block, 0, st, a);
      break;
    case kBF16:
      hipLaunchKernelGGL(few_layer_kernel<kBF16>, grid, block, 0, st, a);
      break;
    case kFP8:
      hipLaunchKernelGGL(few_layer_kernel<kFP8>, grid, block, 0, st, a);
      break;
    default:
      hipLaunchKernelGGL(few_layer_kernel<kFP4>, grid, block, 0, st, a);
      break;
  }
  return hipGetLastError();
}

}  // namespace moe

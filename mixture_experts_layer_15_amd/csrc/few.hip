// The whole layer for a handful of tokens, in two kernels.
//
// "Serving MoE models with expert parallelism on 8xH200" (reviosa), section
// "Batching: MoE needs bigger batches than you think": with few tokens every
// expert that is touched sees one or two rows and the layer streams weights.
// At one token the weights take less time than the launches, partial sums and
// drained chips of a kernel per stage, so here one kernel forms the logits and
// a second does the rest:
//
//  router   a workgroup forms the logits of four experts for up to four tokens
//           (all of K; no partial sums leave it); the counters of the second
//           kernel are cleared.
//  layer    every workgroup selects the top k of every token (a few hundred
//           logits) and lists the touched experts for itself.  The gate/up
//           items (expert, 32 features) are cut into a share per workgroup, and
//           so are the down items (64 columns, a run of the listed experts).
//           The four waves stream an item's two weight blocks of 32 rows into
//           registers, taking turns along K, and multiply them on the matrix
//           cores; column t of the other operand is token t (zeros where it did
//           not choose the expert), so a down item adds its experts in the
//           accumulators, in list order, with the gates applied to h.  The
//           waves' sums meet in LDS.  The next gate/up item's loads are under
//           way before the present one's results are; a down item starts its
//           weights' loads, then waits for its experts' h.  The last of a
//           column group's down items adds the others' sums in order.
//
// Waiting: a share of gate/up items belongs to who claims it first, which is its
// own workgroup if that has started.  Before a workgroup waits for any h, it
// takes every share that is not claimed, so that all of them are held by
// running workgroups, and those do not wait before theirs is done: the wait
// ends whatever else runs on the device, also if only some of the workgroups
// ever become resident.  (Claims lie apart, a word each: tickets from one
// counter took 5.8 us for 512 workgroups, from eight 1.4 us a ticket each.)
//
// What crosses workgroups (h, partial sums, counters) is written and read with
// device-scope accesses, which go past the L2 of the XCD; a store is complete
// (vmcnt) before the counter that announces it moves.
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
constexpr int kGrid = 512;      // workgroups of the layer kernel: two a compute unit
constexpr int kRouterThreads = 1024;
constexpr int kRouterTokens = 4;  // most tokens of a workgroup of the router
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
  uint32_t* ctr;       // claims, then a counter per listed expert and per column group
  int n_ctr;           // words
  void* h;             // [rows][F] float32, or [2][rows][F] bfloat16 planes; rows in the experts' order
  float* y;            // [parts][T][d] sums of the down items
  int log_parts;       // down items of a column group, at most 2^log_parts
  int T, d, E, k, F, e0, El;
};

__device__ __forceinline__ uint32_t* claim(const FewArgs& a, int share) { return a.ctr + share; }
__device__ __forceinline__ uint32_t* expert_counter(const FewArgs& a, int i) { return a.ctr + kGrid + i * kPad; }
__device__ __forceinline__ uint32_t* column_counter(const FewArgs& a, int i) {
  return a.ctr + kGrid + (kMaxSlots + i) * kPad;
}
__device__ __forceinline__ uint32_t device_load(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t device_add(uint32_t* p) {
  return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// TT tokens a workgroup, 1 or 4: one of one token takes 4.2 us (2048 x 128; as one
// of four 4.7), five tokens 5.1, sixteen of 7168 x 256 12.6 (one at a time 33).
// Bound by latency and by the cache lines of the matrix, 8 bytes of each of which
// are a workgroup's.
template <bool kBF16, int TT>
__global__ __launch_bounds__(kRouterThreads) void few_router_kernel(FewArgs a) {
  __shared__ float part[kRouterThreads / kWave][TT * 4];
  const int tid = threadIdx.x;
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * kRouterThreads + tid; i < a.n_ctr; i += gridDim.x * kRouterThreads) a.ctr[i] = 0;
  if (a.w_router == nullptr) return;
  // Neighbouring experts, which share the matrix's lines, to one XCD (workgroup b
  // runs on XCD b % 8).
  const int nx = gridDim.x, per = nx % 8 == 0 ? nx / 8 : 0;
  const int e0 = (per ? blockIdx.x % 8 * per + blockIdx.x / 8 : blockIdx.x) * 4, t0 = blockIdx.y * TT;
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
      const long long at = (long long)min(t0 + t, a.T - 1) * a.d + c;
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
    const int t = t0 + tid / 4, e = e0 + tid % 4;
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
  int idx[kMaxSlots];          // chosen expert of a slot
  float gate[kMaxSlots];
  float raw[kMaxSlots];        // its logit, then exp(logit - largest)
  uint32_t tokens[kMaxExperts];  // tokens that chose a local expert, a bit each
  int expert[kMaxSlots];       // listed experts, by first token and rank: local id
  int row0[kMaxSlots];         // first row of a listed expert in h (a row per token that chose it)
  int place[kMaxExperts];      // the same, by local id
  float row_gate[kMaxSlots];   // gate of a row
  int n, rows;                 // listed experts, rows
  int wave_n[kThreads / kWave], wave_rows[kThreads / kWave];
  int free_share, last;        // on their way to all threads
};

// The k largest of each token's logits (ties to the lower expert), a wave per
// token (at most four tokens).  Lane l holds experts l kV ... sorted, so the
// wave's largest is among the lanes' first, and of equal ones the lowest lane
// has the lowest expert.
template <int kV>
__device__ __forceinline__ void select_by_waves(const FewArgs& a, Plan& p) {
  const int t = threadIdx.x / kWave, l = lane_id();
  if (t >= a.T) return;
  uint32_t key[kV];
  int id[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    id[j] = l * kV + j;
    key[j] = __float_as_uint(a.logits[t * a.E + min(id[j], a.E - 1)]);  // (all loads before any use)
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) key[j] = id[j] < a.E ? logit_key(__uint_as_float(key[j])) : 0;
#pragma unroll
  for (int j = 1; j < kV; ++j)  // insertion: stable
#pragma unroll
    for (int i = j; i > 0; --i) {
      const bool up = key[i] > key[i - 1];
      const uint32_t hi = up ? key[i] : key[i - 1], lo = up ? key[i - 1] : key[i];
      const int hid = up ? id[i] : id[i - 1], lid = up ? id[i - 1] : id[i];
      key[i - 1] = hi, key[i] = lo;
      id[i - 1] = hid, id[i] = lid;
    }
  uint32_t got = 0;  // what lane l has been given: choice l, l + 64, ...
  int got_id = 0;
  for (int i = 0; i < a.k; ++i) {
    const uint32_t m = wave_max(key[0]);
    const int owner = __builtin_ctzll(__ballot(key[0] == m));
    const int e = __builtin_amdgcn_readlane(id[0], owner);
    if (l == (i & (kWave - 1))) {
      got = m;
      got_id = e;
    }
    if (l == owner) {
#pragma unroll
      for (int j = 1; j < kV; ++j) {
        key[j - 1] = key[j];
        id[j - 1] = id[j];
      }
      key[kV - 1] = 0;
    }
    if ((i & (kWave - 1)) == kWave - 1 || i == a.k - 1) {
      const int base = i & ~(kWave - 1);
      if (base + l <= i) {
        p.idx[t * a.k + base + l] = got_id;
        p.raw[t * a.k + base + l] = key_logit(got);
      }
    }
  }
}

// The same, 16 lanes a token, so that a workgroup has all sixteen in one pass
// (k <= 64 then).  Lane r of 16 holds experts r, r + 16, ...
template <int kV>
__device__ __forceinline__ void select_by_rows(const FewArgs& a, Plan& p) {
  const int t = threadIdx.x / 16, l = lane_id(), r = l & 15;
  uint32_t key[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    key[j] = __float_as_uint(a.logits[min(t, a.T - 1) * a.E + min(j * 16 + r, a.E - 1)]);
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) key[j] = t < a.T && j * 16 + r < a.E ? logit_key(__uint_as_float(key[j])) : 0;
  for (int i = 0; i < a.k; ++i) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < kV; ++j) {
      const bool up = key[j] > best;
      best = up ? key[j] : best;
      at = up ? j : at;
    }
    const int e = at * 16 + r;
    // the largest key of the 16 lanes, then the lowest expert that has it
    uint32_t m = best;
#define MOE_DPP_ROW(f, v, ctrl) v = f(v, (decltype(v))__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false))
    MOE_DPP_ROW(max, m, 0x128);  // rotations by 8, 4, 2, 1: every lane gets it
    MOE_DPP_ROW(max, m, 0x124);
    MOE_DPP_ROW(max, m, 0x122);
    MOE_DPP_ROW(max, m, 0x121);
    int low = best == m ? e : kMaxExperts;
    MOE_DPP_ROW(min, low, 0x128);
    MOE_DPP_ROW(min, low, 0x124);
    MOE_DPP_ROW(min, low, 0x122);
    MOE_DPP_ROW(min, low, 0x121);
#undef MOE_DPP_ROW
#pragma unroll
    for (int j = 0; j < kV; ++j) key[j] = low == j * 16 + r ? 0 : key[j];
    if (t < a.T && r == (i & 15)) {
      p.idx[t * a.k + i] = low;
      p.raw[t * a.k + i] = key_logit(m);
    }
  }
}

// Gates, and the touched local experts with their slots: experts in the order
// of their first token (and its choices), an expert's slots by token.
__device__ __forceinline__ void make_plan(const FewArgs& a, Plan& p) {
  for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) p.tokens[e] = 0;
  if (a.T <= kThreads / kWave) {
    if (a.E <= 128) select_by_waves<2>(a, p);
    else if (a.E <= 256) select_by_waves<4>(a, p);
    else select_by_waves<8>(a, p);
  } else {
    if (a.E <= 128) select_by_rows<8>(a, p);
    else if (a.E <= 256) select_by_rows<16>(a, p);
    else select_by_rows<32>(a, p);
  }
  __syncthreads();
  const int s = threadIdx.x, S = a.T * a.k, t = s / a.k;
  const int wave = s / kWave, l = lane_id();
  int e = -1;
  float w = 0.0f;
  if (s < S) {
    e = p.idx[s] - a.e0;
    if (e >= a.El) e = -1;
    w = expf(p.raw[s] - p.raw[t * a.k]);
    if (e >= 0) atomicOr(&p.tokens[e], 1u << t);
  }
  __syncthreads();
  if (s < S) p.raw[s] = w;
  const uint32_t mask = e >= 0 ? p.tokens[e] : 0;
  const bool first = mask && __builtin_ctz(mask) == t;
  // prefix sums of listed experts and of their rows
  const uint64_t b = __ballot(first);
  int rank = __builtin_popcountll(b & ((1ull << l) - 1));
  const int count = first ? __builtin_popcount(mask) : 0;
  int row = count;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(row, o, kWave);
    if (l >= o) row += v;
  }
  if (l == kWave - 1) {
    p.wave_n[wave] = __builtin_popcountll(b);
    p.wave_rows[wave] = row;
  }
  row -= count;
  __syncthreads();
  if (s < S) {
    float sum = 0.0f;
    for (int i = t * a.k; i < (t + 1) * a.k; ++i) sum += p.raw[i];
    p.gate[s] = w / sum;
  }
  int n = 0, rows = 0;
#pragma unroll
  for (int v = 0; v < kThreads / kWave; ++v) {
    if (v == wave) {
      rank += n;
      row += rows;
    }
    n += p.wave_n[v];
    rows += p.wave_rows[v];
  }
  if (first) {
    p.expert[rank] = e;
    p.row0[rank] = row;
    p.place[e] = row;
  }
  if (s == 0) {
    p.n = n;
    p.rows = rows;
  }
  __syncthreads();
  if (mask) p.row_gate[p.place[e] + __builtin_popcount(mask & ((1u << t) - 1))] = p.gate[s];
  __syncthreads();
}

// ---- the products

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// cache policies of raw buffer loads: blocked weights pass once (nt; of a
// row-major matrix a load takes half of a line or less, and others the rest);
// what another workgroup of this launch wrote is read
// at device scope (sc1).  (An acquire fence and cached reads instead: 4 us more
// until the first products, as the weights under way are dropped with the rest.)
constexpr int kOnce = 2, kDevice = 16;

// An offset behind every array of activations: such a lane reads zeros.
constexpr uint32_t kNowhere = 0x40000000u;

// kV: values of a lane's 16-byte piece; a load covers 32 rows of 2 kV values of
// K: lane l holds row l % 32, values (l / 32) kV ...  In either weight layout
// the loads of a block follow each other at a fixed step.
template <int kFmt, bool kBlocked, bool kDown>
struct Format {
  static constexpr bool kAct32 = kFmt == kF32;
  static constexpr int kV = kFmt == kF32 ? 4 : kFmt == kBF16 ? 8 : kFmt == kFP8 ? 16 : 32;
  static constexpr int kPieces = kFmt == kF32 ? 1 : kV / 8;  // 16-byte pieces of activations
  // h is two bfloat16 planes, value and remainder (one alone would add as much
  // error as the rounding of the output): the remainders are columns 16 .. 31
  // of the operand, so they cost no load and no product of their own.
  static constexpr bool kPlanes = kDown && kFmt != kF32;
  // In gate/up those columns are idle: their lanes load every second piece for
  // the lanes 16 before them, which get it by a swap of 16-lane rows.
  static constexpr bool kPairs = !kDown && kPieces > 1;
  static constexpr int kXLoads = kPairs ? kPieces / 2 : kPieces;
  // The waves take turns of kRun loads along K: FP8 a scale block, of a
  // row-major matrix whole lines (MXFP4: half of one, as K may be 128).
  // Blocked, one load: adjacent waves on adjacent kilobytes stream 50 MB in 8.8
  // us, a quarter of K each in 10.3.
  static constexpr int kRun = kFmt == kFP8 ? 4 : kBlocked ? 1 : kFmt == kFP4 ? 2 : 4;
  // A run of a row-major matrix is 128 bytes of 32 rows.  Load j takes 64 bytes (a
  // half g of them) of row 4 m + j by lanes 4 m .. 4 m + 3, which then exchange
  // what belongs to each other's rows: four lanes that read 16 bytes of a row
  // each pass the cache at a quarter of the rate.  (So K comes in another order:
  // piece 4 g + j of a run in its step j.  Sixteen tokens of the Qwen3 shape in
  // bfloat16 236 -> 169 us, in FP8 155 -> 115 (102 since the
  // parts' sums are loaded together), five in float32 242 -> 146.)
  static constexpr bool kQuads = !kBlocked && kRun == 4;
  // loads a wave keeps in flight per weight block (two of four KB each do:
  // 6.6 TB/s, as eight or twelve)
  static constexpr int kD = kFmt == kFP4 ? 4 : kFmt == kFP8 && !kDown && kBlocked ? 4 : 8;
  static constexpr int kLoads = 2 + kXLoads + (kFmt == kFP4 ? 2 : 0);  // of a step
  static_assert(kD % kRun == 0 && kD * kLoads < 64, "whole runs in the ring, a countable number of loads");
};

// What a wave streams: two weight blocks of one expert and its activations.
struct Source {
  const unsigned char *w0, *w1;  // the expert's matrices
  uint32_t w_bytes;              // 0: nothing
  uint32_t o0, o1;               // the blocks in them
  const unsigned char *m0, *m1;  // MXFP4 scales
  const float *q0, *q1;          // FP8 scales of the blocks' rows
  uint32_t f0, f1;               // first features of the blocks
  uint32_t x;                    // this lane's activations
};

template <int kFmt, bool kBlocked, bool kDown>
struct Stream {
  using C = Format<kFmt, kBlocked, kDown>;
  const FewArgs& a;
  const int wave, l, g, r;
  const int K, N, runs, steps;  // steps: of a block, padded to whole turns of the ring
  const uint32_t row_bytes, mat, smat, voff, svoff;
  const void* xbase;
  uint32_t x_bytes;
  u32x4_t wb[C::kD][2], xb[C::kD][C::kXLoads];
  uint32_t sb[C::kD][2];
  f32x16_t acc[2], part[2];

  __device__ __forceinline__ Stream(const FewArgs& args)
      : a(args),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)),
        l(lane_id()),
        g(l >> 5),
        r(l & 31),
        K(kDown ? args.F : args.d),
        N(kDown ? args.d : args.F),
        runs(K / (2 * C::kV) / C::kRun),
        steps(((runs + 3) / 4 * C::kRun + C::kD - 1) / C::kD * C::kD),
        row_bytes((uint32_t)K / C::kV * 16u),
        mat((uint32_t)N * row_bytes),
        smat((uint32_t)(K / 32) * N),
        voff(kBlocked      ? 16u * l
             : C::kQuads ? (uint32_t)feature(r & ~3) * row_bytes + 64u * g + 16u * (l & 3)
                         : (uint32_t)feature(r) * row_bytes + 16u * g),
        svoff((uint32_t)g * N + feature(r)) {}

  // permuted weight row of MFMA row r of a 32-row block
  static __device__ __forceinline__ int feature(int r) {
    return (((r >> 2) & 1) << 4) | (((r >> 3) & 3) << 2) | (r & 3);
  }

  // Blocks fb0 and fb1 (gate/up: of either matrix) of local expert e; the
  // lane's row of activations at offset x.
  __device__ __forceinline__ Source source(int e, int fb0, int fb1, uint32_t x) const {
    Source s;
    s.w0 = static_cast<const unsigned char*>(a.W[kDown ? 2 : 0]) + (size_t)e * mat;
    s.w1 = kDown ? s.w0 : static_cast<const unsigned char*>(a.W[1]) + (size_t)e * mat;
    s.w_bytes = mat;
    s.o0 = (uint32_t)fb0 * 32u * row_bytes;
    s.o1 = (uint32_t)fb1 * 32u * row_bytes;
    s.m0 = s.m1 = nullptr;
    s.q0 = s.q1 = nullptr;
    if constexpr (kFmt == kFP4) {  // [K / 32][N]
      s.m0 = static_cast<const unsigned char*>(a.S[kDown ? 2 : 0]) + (size_t)e * smat;
      s.m1 = kDown ? s.m0 : static_cast<const unsigned char*>(a.S[1]) + (size_t)e * smat;
    }
    if constexpr (kFmt == kFP8) {  // [N / 128][K / 128]
      s.q0 = static_cast<const float*>(a.S[kDown ? 2 : 0]) + ((size_t)e * (N / 128) + fb0 / 4) * (K / 128);
      s.q1 = static_cast<const float*>(a.S[kDown ? 2 : 1]) + ((size_t)e * (N / 128) + fb1 / 4) * (K / 128);
    }
    s.f0 = (uint32_t)fb0 * 32u;
    s.f1 = (uint32_t)fb1 * 32u;
    s.x = x + (uint32_t)g * (C::kQuads ? 4 : 1) * C::kV * (C::kAct32 ? 4u : 2u);
    return s;
  }

  // Step j of this wave: its load number along K, and whether there is one (a
  // buffer of no bytes gives zeros: no branches, and exact waits).
  __device__ __forceinline__ int load_of(int j) const { return (j / C::kRun * 4 + wave) * C::kRun + j % C::kRun; }
  __device__ __forceinline__ bool within(int j) const { return j / C::kRun * 4 + wave < runs; }

  __device__ __forceinline__ void issue_w(const Source& s, int j, int e) {
    const bool in = within(j);
    const uint32_t q = load_of(j);
    const uint32_t at = C::kQuads ? q / 4 * 128u + q % 4 * row_bytes : q * (kBlocked ? 1024u : 32u);
    constexpr int kPolicy = kBlocked ? kOnce : 0;
    wb[e][0] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(s.w0, in ? s.w_bytes : 0), voff, s.o0 + at, kPolicy);
    wb[e][1] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(s.w1, in ? s.w_bytes : 0), voff, s.o1 + at, kPolicy);
    if constexpr (kFmt == kFP4) {
      const uint32_t bytes = in && s.w_bytes ? smat : 0;
      sb[e][0] = __builtin_amdgcn_raw_buffer_load_b8(rsrc(s.m0, bytes), svoff, 2 * q * N + s.f0, 0);
      sb[e][1] = __builtin_amdgcn_raw_buffer_load_b8(rsrc(s.m1, bytes), svoff, 2 * q * N + s.f1, 0);
    }
  }

  __device__ __forceinline__ void issue_x(const Source& s, int j, int e) {
    const __amdgpu_buffer_rsrc_t rx = rsrc(xbase, within(j) && s.w_bytes ? x_bytes : 0);
    const uint32_t q4 = load_of(j);
    const uint32_t at = (C::kQuads ? q4 / 4 * 8 + q4 % 4 : 2 * q4) * (C::kV * (C::kAct32 ? 4u : 2u));
#pragma unroll
    for (int q = 0; q < C::kXLoads; ++q)
      xb[e][q] = __builtin_amdgcn_raw_buffer_load_b128(rx, s.x + 16u * q * (C::kPairs ? 2 : 1), at, kDown ? kDevice : 0);
  }

  // Steps e .. e + 3 of a row-major run: lane c of four has piece c of row j in
  // place e + j, and gets piece j of its own row.
  __device__ __forceinline__ void exchange(int e) {
    const bool odd = l & 1, high = l & 2;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = wb[e + j][b][i];
        auto swap = [](uint32_t& lo, uint32_t& hi, bool up, auto perm) {
          const uint32_t from_hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)hi, perm.value, 15, 15, true);
          const uint32_t from_lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)lo, perm.value, 15, 15, true);
          lo = up ? from_hi : lo;
          hi = up ? hi : from_lo;
        };
        std::integral_constant<int, 0xB1> by1;  // quad_perm 1, 0, 3, 2
        std::integral_constant<int, 0x4E> by2;  // 2, 3, 0, 1
        swap(v[0], v[1], odd, by1);
        swap(v[2], v[3], odd, by1);
        swap(v[0], v[2], high, by2);
        swap(v[1], v[3], high, by2);
#pragma unroll
        for (int j = 0; j < 4; ++j) wb[e + j][b][i] = v[j];
      }
    }
  }

  // Piece q of step e's activations (in columns that nobody reads: any other).
  __device__ __forceinline__ bf16x8_t activations(int e, int q) const {
    if constexpr (C::kPairs) {
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = xb[e][q / 2][i];
        v[i] = q % 2 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)[1] : x;
      }
      return __builtin_bit_cast(bf16x8_t, v);
    } else {
      return __builtin_bit_cast(bf16x8_t, xb[e][q]);
    }
  }

  // Step j's products; q0, q1: the FP8 scales of the blocks' rows.
  __device__ __forceinline__ void compute(int j, int e, const float* q0, const float* q1) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if constexpr (kFmt == kF32) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(wb[e][b][q]), __uint_as_float(xb[e][0][q]), acc[b], 0, 0, 0);
      } else {
        f32x16_t& sum = kFmt == kFP8 ? part[b] : acc[b];
        const float sc = kFmt == kFP4 ? e8m0_to_f32(sb[e][b]) : 0.0f;
#pragma unroll
        for (int q = 0; q < C::kPieces; ++q) {
          bf16x8_t w;
          if constexpr (kFmt == kBF16) {
            w = __builtin_bit_cast(bf16x8_t, wb[e][b]);
          } else if constexpr (kFmt == kFP8) {
            const u32x2_t lo = e4m3x4_to_bf16x4(wb[e][b][2 * q]), hi = e4m3x4_to_bf16x4(wb[e][b][2 * q + 1]);
            w = __builtin_bit_cast(bf16x8_t, u32x4_t{lo[0], lo[1], hi[0], hi[1]});
          } else {
            w = e2m1x8_to_bf16x8(wb[e][b][q], sc);
          }
          sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, activations(e, q), sum, 0, 0, 0);
        }
      }
    }
    if constexpr (kFmt == kFP8) {
      if (e % 4 == 3) {  // a scale block ends: its sums enter with its scales
        const int kb = min(load_of(j) / 4, K / 128 - 1);
        const float f0 = q0[kb], f1 = q1[kb];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          acc[0][q] = fmaf(f0, part[0][q], acc[0][q]);
          acc[1][q] = fmaf(f1, part[1][q], acc[1][q]);
        }
        part[0] = part[1] = f32x16_t{};
      }
    }
  }

  __device__ __forceinline__ void clear() { acc[0] = acc[1] = part[0] = part[1] = f32x16_t{}; }

  // A turn of the ring: steps s .. s + kD - 1 of an item with the FP8 scales q0
  // and q1, whose places take the steps from `next` on of `src`.  (sched_barrier
  // keeps the loads in this order: the compiler's waits are then for exactly
  // the loads that a step needs.)
  __device__ __forceinline__ void turn(int s, const float* q0, const float* q1, const Source& src, int next) {
#pragma unroll
    for (int e = 0; e < C::kD; ++e) {
      if (C::kQuads && e % 4 == 0) exchange(e);
      compute(s + e, e, q0, q1);
      issue_w(src, next + e, e);
      issue_x(src, next + e, e);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The waves' results: [block][token][feature], of h's remainders the same again.
typedef float Results[2][kMaxTokens][kRowPad];

// Columns 0 .. 15 to red[0 .. 3], with kBoth also 16 .. 31 to red[4 .. 7].
template <bool kBoth>
__device__ __forceinline__ void to_lds(Results* red, const f32x16_t (&acc)[2]) {
  const int l = lane_id(), g = l >> 5, r = l & 31;
  if (kBoth || r < kMaxTokens) {
    Results& to = red[r / kMaxTokens * 4 + threadIdx.x / kWave];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 16; q += 4)
        *reinterpret_cast<f32x4_t*>(&to[b][r % kMaxTokens][16 * g + q]) =
            f32x4_t{acc[b][q], acc[b][q + 1], acc[b][q + 2], acc[b][q + 3]};
  }
}

__device__ __forceinline__ float all_waves(const Results* red, int b, int r, int f) {
  return ((red[0][b][r][f] + red[1][b][r][f]) + red[2][b][r][f]) + red[3][b][r][f];
}

// At most N of this thread's vector-memory operations are outstanding (they
// complete in the order in which they were issued).
template <int N>
__device__ __forceinline__ void wait_memory() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

template <typename T>
__device__ __forceinline__ void device_store(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Gate/up items [item, end): h of one feature block of one listed expert each.
// Returns the last one's expert, which is not announced yet.
template <int kFmt, bool kBlocked>
__device__ __forceinline__ int up_items(const FewArgs& a, const Plan& p, Results* red, int item, int end) {
  constexpr bool kAct32 = kFmt == kF32;
  const int tid = threadIdx.x;
  const int nf = a.F / 32;
  Stream<kFmt, kBlocked, false> st(a);
  using C = typename Stream<kFmt, kBlocked, false>::C;
  const uint32_t xrow = (uint32_t)a.d * (kAct32 ? 4u : 2u);
  st.xbase = a.x;
  st.x_bytes = (uint32_t)a.T * xrow;
  int i = item / nf, fb = item % nf;    // the item under way
  int in = i, fbn = fb, left = end - item;  // the item to be loaded, and how many are left
  auto source = [&]() {
    if (left == 0) {
      Source s = st.source(0, 0, 0, kNowhere);
      s.w_bytes = 0;
      return s;
    }
    const int e = __builtin_amdgcn_readfirstlane(p.expert[in]);
    const uint32_t mask = p.tokens[e];
    // (a pair's second piece: lanes 16 on)
    const int t = C::kPairs ? st.r % kMaxTokens : st.r;
    Source s = st.source(e, fbn, fbn, mask >> t & 1 ? t * xrow + (st.r - t) : kNowhere);
    --left;
    if (++fbn == nf) {
      fbn = 0;
      ++in;
    }
    return s;
  };
  Source src = source();
#pragma unroll
  for (int e = 0; e < C::kD; ++e) {
    st.issue_w(src, e, e);
    st.issue_x(src, e, e);
    __builtin_amdgcn_sched_barrier(0);
  }
  int stored = -1;  // the expert whose h is stored but not yet announced
  for (int turn = 0; item < end; ++item, ++turn) {
    st.clear();
    const float *q0 = src.q0, *q1 = src.q1;
    for (int s = 0; s < st.steps; s += C::kD) {
      const bool last = s + C::kD == st.steps;  // the next item's first loads take the places
      if (last) src = source();
      st.turn(s, q0, q1, src, last ? 0 : s + C::kD);
    }
    Results* buf = red + (turn & 1) * 4;  // (the other one may still be read)
    to_lds<false>(buf, st.acc);
    // the stores of the item before are older than the loads of the last turn
    wait_memory<C::kD * C::kLoads>();
    __syncthreads();
    if (tid == 0 && stored >= 0) device_add(expert_counter(a, stored));
    const uint32_t mask = p.tokens[p.expert[i]];
    const int row0 = p.row0[i];
    for (int q = tid; q < a.T * 32; q += kThreads) {
      const int t = q / 32, f = q % 32;
      if (!(mask >> t & 1)) continue;  // (the same for the 32 threads of a token)
      const int row = row0 + __builtin_popcount(mask & ((1u << t) - 1));
      const float z = all_waves(buf, 0, t, f), u = all_waves(buf, 1, t, f), gate = p.row_gate[row];
      const long long at = (long long)row * a.F + fb * 32 + f;
      if constexpr (kAct32) {
        device_store(static_cast<float*>(a.h) + at, z / (1.0f + expf(-z)) * u * gate);
      } else {
        const float h = silu_f32(z) * u * gate;
        const uint32_t hi = f32_to_bf16(h);
        // (an h that is infinite as bfloat16 has no remainder: it stays infinite)
        const float rest = __builtin_isinf(bf16_to_f32(hi)) ? 0.0f : h - bf16_to_f32(hi);
        const uint32_t v = hi | (uint32_t)f32_to_bf16(rest) << 16;
        const uint32_t w = (uint32_t)__shfl_xor((int)v, 1, kWave);
        // the even lane stores both features' values, the odd one their remainders
        uint16_t* to = static_cast<uint16_t*>(a.h) + (f % 2 ? (long long)p.rows * a.F - 1 : 0) + at;
        device_store(reinterpret_cast<uint32_t*>(to), f % 2 ? w >> 16 | (v & 0xffff0000u) : (v & 0xffffu) | w << 16);
      }
    }
    stored = i;
    if (++fb == nf) {
      fb = 0;
      ++i;
    }
  }
  return stored;
}

// Claims a share of the gate/up items that no workgroup has claimed; `free` is
// the lowest one that this thread saw.  -1: another workgroup was faster.
__device__ __forceinline__ int claim_share(const FewArgs& a, Plan& p, int free) {
  if (threadIdx.x == 0) p.free_share = kGrid;
  __syncthreads();
  atomicMin(&p.free_share, free);
  __syncthreads();
  const int share = p.free_share;
  if (threadIdx.x == 0)
    p.last = __hip_atomic_exchange(claim(a, share), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0;
  __syncthreads();
  const int got = p.last ? share : -1;
  __syncthreads();
  return got;
}

// One token of the Qwen3 shape (75 MB of bfloat16 weights, blocked) 20 us: 4.5 us
// until the plan stands, 10 of gate/up and down at 6 TB/s and more, and the chip's
// filling and draining twice.  Sixteen tokens of a rank of the DeepSeek-V3 shape
// (565 MB of FP8) 102 us in a steady loop, 111 to 124 traced.  Five tokens with MXFP4
// weights (89 MB) 35 us blocked and 42 row-major, sixteen (200 MB) 59 and 81: 1.5 to
// 2.5 times their bytes' time.  There the matrix cores are busy for 14 to 23 % of the
// cycles and the vector units for 25 to 34; a wave waits for 35 to 43 % of its own.
// Neither fewer nor more loads in flight change it; what it waits for is not known.
template <int kFmt, bool kBlocked>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
  constexpr bool kAct32 = kFmt == kF32;
  __shared__ Plan p;
  __shared__ __attribute__((aligned(16))) Results red[8];
  __shared__ int mine;     // whether this workgroup's own share is its
  __shared__ int spoiled;  // whether a result of the down item under way is not finite
  // shares are a power of two, and so are the parts of a column group
  const int tid = threadIdx.x, shares = gridDim.x, log_shares = __builtin_ctz(gridDim.x);
  if (tid == 0) spoiled = 0;
  // (by the last wave: the first one's loads would wait behind it)
  if (tid == kThreads - 1)
    mine = __hip_atomic_exchange(claim(a, blockIdx.x), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0;
  make_plan(a, p);
  if (blockIdx.x == 0 && tid < a.T * a.k) {
    if (a.topk_idx) a.topk_idx[tid] = p.idx[tid];
    if (a.topk_w) a.topk_w[tid] = p.gate[tid];
  }
  if (p.n == 0) {  // no local expert is touched
    const int size = a.T * a.d * (kAct32 ? 4 : 2) / 16;  // d is a multiple of 128
    for (int i = blockIdx.x * kThreads + tid; i < size; i += shares * kThreads)
      static_cast<u32x4_t*>(a.out)[i] = u32x4_t{0, 0, 0, 0};
    return;
  }
  const int n = __builtin_amdgcn_readfirstlane(p.n), rows = __builtin_amdgcn_readfirstlane(p.rows);
  const int nf = a.F / 32;
  const uint32_t n_up = n * nf;  // at most 256 experts of 2048 blocks; times 512 shares: 32 bits

  // gate/up items: this workgroup's share, and those whose workgroups have not
  // started by then (which does not happen unless the device is busy otherwise)
  for (int share = mine ? (int)blockIdx.x : -1;;) {
    int stored = -1;
    if (share >= 0) {
      const int u0 = n_up * share >> log_shares, u1 = n_up * (share + 1) >> log_shares;
      if (u0 < u1) stored = up_items<kFmt, kBlocked>(a, p, red, u0, u1);
    }
    int free = kGrid;
#pragma unroll
    for (int q = kGrid / kThreads - 1; q >= 0; --q) {
      const int i = min(tid + q * kThreads, shares - 1);
      if (device_load(claim(a, i)) == 0) free = i;
    }
    wait_memory<0>();  // (h is stored)
    const bool any = __syncthreads_or(free < kGrid);
    if (tid == 0 && stored >= 0) device_add(expert_counter(a, stored));
    if (!any) break;
    share = claim_share(a, p, free);
  }

  const int log_parts = min(a.log_parts, 31 - __builtin_clz(n)), parts = 1 << log_parts;
  const int n_down = a.d / 64 * parts;
  // Down item (column group c, part j of the list): those experts' sums for 64
  // columns of every token; the last part's workgroup adds the parts.
  // Tokens that did not choose an expert enter its product as zeros, which add
  // nothing as long as the weights are finite.  Where a result is not finite, the
  // item is taken again, expert by expert: between them the sums wait in `red`,
  // where only the lanes of tokens that chose the expert renew theirs.  So an
  // infinity or a NaN stays with those tokens, and the others get the bits that
  // they get without it.
  Stream<kFmt, kBlocked, true> st(a);
  using C = typename Stream<kFmt, kBlocked, true>::C;
  const uint32_t hrow = (uint32_t)a.F * (kAct32 ? 4u : 2u);
  st.xbase = a.h;
  st.x_bytes = (uint32_t)rows * hrow * (kAct32 ? 1 : 2);
  int c = 0, i0 = 0, i1 = 0;
  int single = -1;  // an item taken again: which of its experts is under way
  bool more = false;  // and whether others follow
  auto place = [&](int item) {
    c = item >> log_parts;
    const int j = item & (parts - 1);
    i0 = n * j >> log_parts;
    i1 = n * (j + 1) >> log_parts;
    more = false;
    if (__builtin_expect(single >= 0, 0)) {
      i0 += single;
      more = i0 + 1 < i1;
      i1 = i0 + 1;
    }
  };
  f32x4_t* const kept = reinterpret_cast<f32x4_t*>(red) + tid;  // this lane's sums, four at a time
  static_assert(sizeof(red) >= 8 * kThreads * sizeof(f32x4_t), "32 sums a lane");
  auto source = [&](int i) {
    const int ii = min(i, n - 1);
    const int e = __builtin_amdgcn_readfirstlane(p.expert[ii]);
    const uint32_t mask = p.tokens[e];
    // column t: token t; column 16 + t: its remainders
    const int t = kAct32 ? st.r : st.r % kMaxTokens;
    const uint32_t row = p.row0[ii] + __builtin_popcount(mask & ((1u << t) - 1)) + (t < st.r ? rows : 0);
    Source s = st.source(e, 2 * c, 2 * c + 1, mask >> t & 1 ? row * hrow : kNowhere);
    if (i >= i1) s.w_bytes = 0;
    return s;
  };
  Source src;
  int item = blockIdx.x;
  auto begin = [&] {  // the first weights of the item
    place(item);
    src = source(i0);
#pragma unroll
    for (int e = 0; e < C::kD; ++e) {
      st.issue_w(src, e, e);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (item < n_down) begin();
  while (item < n_down) {
    for (int i = i0 + tid; i < i1; i += kThreads)
      while (device_load(expert_counter(a, i)) < (uint32_t)nf) __builtin_amdgcn_s_sleep(1);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < C::kD; ++e) {
      st.issue_x(src, e, e);
      __builtin_amdgcn_sched_barrier(0);
    }
    st.clear();
    if (__builtin_expect(single > 0, 0)) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.acc[q / 4][q % 4 * 4 + j] = kept[q * kThreads][j];
    }
    int i = i0, s = 0;
    auto turn = [&] {
      const float *q0 = src.q0, *q1 = src.q1;
      const bool last = s + C::kD == st.steps;  // the next expert's first loads take the places
      if (last) src = source(i + 1);
      st.turn(s, q0, q1, src, last ? 0 : s + C::kD);
      s = last ? 0 : s + C::kD;
      i += last;
    };
    turn();  // (stands apart, as its loads were issued in another order)
    while (i < i1) turn();
    if (__builtin_expect(single >= 0, 0)) {
      const bool chosen = p.tokens[p.expert[i0]] >> (kAct32 ? st.r : st.r % kMaxTokens) & 1;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const f32x16_t& v = st.acc[q / 4];
        const f32x4_t sums = {v[q % 4 * 4], v[q % 4 * 4 + 1], v[q % 4 * 4 + 2], v[q % 4 * 4 + 3]};
        if (chosen) kept[q * kThreads] = sums;
        else if (single == 0) kept[q * kThreads] = f32x4_t{0, 0, 0, 0};
      }
      if (more) {
        ++single;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) st.acc[q / 4][q % 4 * 4 + j] = kept[q * kThreads][j];
        __syncthreads();  // (the results take the place of the kept sums)
      }
    }
    bool again = true;
    if (!more) {
      to_lds<C::kPlanes>(red, st.acc);
      __syncthreads();
      const int j = item & (parts - 1);
      for (int q = tid; q < a.T * 64; q += kThreads) {
        const int t = q / 64, col = c * 64 + q % 64;
        float v = all_waves(red, q / 32 % 2, t, q % 32);
        if constexpr (C::kPlanes) {
          // (a product that is not finite is so in the values' sum; the remainders
          // would make a NaN of an infinity)
          const float rest = all_waves(red + 4, q / 32 % 2, t, q % 32);
          if (__builtin_isfinite(rest)) v += rest;
        }
        if (single < 0 && !__builtin_isfinite(v)) spoiled = 1;
        if (parts > 1) device_store(a.y + ((long long)j * a.T + t) * a.d + col, v);
        else if constexpr (kAct32) static_cast<float*>(a.out)[(long long)t * a.d + col] = v;
        else static_cast<uint16_t*>(a.out)[(long long)t * a.d + col] = f32_to_bf16(v);
      }
      if (parts > 1) wait_memory<0>();  // (the sums are stored)
      __syncthreads();
      again = single < 0 && __builtin_amdgcn_readfirstlane(spoiled);
      single = again ? 0 : -1;
      if (parts > 1 && !again) {
        if (tid == 0) p.last = device_add(column_counter(a, c)) == (uint32_t)(parts - 1);
        __syncthreads();
        if (p.last) {
          for (int q = tid; q < a.T * 64; q += kThreads) {
            const int t = q / 64, col = c * 64 + q % 64;
            float sum = 0.0f;
            for (int m = 0; m < parts; m += 8) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                v[i] = __hip_atomic_load(a.y + ((long long)min(m + i, parts - 1) * a.T + t) * a.d + col, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
              __builtin_amdgcn_sched_barrier(0);  // (all loads before the first sum: one by one,
                                                  // as the compiler may leave them, MXFP4 blocked, 16 tokens, takes 77 us, not 64)
#pragma unroll
              for (int i = 0; i < 8; ++i) sum += m + i < parts ? v[i] : 0.0f;
            }
            if constexpr (kAct32) static_cast<float*>(a.out)[(long long)t * a.d + col] = sum;
            else static_cast<uint16_t*>(a.out)[(long long)t * a.d + col] = f32_to_bf16(sum);
          }
        }
      }
    }
    if (!again) item += shares;
    if (item < n_down) {
      __syncthreads();
      if (tid == 0) spoiled = 0;
      begin();
    }
  }
}

struct FewLayout {
  size_t ctr, logits, h, y, total;
  int n_ctr, log_parts;
};

FewLayout few_layout(const Shape& s) {
  FewLayout L{};
  L.n_ctr = kGrid + (kMaxSlots + s.d / 64) * kPad;
  // down items of a column group: two workgroups a compute unit have one each
  const long long parts = std::min<long long>(kGrid / (s.d / 64), std::min<long long>(s.S, s.El));
  while ((2LL << L.log_parts) <= parts) ++L.log_parts;
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.ctr = take((size_t)L.n_ctr * 4);
  L.logits = take((size_t)s.T * s.E * 4);
  L.h = take((size_t)s.S * s.F * 4);
  L.y = take(L.log_parts > 0 ? ((size_t)s.T * s.d * 4) << L.log_parts : 0);
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
  a.log_parts = L.log_parts;
  a.h = base + L.h;
  a.y = reinterpret_cast<float*>(base + L.y);
  a.T = s.T;
  a.d = s.d;
  a.E = s.E;
  a.k = s.k;
  a.F = s.F;
  a.e0 = s.e0;
  a.El = s.El;
  auto router = [&](auto bf16, auto tt) {
    const dim3 grid((s.E + 3) / 4, f.w_router ? (s.T + tt.value - 1) / tt.value : 1);
    hipLaunchKernelGGL((few_router_kernel<bf16.value, tt.value>), grid, dim3(kRouterThreads), 0, st, a);
  };
  using std::integral_constant;
  auto by_tokens = [&](auto bf16) {
    if (s.T == 1) router(bf16, integral_constant<int, 1>{});
    else router(bf16, integral_constant<int, kRouterTokens>{});
  };
  if (s.act == kBF16) by_tokens(std::true_type{});
  else by_tokens(std::false_type{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // fewer workgroups where there are fewer items
  const long long experts = std::min<long long>(s.S, s.El);
  const long long items = std::max(experts * (s.F / 32), (long long)(s.d / 64) << L.log_parts);
  unsigned shares = 1;
  while (shares < kGrid && shares < items) shares *= 2;
  const dim3 grid(shares), block(kThreads);
  auto layer = [&](auto kern) { hipLaunchKernelGGL(kern, grid, block, 0, st, a); };
  if (s.weight == kF32) layer(few_layer_kernel<kF32, false>);
  else if (s.weight == kBF16) s.blocked ? layer(few_layer_kernel<kBF16, true>) : layer(few_layer_kernel<kBF16, false>);
  else if (s.weight == kFP8) s.blocked ? layer(few_layer_kernel<kFP8, true>) : layer(few_layer_kernel<kFP8, false>);
  else s.blocked ? layer(few_layer_kernel<kFP4, true>) : layer(few_layer_kernel<kFP4, false>);
  return hipGetLastError();
}

}  // namespace moe

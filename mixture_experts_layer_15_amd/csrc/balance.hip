// Balance loss over the router's softmax, per-expert counts, and the gradient
// of gates and losses with respect to the logits.
//
// With V the tokens that the mask keeps, N = |V|, p[t] the softmax of row t
// over all E experts and lse[t] its log-sum-exp:
//   counts[e]   = number of slots (t, i) with t in V and topk_idx[t][i] = e
//   P[e]        = (1/N) sum_{t in V} p[t][e]
//   balance     = E / (N k) * sum_e counts[e] P[e]
//   z           = (1/N) sum_{t in V} lse[t]^2
// The counts are constants of the gradient (they are piecewise constant in
// the logits), so with a, b the gradients of the two losses and g, w the
// gates' gradient and value:
//   dL[t][e] = sum_{i: idx[t][i] = e} w[t][i] (g[t][i] - sum_j w[t][j] g[t][j])
//            + a E / (N^2 k) p[t][e] (counts[e] - sum_j counts[j] p[t][j])
//            + b (2 / N) lse[t] p[t][e]
// Since sum_j p[t][j] = 1, the counts may be shifted by any constant: they
// are centred on their mean (exactly, in integers), which leaves no
// cancellation for a load near balance.
//
// Both passes read the [T][E] logits once; small batches are bound by the
// launches, large ones by that read and the exponentials (a quarter of the
// rate of other instructions).  A row lies on a group of L lanes with up to
// 16 logits each: the fewer lanes a row has, the fewer steps its maximum and
// sum take, and the several rows of a wave share each step; L is at least
// four where E allows, so that a load covers 64 consecutive bytes of a row.
#include "moe_device.h"
#include "moe_internal.h"
#include "route_plan.h"

namespace moe {
namespace {

constexpr int kThreads = kBalanceThreads;
constexpr int kWaves = kThreads / kWave;
constexpr int kGradThreads = kGateThreads;
constexpr int kGradWaves = kGradThreads / kWave;
static_assert(kRowWave == kWave, "lanes of a wave");

// A RowGeom as a type.
template <int V_, int L_, int C_>
struct RowShape {
  static constexpr int V = V_, L = L_, C = C_;
  static constexpr int Q = C * V;       // logits of a lane
  static constexpr int R = kWave / L;   // rows of a wave
  __device__ static int elem(int g, int q) { return ((q / V) * L + g) * V + q % V; }
};

template <int V, int L, int C, class F>
bool if_geom(const RowGeom& g, F& f) {
  if (g.V != V || g.L != L || g.C != C) return false;
  f(RowShape<V, L, C>{});
  return true;
}

// Calls f with the shape of a geometry that row_geom or wide_row_geom gives.
template <class F>
void with_row_shape(const RowGeom& g, F f) {
  (void)(if_geom<4, 1, 1>(g, f) || if_geom<4, 2, 1>(g, f) || if_geom<4, 4, 1>(g, f) ||
         if_geom<4, 4, 2>(g, f) || if_geom<4, 4, 4>(g, f) || if_geom<4, 8, 4>(g, f) ||
         if_geom<4, 16, 4>(g, f) || if_geom<4, 32, 4>(g, f) || if_geom<4, 8, 1>(g, f) ||
         if_geom<4, 16, 1>(g, f) || if_geom<4, 32, 1>(g, f) || if_geom<4, 64, 1>(g, f) ||
         if_geom<4, 64, 2>(g, f) || if_geom<1, 4, 1>(g, f) || if_geom<1, 16, 1>(g, f) ||
         if_geom<1, 16, 2>(g, f) || if_geom<1, 16, 4>(g, f) || if_geom<1, 16, 8>(g, f) ||
         if_geom<1, 16, 16>(g, f) || if_geom<1, 32, 16>(g, f) || if_geom<1, 32, 1>(g, f) ||
         if_geom<1, 64, 1>(g, f) || if_geom<1, 64, 2>(g, f) || if_geom<1, 64, 4>(g, f) ||
         if_geom<1, 64, 8>(g, f));
}

template <class S>
__device__ __forceinline__ void load_row(const float* row, int E, int g, float (&v)[S::Q]) {
#pragma unroll
  for (int c = 0; c < S::C; ++c) {
    const int e = (c * S::L + g) * S::V;
    if constexpr (S::V == 4) {
      f32x4_t r = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < E) r = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c * 4 + i] = r[i];
    } else {
      v[c] = e < E ? row[e] : -INFINITY;
    }
  }
}

// Reduction over the aligned groups of L lanes; every lane gets the result
// (the steps pair equal partial results, so all lanes have the same bits).
// Up to 16 lanes by DPP: exchanges inside quads, then mirrors of 8 and 16.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, false));
}

template <int L, class F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  if constexpr (L >= 2) v = f(v, dpp<0xB1>(v));
  if constexpr (L >= 4) v = f(v, dpp<0x4E>(v));
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16, kWave));
  if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32, kWave));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Logits -> exponentials of the softmax, in place; returns the log-sum-exp,
// and `inv`, the factor that makes them probabilities.  A row of -inf only
// gives zeros; a NaN or +inf makes the whole row NaN (the maximum drops NaN,
// the sum does not).  The exponential is the hardware one: its argument is at
// most 0, and its absolute error is below 2^-22 of the largest term.
template <class S>
__device__ __forceinline__ float row_exp(float (&v)[S::Q], float& inv) {
  float m = v[0];
#pragma unroll
  for (int q = 1; q < S::Q; ++q) m = fmaxf(m, v[q]);
  m = group_max<S::L>(m);
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < S::Q; ++q) {
    v[q] = __expf(v[q] - base);
    s += v[q];
  }
  s = group_sum<S::L>(s);
  const bool dead = s == 0.0f;
  inv = dead ? 0.0f : 1.0f / s;
  return dead ? 0.0f : base + logf(s);
}

// Column sums of a workgroup: the lanes' sums acc over their rows, added over
// the rows of a wave by lane exchanges and over the waves through LDS
// (red [waves][E], filled here; sums in float64 by col_total after a
// barrier), all in a fixed order.
template <class S>
__device__ __forceinline__ void col_partials(float (&acc)[S::Q], int E, float* red) {
  const int l = threadIdx.x % kWave, w = threadIdx.x / kWave;
  const int g = l % S::L;
#pragma unroll
  for (int q = 0; q < S::Q; ++q) {
#pragma unroll
    for (int o = S::L; o < kWave; o *= 2) acc[q] += __shfl_xor(acc[q], o, kWave);
    const int e = S::elem(g, q);
    if (l < S::L && e < E) red[w * E + e] = acc[q];
  }
}
template <int kW>
__device__ __forceinline__ double col_total(const float* red, int E, int e) {
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kW; ++w) s += red[w * E + e];
  return s;
}

// One expert's share of a workgroup's partial sums.
struct ColPart {
  float p;
  int c;
};

struct BalanceArgs {
  const float* logits;
  const int32_t* idx;
  const uint8_t* mask;
  long long T;
  int E, k;
  long long rows_per_block;
  ColPart* part;   // [nb][E]
  double* zpart;   // [nb]
  int* npart;      // [nb]
  unsigned long long* joined;  // the second kernel's arrivals and sum, cleared by the first
  int32_t* counts;
  int32_t* n_tokens;
  float* prob_mean;
  float* losses;
  int nb;
};

// First pass: workgroup b sums the softmax rows, the squared log-sum-exps and
// the slots per expert of its consecutive rows.  kSolo: the only workgroup,
// which also forms the results.
template <class S, bool kSolo>
__global__ __launch_bounds__(kThreads) void balance_rows(BalanceArgs a) {
  __shared__ float red[kWaves * kMaxExperts];
  __shared__ int hist[kMaxExperts];
  __shared__ double wz[kWaves];
  __shared__ int wn[kWaves];
  const int tid = threadIdx.x;
  const int w = tid / kWave, l = tid % kWave;
  const int g = l % S::L, r = l / S::L;
  const long long t0 = blockIdx.x * a.rows_per_block;
  const int rows = (int)min((long long)a.rows_per_block, a.T - t0);
  const float* logits = a.logits + t0 * a.E;
  const int32_t* idx = a.idx + t0 * a.k;
  const uint8_t* mask = a.mask ? a.mask + t0 : nullptr;
  // a row's logits are loaded one row ahead, the first before the counting
  // (masked rows too: what they hold is dropped)
  float cur[S::Q];
  int keep = 0;
  auto load = [&](int t) {
    t = min(t, rows - 1);
    load_row<S>(logits + (long long)t * a.E, a.E, g, cur);
    keep = mask ? mask[t] : 1;
  };
  int t = w * S::R + r;
  if (rows > 0) load(t);  // (0: the only workgroup, of no tokens)
  for (int e = tid; e < a.E; e += kThreads) hist[e] = 0;
  if (!kSolo && blockIdx.x == 0 && tid == 0) *a.joined = 0;
  __syncthreads();
  // slots per expert: integer sums, so the order of the atomics is free
  const long long slots = (long long)rows * a.k;
  for (long long s = tid; s < slots; s += kThreads) {
    if (mask && mask[(uint32_t)s / (uint32_t)a.k] == 0) continue;  // (T k < 2^31)
    const int e = idx[s];
    if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
  }
  float acc[S::Q];
#pragma unroll
  for (int q = 0; q < S::Q; ++q) acc[q] = 0.0f;
  double z = 0.0;
  int n = 0;
  for (; t < rows; t += kWaves * S::R) {
    float v[S::Q], inv;
#pragma unroll
    for (int q = 0; q < S::Q; ++q) v[q] = cur[q];
    const int live = keep;  // the same for the group's lanes
    load(t + kWaves * S::R);
    if (!live) continue;
    const float lse = row_exp<S>(v, inv);
#pragma unroll
    for (int q = 0; q < S::Q; ++q) acc[q] = fmaf(v[q], inv, acc[q]);
    if (g == 0) {
      z += (double)lse * lse;
      ++n;
    }
  }
  col_partials<S>(acc, a.E, red);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    z += __shfl_xor(z, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  if (l == 0) {
    wz[w] = z;
    wn[w] = n;
  }
  __syncthreads();
  z = 0.0;
  n = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    z += wz[i];
    n += wn[i];
  }
  const double inv_n = n > 0 ? 1.0 / n : 0.0;
  double bal = 0.0;
  for (int e = tid; e < a.E; e += kThreads) {  // (at most one: E <= kThreads)
    const double s = col_total<kWaves>(red, a.E, e);
    if constexpr (kSolo) {
      a.counts[e] = hist[e];
      a.prob_mean[e] = (float)(s * inv_n);
      bal += hist[e] * (s * inv_n);
    } else {
      a.part[(size_t)blockIdx.x * a.E + e] = ColPart{(float)s, hist[e]};
    }
  }
  if constexpr (kSolo) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) bal += __shfl_xor(bal, o, kWave);
    __syncthreads();  // wz has been read
    if (l == 0) wz[w] = bal;
    __syncthreads();
    if (tid == 0) {
      bal = 0.0;
      for (int i = 0; i < kWaves; ++i) bal += wz[i];
      *a.n_tokens = n;
      a.losses[0] = (float)(bal * a.E / a.k * inv_n);
      a.losses[1] = (float)(z * inv_n);
    }
  } else if (tid == 0) {
    a.zpart[blockIdx.x] = z;
    a.npart[blockIdx.x] = n;
  }
}

// Second pass: workgroup j adds the partial sums of 16 experts, 64 of them
// abreast, in a fixed order.  The workgroups' shares of the balance loss meet
// in one 64-bit atomic: arrivals in the top six bits (at most 32 workgroups),
// below them the sum in fixed point, 48 bits behind the point (the loss is at
// most E = 512; with the ids of each row's largest logits it is at least
// 1 / (k E) >= 2^-18, so that 32 halves of 2^-48 are below a float32's half
// step).  An integer sum has no order, and the last to arrive has it
// from the atomic itself, without a fence (which cost 2 us).
constexpr int kFinThreads = 1024;
constexpr int kFinCols = 16;
constexpr int kFinRows = kFinThreads / kFinCols;
constexpr int kFinWaves = kFinThreads / kWave;

__global__ __launch_bounds__(kFinThreads) void balance_finish(BalanceArgs a) {
  __shared__ double sp[kFinWaves][kFinCols];
  __shared__ int sc[kFinWaves][kFinCols];
  __shared__ double wz[kFinWaves];
  __shared__ int wn[kFinWaves];
  const int tid = threadIdx.x;
  const int w = tid / kWave, l = tid % kWave;
  const int j = tid % kFinCols, r = tid / kFinCols;
  const int e = blockIdx.x * kFinCols + j;
  static_assert(kMaxRowBlocks <= kFinThreads && kMaxRowBlocks % kFinRows == 0, "one load each");
  double z = tid < a.nb ? a.zpart[tid] : 0.0;
  int n = tid < a.nb ? a.npart[tid] : 0;
  ColPart v[kMaxRowBlocks / kFinRows];  // all loads at once
#pragma unroll
  for (int i = 0; i < kMaxRowBlocks / kFinRows; ++i) {
    const int b = r + i * kFinRows;
    v[i] = ColPart{0.0f, 0};
    if (b < a.nb && e < a.E) v[i] = a.part[(size_t)b * a.E + e];
  }
  double p = 0.0;
  int c = 0;
#pragma unroll
  for (int i = 0; i < kMaxRowBlocks / kFinRows; ++i) {
    p += v[i].p;
    c += v[i].c;
  }
#pragma unroll
  for (int o = kFinCols; o < kWave; o *= 2) {
    p += __shfl_xor(p, o, kWave);
    c += __shfl_xor(c, o, kWave);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    z += __shfl_xor(z, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  if (l < kFinCols) {
    sp[w][l] = p;
    sc[w][l] = c;
  }
  if (l == 0) {
    wz[w] = z;
    wn[w] = n;
  }
  __syncthreads();
  if (w != 0) return;
  p = z = 0.0;
  c = n = 0;
#pragma unroll
  for (int i = 0; i < kFinWaves; ++i) {
    p += sp[i][j];
    c += sc[i][j];
    z += wz[i];
    n += wn[i];
  }
  const double inv_n = n > 0 ? 1.0 / n : 0.0;
  double bal = 0.0;
  if (l < kFinCols && e < a.E) {
    a.counts[e] = c;
    a.prob_mean[e] = (float)(p * inv_n);
    bal = c * (p * inv_n) * a.E / a.k * inv_n;
  }
#pragma unroll
  for (int o = kFinCols / 2; o >= 1; o >>= 1) bal += __shfl_xor(bal, o, kWave);
  if (l != 0) return;
  // a NaN (which z shows) adds nothing
  const unsigned long long fixed =
      z == z ? (unsigned long long)(bal * (double)(1ULL << 48) + 0.5) : 0;
  const unsigned long long mine = (1ULL << 58) + fixed;
  const unsigned long long before =
      __hip_atomic_fetch_add(a.joined, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (before >> 58 != gridDim.x - 1) return;
  const unsigned long long sum = (before & ((1ULL << 58) - 1)) + fixed;
  *a.n_tokens = n;
  a.losses[0] = z == z ? (float)((double)sum / (double)(1ULL << 48)) : (float)z;
  a.losses[1] = (float)(z * inv_n);
}

// ---- gradient with respect to the logits

struct GateGradKernelArgs {
  GateGradArgs a;
  long long T;
  int E, k, Ep;
  int blocks;               // workgroups of the rows; those behind copy pad_src
  int act_bytes;
  long long rows_per_block;
};

// Zeros from value E to Ep (a multiple of 32) of a row whose start is 16-byte
// aligned, by the L lanes of its group.
template <int L, class T>
__device__ __forceinline__ void clear_tail(T* row, int E, int Ep, int g) {
  constexpr int V = 16 / sizeof(T);
  const int up = (E + V - 1) / V * V;
  for (int e = E + g; e < up; e += L) row[e] = T(0);
  for (int e = up + g * V; e < Ep; e += L * V)
    *reinterpret_cast<u32x4_t*>(row + e) = u32x4_t{0, 0, 0, 0};
}

// float32 -> bfloat16 rounding and what it leaves (none of an infinite or
// NaN value, so that it is not turned into another one).
__device__ __forceinline__ uint16_t split_bf16(float& v) {
  const uint16_t h = f32_to_bf16(v);
  const float b = bf16_to_f32(h);
  v = __builtin_isfinite(b) ? v - b : 0.0f;
  return h;
}

// Workgroup b: consecutive rows.  Writes the float32 gradient, what the
// products read (bfloat16 planes whose sum is the value: three hold all 24
// bits, two 16; or the float32 row; columns E .. Ep - 1 are zero), and the
// workgroup's column sums.
//
// The gates' gradient has k values of a row's E.  Lane j of the row's group
// forms that of slot j (then j + L, ...) and adds it to a row of zeros in LDS
// (wave-private; the additions of one instruction to one address are made in
// lane order, and the LDS keeps a wave's instructions in order), from which
// every lane picks its logits' values; comparing every logit with every id
// instead took 2 k instructions a logit.
template <class S>
__global__ __launch_bounds__(kGradThreads) void gate_grad_rows(GateGradKernelArgs ka) {
  __shared__ float red[kGradWaves * kMaxExperts];
  __shared__ __align__(16) float sparse[kGradWaves * kWave * S::Q];  // [wave][row][L Q >= E]
  const GateGradArgs& a = ka.a;
  const int E = ka.E, k = ka.k;
  const int tid = threadIdx.x;
  const int w = tid / kWave, l = tid % kWave;
  if ((int)blockIdx.x >= ka.blocks) {  // a row of pad_src per wave
    const int r = ((int)blockIdx.x - ka.blocks) * kGradWaves + w;
    if (ka.act_bytes == 2) {
      const uint16_t* from = static_cast<const uint16_t*>(a.pad_src) + (size_t)r * E;
      uint16_t* to = static_cast<uint16_t*>(a.pad_dst) + (size_t)r * ka.Ep;
#pragma unroll 4
      for (int e = l; e < ka.Ep; e += kWave) to[e] = e < E ? from[e] : uint16_t(0);
    } else {
      const float* from = static_cast<const float*>(a.pad_src) + (size_t)r * E;
      float* to = static_cast<float*>(a.pad_dst) + (size_t)r * ka.Ep;
#pragma unroll 4
      for (int e = l; e < ka.Ep; e += kWave) to[e] = e < E ? from[e] : 0.0f;
    }
    return;
  }
  const int g = l % S::L, r = l / S::L;
  bool losses = a.dlosses != nullptr;  // (also N > 0, below)
  const bool gates = a.dtopk_w != nullptr;
  const long long t0 = blockIdx.x * ka.rows_per_block;
  const long long t1 = min(t0 + ka.rows_per_block, ka.T);

  // what a row's lanes read, loaded one row ahead
  struct Row {
    float v[S::Q];
    int id;
    float gw, dg;
    int keep;
  };
  // (no value is looked at here, so that the loads are all in flight at once;
  // behind the last row it is read again)
  auto load = [&](long long t, Row& x) {
    t = min(t, t1 - 1);
    x.id = -1;
    x.gw = x.dg = 0.0f;
    x.keep = 1;
#pragma unroll
    for (int q = 0; q < S::Q; ++q) x.v[q] = 0.0f;
    if (losses) load_row<S>(a.logits + t * E, E, g, x.v);
    if (gates && g < k) {
      x.id = a.idx[t * k + g];
      x.gw = a.topk_w[t * k + g];
      x.dg = a.dtopk_w[t * k + g];
    }
    if (a.mask) x.keep = a.mask[t];
  };
  long long t = t0 + w * S::R + r;
  Row cur;
  load(t, cur);

  float* srow = sparse + (w * S::R + r) * (S::L * S::Q);
  float cen[S::Q];  // centred counts, times E
  float ca = 0.0f, cz = 0.0f;
  int cnt[S::Q];
#pragma unroll
  for (int q = 0; q < S::Q; ++q) {
    const int e = S::elem(g, q);
    srow[e] = 0.0f;
    cnt[q] = losses && e < E ? a.counts[e] : 0;
    cen[q] = 0.0f;
  }
  if (losses) {
    const int n = *a.n_tokens;
    const double da = a.dlosses[0], dz = a.dlosses[1];
    // integers in float64 (exact): the counts of many ranks' tokens may pass
    // 2^31 in sum
    double mine = 0.0;
#pragma unroll
    for (int q = 0; q < S::Q; ++q) mine += cnt[q];
#pragma unroll
    for (int o = S::L / 2; o >= 1; o >>= 1) mine += __shfl_xor(mine, o, kWave);
#pragma unroll
    for (int q = 0; q < S::Q; ++q)
      if (S::elem(g, q) < E) cen[q] = (float)((double)cnt[q] * E - mine);  // (an integer below 2^40)
    losses = n > 0;
    if (losses) {
      ca = (float)(da / ((double)n * n * k));
      cz = (float)(dz * 2.0 / n);
    }
  }
  if (blockIdx.x == 0 && tid < kZeroLineBytes / 4)
    reinterpret_cast<uint32_t*>(a.zero_line)[tid] = 0;
  float colsum[S::Q];
#pragma unroll
  for (int q = 0; q < S::Q; ++q) colsum[q] = 0.0f;
  for (; t < t1; t += kGradWaves * S::R) {
    Row x = cur;
    load(t + kGradWaves * S::R, cur);
    float (&v)[S::Q] = x.v;
    if (x.keep) {
      if (gates) {
        const bool ok = (unsigned)x.id < (unsigned)E;
        float gmean = ok ? x.gw * x.dg : 0.0f;
        for (int j = g + S::L; j < k; j += S::L)
          if ((unsigned)a.idx[t * k + j] < (unsigned)E)
            gmean = fmaf(a.topk_w[t * k + j], a.dtopk_w[t * k + j], gmean);
        gmean = group_sum<S::L>(gmean);
        if (ok) unsafeAtomicAdd(&srow[x.id], x.gw * (x.dg - gmean));
        for (int j = g + S::L; j < k; j += S::L) {
          const int e = a.idx[t * k + j];
          if ((unsigned)e < (unsigned)E)
            unsafeAtomicAdd(&srow[e], a.topk_w[t * k + j] * (a.dtopk_w[t * k + j] - gmean));
        }
      }
      if (losses) {
        float inv;
        const float lse = row_exp<S>(v, inv);
        float mean = 0.0f;
#pragma unroll
        for (int q = 0; q < S::Q; ++q) mean = fmaf(v[q], cen[q], mean);
        mean = group_sum<S::L>(mean) * inv;
        const float zl = cz * lse;
#pragma unroll
        for (int q = 0; q < S::Q; ++q) v[q] = v[q] * inv * fmaf(ca, cen[q] - mean, zl);
      } else {
#pragma unroll
        for (int q = 0; q < S::Q; ++q) v[q] = 0.0f;  // (logits, if they were read for N <= 0)
      }
      if (gates) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int c = 0; c < S::C; ++c) {
          if constexpr (S::V == 4) {
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(srow + (c * S::L + g) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[c * 4 + i] += y[i];
          } else {
            v[c] += srow[c * S::L + g];
          }
        }
        asm volatile("" ::: "memory");
        if ((unsigned)x.id < (unsigned)E) srow[x.id] = 0.0f;
        for (int j = g + S::L; j < k; j += S::L) {
          const int e = a.idx[t * k + j];
          if ((unsigned)e < (unsigned)E) srow[e] = 0.0f;
        }
        asm volatile("" ::: "memory");
      }
    } else {
#pragma unroll
      for (int q = 0; q < S::Q; ++q) v[q] = 0.0f;
    }
#pragma unroll
    for (int q = 0; q < S::Q; ++q) colsum[q] += v[q];
#pragma unroll
    for (int c = 0; c < S::C; ++c) {
      const int e = (c * S::L + g) * S::V;
      if constexpr (S::V == 4) {
        if (a.dlogits && e < E)
          *reinterpret_cast<f32x4_t*>(a.dlogits + t * E + e) =
              f32x4_t{v[c * 4], v[c * 4 + 1], v[c * 4 + 2], v[c * 4 + 3]};
      } else {
        if (a.dlogits && e < E) a.dlogits[t * E + e] = v[c];
      }
    }
    if (a.dl_rows) {
      float* row = a.dl_rows + t * ka.Ep;
#pragma unroll
      for (int c = 0; c < S::C; ++c) {
        const int e = (c * S::L + g) * S::V;
        if constexpr (S::V == 4) {
          if (e < E)
            *reinterpret_cast<f32x4_t*>(row + e) =
                f32x4_t{v[c * 4], v[c * 4 + 1], v[c * 4 + 2], v[c * 4 + 3]};
        } else {
          if (e < E) row[e] = v[c];
        }
      }
      clear_tail<S::L>(row, E, ka.Ep, g);
    }
    if (a.live && g == 0) a.live[t] = x.keep;
    if (!a.planes) continue;
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) {
      if (pl >= a.nplanes) break;
      uint16_t* row = a.planes + ((size_t)pl * ka.T + t) * ka.Ep;
#pragma unroll
      for (int c = 0; c < S::C; ++c) {
        const int e = (c * S::L + g) * S::V;
        if constexpr (S::V == 4) {
          uint16_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = split_bf16(v[c * 4 + i]);
          if (e < E)
            *reinterpret_cast<u32x2_t*>(row + e) =
                u32x2_t{h[0] | (uint32_t(h[1]) << 16), h[2] | (uint32_t(h[3]) << 16)};
        } else {
          const uint16_t h = split_bf16(v[c]);
          if (e < E) row[e] = h;
        }
      }
      clear_tail<S::L>(row, E, ka.Ep, g);
    }
  }
  if (!a.bias_part) return;
  col_partials<S>(colsum, E, red);
  __syncthreads();
  for (int e = tid; e < E; e += kGradThreads)
    a.bias_part[(size_t)blockIdx.x * E + e] = (float)col_total<kGradWaves>(red, E, e);
}

struct BalanceLayout {
  size_t part, zpart, npart, joined, total;
};

BalanceLayout balance_layout(const Shape& s) {
  BalanceLayout L{};
  long long rows;
  const int nb = balance_blocks(s.T, s.E, &rows);
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.part = take((size_t)nb * s.E * sizeof(ColPart));
  L.zpart = take((size_t)nb * sizeof(double));
  L.npart = take((size_t)nb * sizeof(int));
  L.joined = take(sizeof(unsigned long long));
  L.total = o;
  return L;
}

}  // namespace

size_t balance_ws_bytes(const Shape& s) { return balance_layout(s).total; }

hipError_t balance_loss(const Shape& s, const float* logits, const int32_t* topk_idx,
                        const uint8_t* mask, int32_t* counts, int32_t* n_tokens,
                        float* prob_mean, float* losses, void* ws, hipStream_t st) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  const BalanceLayout lay = balance_layout(s);
  BalanceArgs a{};
  a.logits = logits;
  a.idx = topk_idx;
  a.mask = mask;
  a.T = s.T;
  a.E = s.E;
  a.k = s.k;
  a.nb = balance_blocks(s.T, s.E, &a.rows_per_block);
  a.part = reinterpret_cast<ColPart*>(base + lay.part);
  a.zpart = reinterpret_cast<double*>(base + lay.zpart);
  a.npart = reinterpret_cast<int*>(base + lay.npart);
  a.joined = reinterpret_cast<unsigned long long*>(base + lay.joined);
  a.counts = counts;
  a.n_tokens = n_tokens;
  a.prob_mean = prob_mean;
  a.losses = losses;
  with_row_shape(balance_geom(s.T, s.E), [&](auto sh) {
    using S = decltype(sh);
    if (a.nb == 1)
      hipLaunchKernelGGL((balance_rows<S, true>), dim3(1), dim3(kThreads), 0, st, a);
    else
      hipLaunchKernelGGL((balance_rows<S, false>), dim3(a.nb), dim3(kThreads), 0,
                         st, a);
  });
  if (a.nb > 1)
    hipLaunchKernelGGL(balance_finish, dim3((s.E + kFinCols - 1) / kFinCols), dim3(kFinThreads), 0,
                       st, a);
  return hipGetLastError();
}

int gate_grad_blocks(const Shape& s) {
  long long rows;
  return gate_blocks(s.T, s.E, &rows);
}

hipError_t gate_grad(const Shape& s, const GateGradArgs& a, int Ep, hipStream_t st) {
  GateGradKernelArgs ka{};
  ka.a = a;
  ka.T = s.T;
  ka.E = s.E;
  ka.k = s.k;
  ka.Ep = Ep;
  ka.blocks = gate_blocks(s.T, s.E, &ka.rows_per_block);
  ka.act_bytes = act_bytes(s);
  const int nb = ka.blocks + (a.pad_src ? s.d / kGradWaves : 0);
  with_row_shape(gate_geom(s.T, s.E), [&](auto sh) {
    using S = decltype(sh);
    hipLaunchKernelGGL((gate_grad_rows<S>), dim3(nb), dim3(kGradThreads), 0, st, ka);
  });
  return hipGetLastError();
}

}  // namespace moe

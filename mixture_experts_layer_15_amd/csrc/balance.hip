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
// Both passes read the [T][E] logits once and are bound by that read; small
// batches by the launches.  A row is held by a group of L lanes (L the
// smallest power of two that covers it, at most a wave), so several short
// rows share a wave and every lane of a load carries a logit.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// A row of E logits on L lanes: lane g holds elements (c L + g) V + v,
// c < C, v < V (V = 4: 16-byte loads, E a multiple of 4).
template <int V, int L, int C>
__device__ __forceinline__ int row_elem(int g, int q) {
  return ((q / V) * L + g) * V + q % V;
}

template <int V, int L, int C>
__device__ __forceinline__ void load_row(const float* row, int E, int g, float (&v)[C * V]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = (c * L + g) * V;
    if constexpr (V == 4) {
      f32x4_t r = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (e < E) r = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c * 4 + i] = r[i];
    } else {
      v[c] = e < E ? row[e] : -INFINITY;
    }
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

// Logits -> softmax in place; returns the log-sum-exp.  A row of -inf only
// gives p = 0 and 0; a NaN or +inf makes the whole row NaN (the maximum drops
// NaN, the sum does not).  The exponential is the hardware one: its argument
// is at most 0, and its absolute error is below 2^-22 of the largest term.
template <int Q, int L>
__device__ __forceinline__ float row_softmax(float (&v)[Q]) {
  float m = v[0];
#pragma unroll
  for (int q = 1; q < Q; ++q) m = fmaxf(m, v[q]);
  m = group_max<L>(m);
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    v[q] = __expf(v[q] - base);
    s += v[q];
  }
  s = group_sum<L>(s);
  const bool dead = s == 0.0f;
  const float inv = dead ? 0.0f : 1.0f / s;
#pragma unroll
  for (int q = 0; q < Q; ++q) v[q] *= inv;
  return dead ? 0.0f : base + logf(s);
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
  int* ticket;     // arrivals of the second kernel, cleared by the first
  double* lpart;   // [E / 32] the second kernel's sums of counts * P
  int32_t* counts;
  int32_t* n_tokens;
  float* prob_mean;
  float* losses;
  int nb;
};

// Sum of a double over the workgroup (fixed order); every thread gets it.
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  const int w = threadIdx.x / kWave;
  __syncthreads();
  if (lane_id() == 0) lds[w] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < (int)blockDim.x / kWave; ++i) s += lds[i];
  return s;
}

// First pass: workgroup b sums the softmax rows, the squared log-sum-exps and
// the slots per expert of its consecutive rows.  kSolo: the only workgroup,
// which also forms the results.
template <int V, int L, int C, bool kSolo>
__global__ __launch_bounds__(kThreads) void balance_rows(BalanceArgs a) {
  constexpr int Q = C * V;
  constexpr int R = kWave / L;  // rows of a wave
  __shared__ float red[kThreads * Q];
  __shared__ int hist[kMaxExperts];
  __shared__ double wsum[kWaves];
  const int tid = threadIdx.x;
  const int w = tid / kWave, l = tid % kWave;
  const int g = l % L, r = l / L;
  const long long t0 = blockIdx.x * a.rows_per_block;
  const long long t1 = min(t0 + a.rows_per_block, a.T);
  for (int e = tid; e < a.E; e += kThreads) hist[e] = 0;
  if (!kSolo && blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  __syncthreads();
  // slots per expert: integer sums, so the order of the atomics is free
  for (long long s = t0 * a.k + tid; s < t1 * a.k; s += kThreads) {
    if (a.mask && a.mask[s / a.k] == 0) continue;
    const int e = a.idx[s];
    if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
  }
  float acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = 0.0f;
  double z = 0.0;
  int n = 0;
  for (long long t = t0 + w * R + r; t < t1; t += kWaves * R) {
    if (a.mask && a.mask[t] == 0) continue;  // the same for the group's lanes
    float v[Q];
    load_row<V, L, C>(a.logits + t * a.E, a.E, g, v);
    const float lse = row_softmax<Q, L>(v);
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] += v[q];
    if (g == 0) {
      z += (double)lse * lse;
      ++n;
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) red[((w * R + r) * Q + q) * L + g] = acc[q];
  const double zsum = block_sum(z, wsum);
  const int nsum = (int)block_sum((double)n, wsum);
  double bal = 0.0;
  const double inv_n = nsum > 0 ? 1.0 / nsum : 0.0;
  for (int e = tid; e < a.E; e += kThreads) {
    const int q = e / (L * V) * V + e % V, gg = e / V % L;
    double s = 0.0;
    for (int i = 0; i < kWaves * R; ++i) s += red[(i * Q + q) * L + gg];
    if constexpr (kSolo) {
      a.counts[e] = hist[e];
      a.prob_mean[e] = (float)(s * inv_n);
      bal += hist[e] * (s * inv_n);
    } else {
      a.part[(size_t)blockIdx.x * a.E + e] = ColPart{(float)s, hist[e]};
    }
  }
  if constexpr (kSolo) {
    bal = block_sum(bal, wsum);
    if (tid == 0) {
      *a.n_tokens = nsum;
      a.losses[0] = (float)(bal * a.E / a.k * inv_n);
      a.losses[1] = (float)(zsum * inv_n);
    }
  } else if (tid == 0) {
    a.zpart[blockIdx.x] = zsum;
    a.npart[blockIdx.x] = nsum;
  }
}

// Second pass: workgroup j adds the partial sums of 32 experts (32 threads
// abreast, 32 partials at a time) in a fixed order; the last one to arrive
// adds the workgroups' shares of the loss, again in a fixed order.
constexpr int kFinThreads = 1024;
constexpr int kFinCols = 32;

__global__ __launch_bounds__(kFinThreads) void balance_finish(BalanceArgs a) {
  constexpr int kRows = kFinThreads / kFinCols;
  __shared__ double sp[kRows][kFinCols];
  __shared__ int sc[kRows][kFinCols];
  __shared__ double wsum[kFinThreads / kWave];
  __shared__ bool last;
  const int tid = threadIdx.x;
  const int j = tid % kFinCols, r = tid / kFinCols;
  const int e = blockIdx.x * kFinCols + j;
  double p = 0.0;
  int c = 0;
  if (e < a.E) {
    for (int b = r; b < a.nb; b += kRows) {
      const ColPart v = a.part[(size_t)b * a.E + e];
      p += v.p;
      c += v.c;
    }
  }
  sp[r][j] = p;
  sc[r][j] = c;
  int n = 0;
  double z = 0.0;
  for (int b = tid; b < a.nb; b += kFinThreads) {
    n += a.npart[b];
    z += a.zpart[b];
  }
  const int nsum = (int)block_sum((double)n, wsum);
  const double zsum = block_sum(z, wsum);
  const double inv_n = nsum > 0 ? 1.0 / nsum : 0.0;
  double bal = 0.0;
  if (r == 0 && e < a.E) {
    p = 0.0;
    c = 0;
    for (int i = 0; i < kRows; ++i) {
      p += sp[i][j];
      c += sc[i][j];
    }
    a.counts[e] = c;
    a.prob_mean[e] = (float)(p * inv_n);
    bal = c * (p * inv_n);
  }
  bal = block_sum(bal, wsum);
  if (tid == 0) {
    __hip_atomic_store(&a.lpart[blockIdx.x], bal, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           (int)gridDim.x - 1;
    if (last) {
      double s = 0.0;
      for (unsigned i = 0; i < gridDim.x; ++i)
        s += __hip_atomic_load(&a.lpart[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *a.n_tokens = nsum;
      a.losses[0] = (float)(s * a.E / a.k * inv_n);
      a.losses[1] = (float)(zsum * inv_n);
    }
  }
}

// ---- gradient with respect to the logits

struct GateGradKernelArgs {
  GateGradArgs a;
  long long T;
  int E, k, Ep;
  long long rows_per_block;
};

// float32 -> bfloat16 rounding and what it leaves (none of an infinite or
// NaN value, so that it is not turned into another one).
__device__ __forceinline__ uint16_t split_bf16(float& v) {
  const uint16_t h = f32_to_bf16(v);
  const float b = bf16_to_f32(h);
  v = __builtin_isfinite(b) ? v - b : 0.0f;
  return h;
}

// Workgroup b: consecutive rows.  Writes the float32 gradient, its split into
// `nplanes` bfloat16 planes [T][Ep] (their sum is the value: three hold all 24
// bits; columns E .. Ep - 1 are zero), and the workgroup's column sums.
template <int V, int L, int C>
__global__ __launch_bounds__(kThreads) void gate_grad_rows(GateGradKernelArgs ka) {
  constexpr int Q = C * V;
  constexpr int R = kWave / L;
  __shared__ float red[kThreads * Q];
  __shared__ int wtot[kWaves];
  const GateGradArgs& a = ka.a;
  const int E = ka.E, k = ka.k;
  const int tid = threadIdx.x;
  const int w = tid / kWave, l = tid % kWave;
  const int g = l % L, r = l / L;
  const bool losses = a.dlosses != nullptr;
  float cen[Q];  // centred counts
  float ca = 0.0f, cz = 0.0f;
#pragma unroll
  for (int q = 0; q < Q; ++q) cen[q] = 0.0f;
  if (losses) {
    // the sum of the counts, in integers (below 2^31 slots)
    int s = 0;
    for (int e = tid; e < E; e += kThreads) s += a.counts[e];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, kWave);
    if (l == 0) wtot[w] = s;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < kWaves; ++i) total += wtot[i];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = row_elem<V, L, C>(g, q);
      if (e < E) cen[q] = (float)((double)((long long)a.counts[e] * E - total) / E);
    }
    const int n = *a.n_tokens;
    if (n > 0) {
      ca = (float)((double)a.dlosses[0] * E / ((double)n * n * k));
      cz = (float)((double)a.dlosses[1] * 2.0 / n);
    }
  }
  if (blockIdx.x == 0 && tid < kZeroLineBytes / 4)
    reinterpret_cast<uint32_t*>(a.zero_line)[tid] = 0;
  float colsum[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) colsum[q] = 0.0f;
  const long long t0 = blockIdx.x * ka.rows_per_block;
  const long long t1 = min(t0 + ka.rows_per_block, ka.T);
  for (long long t = t0 + w * R + r; t < t1; t += kWaves * R) {
    float v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = 0.0f;
    if (!a.mask || a.mask[t] != 0) {
      if (losses) {
        load_row<V, L, C>(a.logits + t * E, E, g, v);
        const float lse = row_softmax<Q, L>(v);
        float mean = 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q) mean = fmaf(v[q], cen[q], mean);
        mean = group_sum<L>(mean);
        const float zl = cz * lse;
#pragma unroll
        for (int q = 0; q < Q; ++q) v[q] *= fmaf(ca, cen[q] - mean, zl);
      }
      if (a.dtopk_w) {
        const int32_t* id = a.idx + t * k;
        const float* gw = a.topk_w + t * k;
        const float* dg = a.dtopk_w + t * k;
        float mean = 0.0f;
        for (int i = 0; i < k; ++i)
          if ((unsigned)id[i] < (unsigned)E) mean = fmaf(gw[i], dg[i], mean);
        for (int i = 0; i < k; ++i) {
          const int e = id[i];
          const float d = gw[i] * (dg[i] - mean);
#pragma unroll
          for (int q = 0; q < Q; ++q)
            if (e == row_elem<V, L, C>(g, q) && e < E) v[q] += d;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) colsum[q] += v[q];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * L + g) * V;
      if constexpr (V == 4) {
        if (a.dlogits && e < E)
          *reinterpret_cast<f32x4_t*>(a.dlogits + t * E + e) =
              f32x4_t{v[c * 4], v[c * 4 + 1], v[c * 4 + 2], v[c * 4 + 3]};
      } else {
        if (a.dlogits && e < E) a.dlogits[t * E + e] = v[c];
      }
    }
    for (int pl = 0; pl < a.nplanes; ++pl) {
      uint16_t* row = a.planes + ((size_t)pl * ka.T + t) * ka.Ep;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = (c * L + g) * V;
        if constexpr (V == 4) {
          u32x2_t o;
          uint16_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = split_bf16(v[c * 4 + i]);
          o[0] = h[0] | (uint32_t(h[1]) << 16);
          o[1] = h[2] | (uint32_t(h[3]) << 16);
          if (e < E) *reinterpret_cast<u32x2_t*>(row + e) = o;
        } else {
          const uint16_t h = split_bf16(v[c]);
          if (e < E) row[e] = h;
        }
      }
      for (int e = E + g; e < ka.Ep; e += L) row[e] = 0;
    }
  }
  if (!a.bias_part) return;
#pragma unroll
  for (int q = 0; q < Q; ++q) red[((w * R + r) * Q + q) * L + g] = colsum[q];
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) {
    const int q = e / (L * V) * V + e % V, gg = e / V % L;
    double s = 0.0;
    for (int i = 0; i < kWaves * R; ++i) s += red[(i * Q + q) * L + gg];
    a.bias_part[(size_t)blockIdx.x * E + e] = (float)s;
  }
}

// Row groups for E experts: calls f with the lanes, vector width and chunks
// as compile-time constants.
template <int V, int L, int C>
struct RowShape {
  static constexpr int v = V, l = L, c = C;
};

template <class F>
void with_row_shape(int E, F f) {
  if (E % 4 == 0) {
    const int n = E / 4;
    if (n <= 1) return f(RowShape<4, 1, 1>{});
    if (n <= 2) return f(RowShape<4, 2, 1>{});
    if (n <= 4) return f(RowShape<4, 4, 1>{});
    if (n <= 8) return f(RowShape<4, 8, 1>{});
    if (n <= 16) return f(RowShape<4, 16, 1>{});
    if (n <= 32) return f(RowShape<4, 32, 1>{});
    if (n <= 64) return f(RowShape<4, 64, 1>{});
    return f(RowShape<4, 64, 2>{});
  }
  if (E <= 4) return f(RowShape<1, 4, 1>{});
  if (E <= 16) return f(RowShape<1, 16, 1>{});
  if (E <= 32) return f(RowShape<1, 32, 1>{});
  if (E <= 64) return f(RowShape<1, 64, 1>{});
  if (E <= 128) return f(RowShape<1, 64, 2>{});
  if (E <= 256) return f(RowShape<1, 64, 4>{});
  return f(RowShape<1, 64, 8>{});
}

// Workgroups of the row kernels: at least 16 rows each, at most 512.
int row_blocks(long long T, long long* rows_per_block) {
  const long long nb = std::min<long long>(std::max<long long>((T + 15) / 16, 1), 512);
  *rows_per_block = std::max<long long>((T + nb - 1) / nb, 1);
  return (int)std::max<long long>((T + *rows_per_block - 1) / *rows_per_block, 1);
}

struct BalanceLayout {
  size_t part, zpart, npart, ticket, lpart, total;
};

BalanceLayout balance_layout(const Shape& s) {
  BalanceLayout L{};
  long long rows;
  const int nb = row_blocks(s.T, &rows);
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.part = take((size_t)nb * s.E * sizeof(ColPart));
  L.zpart = take((size_t)nb * sizeof(double));
  L.npart = take((size_t)nb * sizeof(int));
  L.ticket = take(sizeof(int));
  L.lpart = take((size_t)((s.E + kFinCols - 1) / kFinCols) * sizeof(double));
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
  a.nb = row_blocks(s.T, &a.rows_per_block);
  a.part = reinterpret_cast<ColPart*>(base + lay.part);
  a.zpart = reinterpret_cast<double*>(base + lay.zpart);
  a.npart = reinterpret_cast<int*>(base + lay.npart);
  a.ticket = reinterpret_cast<int*>(base + lay.ticket);
  a.lpart = reinterpret_cast<double*>(base + lay.lpart);
  a.counts = counts;
  a.n_tokens = n_tokens;
  a.prob_mean = prob_mean;
  a.losses = losses;
  with_row_shape(s.E, [&](auto sh) {
    using S = decltype(sh);
    if (a.nb == 1)
      hipLaunchKernelGGL((balance_rows<S::v, S::l, S::c, true>), dim3(1), dim3(kThreads), 0, st, a);
    else
      hipLaunchKernelGGL((balance_rows<S::v, S::l, S::c, false>), dim3(a.nb), dim3(kThreads), 0,
                         st, a);
  });
  if (a.nb > 1)
    hipLaunchKernelGGL(balance_finish, dim3((s.E + kFinCols - 1) / kFinCols), dim3(kFinThreads), 0,
                       st, a);
  return hipGetLastError();
}

int gate_grad_blocks(const Shape& s) {
  long long rows;
  return row_blocks(s.T, &rows);
}

hipError_t gate_grad(const Shape& s, const GateGradArgs& a, int Ep, hipStream_t st) {
  GateGradKernelArgs ka{};
  ka.a = a;
  ka.T = s.T;
  ka.E = s.E;
  ka.k = s.k;
  ka.Ep = Ep;
  const int nb = row_blocks(s.T, &ka.rows_per_block);
  with_row_shape(s.E, [&](auto sh) {
    using S = decltype(sh);
    hipLaunchKernelGGL((gate_grad_rows<S::v, S::l, S::c>), dim3(nb), dim3(kThreads), 0, st, ka);
  });
  return hipGetLastError();
}

}  // namespace moe

// The norms around the layer, with their backward passes:
//
//   before:  x   = h r(h) w,                     r(v) = 1 / sqrt(mean(v^2) + eps)
//   after:   out = s h + g * (c r(c) w),         c = sum_i gate_i y_i  (the combine)
//            and, of the rounded out, the next block's norm
//
//   before, backward (r saved):  n = h r, u = w dx
//            dh = r (u - n mean(n u)) + s dout,  dw = sum_t dx n
//   after, backward:             n = c r, u = w g dout
//            dc = r (u - n mean(n u)),  dy_i = gate_i dc,  dgate_i = <dc, y_i>
//            dw = g S, dg = w S  with  S = sum_t dout n   (w and g are per channel)
//
// Every kernel gives a row to a group of L threads (one workgroup) that holds
// it, V chunks of 8 columns a thread, so that every array passes HBM once: these
// are HBM-bound passes.  Registers hold all of it up to 16384
// columns, in combine_norm_backward up to 4096 (float32: 44 of them spilled beyond;
// bfloat16 in two passes: 79 beyond 8192); at four chunks a thread up to 166 are
// spilled, at eight up to 555.  Sums are float32 in a fixed order (a
// wave's butterfly, then the waves in order; over tokens each workgroup adds
// its rows in order and a second kernel the workgroups).  Nothing is rounded
// but what is stored.
#include <algorithm>
#include <type_traits>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

// ---- 8 columns of a row
template <bool kBF16>
struct Chunk {
  u32x4_t v[kBF16 ? 1 : 2];
};

template <bool kBF16, bool kStream = false>
__device__ __forceinline__ Chunk<kBF16> load8(const void* base, long long at) {
  Chunk<kBF16> c;
  const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const unsigned char*>(base) +
                                                      at * (kBF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (kBF16 ? 1 : 2); ++i)
    c.v[i] = kStream ? __builtin_nontemporal_load(p + i) : p[i];
  return c;
}

template <bool kBF16>
__device__ __forceinline__ float at8(const Chunk<kBF16>& c, int q) {
  if constexpr (kBF16) {
    const uint32_t u = c.v[0][q >> 1];
    return __uint_as_float(q & 1 ? u & 0xffff0000u : u << 16);
  } else {
    return __uint_as_float(c.v[q >> 2][q & 3]);
  }
}

template <bool kBF16>
__device__ __forceinline__ Chunk<kBF16> pack8(const float* f) {
  Chunk<kBF16> c;
  if constexpr (kBF16) {
    c.v[0] = u32x4_t{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                     bf16_pair(f[6], f[7])};
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) c.v[q >> 2][q & 3] = __float_as_uint(f[q]);
  }
  return c;
}

template <bool kBF16, bool kStream = false>
__device__ __forceinline__ void store8(void* base, long long at, const Chunk<kBF16>& c) {
  u32x4_t* p = reinterpret_cast<u32x4_t*>(static_cast<unsigned char*>(base) + at * (kBF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (kBF16 ? 1 : 2); ++i) {
    if (kStream) __builtin_nontemporal_store(c.v[i], p + i);
    else p[i] = c.v[i];
  }
}

// 8 float32 values of a per-channel vector
__device__ __forceinline__ void vec8(const float* w, int c, float* f) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(w + c);
  const f32x4_t b = *reinterpret_cast<const f32x4_t*>(w + c + 4);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[q] = a[q];
    f[4 + q] = b[q];
  }
}

// Sums of N values over the L threads of the workgroup, the same bits in every
// thread.  Consecutive calls take turns between two halves of `lds`, kHalf
// values a wave each (turn 0, 1, 0, ...): one barrier a call.
template <int L, int kHalf, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* lds, int turn) {
  static_assert(N <= kHalf, "a half holds the waves' sums");
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if constexpr (L > kWave) {
    constexpr int kW = L / kWave;
    float* at = lds + turn * (kW * kHalf);
    if (lane_id() == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) at[(threadIdx.x / kWave) * N + n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = at[n];
#pragma unroll
      for (int w = 1; w < kW; ++w) v[n] += at[w * N + n];
    }
  }
}

// Sums of the first N of v (a power of two) over the wave: lane l ends with one
// of them in v[0], the one whose number it returns.  A step halves the values:
// N + 5 exchanges rather than 6 N.
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

__device__ __forceinline__ float inv_norm(float sum, int d, float eps) {
  return 1.0f / sqrtf(sum / (float)d + eps);
}

// ---- before the layer

struct NormArgs {
  const void* h;
  const float* weight;
  void* x;
  float* rstd;  // or null
  int d;
  float eps;
};

// (8192 x 7168: 43 us, 5.4 TB/s; 64 x 2048: 2.8 us.)
template <bool kBF16, int L, int V>
__global__ __launch_bounds__(L) void norm_kernel(NormArgs a) {
  __shared__ float lds[2 * (L / kWave)];
  const long long row = (long long)blockIdx.x * a.d;
  Chunk<kBF16> h[V];
  float s[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * L + threadIdx.x) * 8;
    if (c < a.d) h[j] = load8<kBF16>(a.h, row + c);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if ((j * L + (int)threadIdx.x) * 8 < a.d) {
#pragma unroll
      for (int q = 0; q < 8; ++q) s[0] = fmaf(at8(h[j], q), at8(h[j], q), s[0]);
    }
  }
  group_sum<L, 1>(s, lds, 0);
  const float r = inv_norm(s[0], a.d, a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[blockIdx.x] = r;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * L + threadIdx.x) * 8;
    if (c < a.d) {
      float w[8], o[8];
      vec8(a.weight, c, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = at8(h[j], q) * r * w[q];
      store8(a.x, row + c, pack8<kBF16>(o));
    }
  }
}

struct NormGradArgs {
  const void* dx;
  const void* h;
  const float* weight;
  const float* rstd;
  const void* dout;  // or null
  float res_scale;
  void* dh;          // or null
  float* part;       // [gridDim.x][d] column sums of a workgroup's rows, or null
  int T, d;
};

// A workgroup walks rows blockIdx.x, + gridDim.x, ...; the next row is loaded
// before the present one is reduced.  (16384 x 7168 with dout: 179 us, 5.2 TB/s,
// and 6 us for the column sums.)
template <bool kBF16, int L, int V>
__global__ __launch_bounds__(L) void norm_backward_kernel(NormGradArgs a) {
  __shared__ float lds[2 * (L / kWave)];
  // (as far as the registers of 1024 threads hold two rows)
  constexpr bool kAhead = L < 1024 || V * (kBF16 ? 1 : 2) <= 2;
  Chunk<kBF16> dx[V], h[V], dout[V];
  float r = 0.0f;
  auto load = [&](int t) {
    const long long row = (long long)t * a.d;
    r = a.rstd[t];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        dx[j] = load8<kBF16, true>(a.dx, row + c);
        h[j] = load8<kBF16, true>(a.h, row + c);
        if (a.dout) dout[j] = load8<kBF16, true>(a.dout, row + c);
      }
    }
  };
  float acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[j][q] = 0.0f;
  if constexpr (kAhead) load(blockIdx.x);
  int turn = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const long long row = (long long)t * a.d;
    if constexpr (!kAhead) load(t);
    Chunk<kBF16> cdx[V], ch[V], cdo[V];
    const float cr = r;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      cdx[j] = dx[j];
      ch[j] = h[j];
      cdo[j] = dout[j];
    }
    if (kAhead && t + (int)gridDim.x < a.T) load(t + gridDim.x);
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        float w[8];
        vec8(a.weight, c, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float n = at8(ch[j], q) * cr, g = at8(cdx[j], q);
          s[0] = fmaf(n, g * w[q], s[0]);
          acc[j][q] = fmaf(g, n, acc[j][q]);
        }
      }
    }
    if (a.dh == nullptr) continue;  // (the same for every thread)
    group_sum<L, 1>(s, lds, turn);
    const float m = s[0] / (float)a.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        float w[8], o[8];
        vec8(a.weight, c, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float n = at8(ch[j], q) * cr;
          o[q] = cr * (at8(cdx[j], q) * w[q] - n * m);
          if (a.dout) o[q] = fmaf(a.res_scale, at8(cdo[j], q), o[q]);
        }
        store8<kBF16, true>(a.dh, row + c, pack8<kBF16>(o));
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        float* p = a.part + (long long)blockIdx.x * a.d + c;
        *reinterpret_cast<f32x4_t*>(p) = f32x4_t{acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
        *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{acc[j][4], acc[j][5], acc[j][6], acc[j][7]};
      }
    }
  }
}

// ---- after the layer

constexpr int kBatch = 8;  // slots whose rows are in flight together

// Positions and gates of slots i0 .. i0 + N - 1 of token t; -1: not kept.
template <int N>
__device__ __forceinline__ void slots8(const int32_t* pos, const float* w, long long t, int k,
                                       int i0, long long S, int (&p)[N], float (&g)[N]) {
#pragma unroll
  for (int b = 0; b < N; ++b) {
    const long long s = t * k + i0 + b;
    p[b] = -1;
    g[b] = 1.0f;
    if (i0 + b < k) {
      p[b] = pos ? pos[s] : (int)t;
      if (p[b] >= S) p[b] = -1;
      if (w) g[b] = w[s];
    }
  }
}

template <bool kBF16, int N>
__device__ __forceinline__ void rows8(const void* y, const int (&p)[N], int d, int c,
                                      Chunk<kBF16> (&raw)[N]) {
#pragma unroll
  for (int b = 0; b < N; ++b)
    if (p[b] >= 0) raw[b] = load8<kBF16, true>(y, (long long)p[b] * d + c);
}

template <bool kBF16, int N>
__device__ __forceinline__ void add8(const Chunk<kBF16> (&raw)[N], const int (&p)[N],
                                     const float (&g)[N], float* acc) {
#pragma unroll
  for (int b = 0; b < N; ++b) {
    if (p[b] < 0) continue;
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = fmaf(at8(raw[b], q), g[b], acc[q]);
  }
}

struct CombineNormArgs {
  const void* y;
  const int32_t* pos;   // null: row t of y is token t's
  const float* topk_w;  // or null
  const void* h;
  const float* weight;
  const float* gate;    // or null
  void* out;
  float* rstd;          // or null
  const float* next_weight;  // or null
  void* next_x;
  float* next_rstd;     // or null
  long long S;
  int d, k;
  float eps, res_scale;
};

// (8192 x 2048, k = 8, 369 MB: 68 us, 5.4 TB/s; with stores into the cache, where
// they displace the expert rows still to be read, 73.)
template <bool kBF16, int L, int V>
__global__ __launch_bounds__(L) void combine_norm_kernel(CombineNormArgs a) {
  __shared__ float lds[2 * (L / kWave)];
  const long long t = blockIdx.x, row = t * a.d;
  float acc[V][8];
  Chunk<kBF16> h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[j][q] = 0.0f;
    const int c = (j * L + threadIdx.x) * 8;
    if (c < a.d) h[j] = load8<kBF16>(a.h, row + c);
  }
  for (int i0 = 0; i0 < a.k; i0 += kBatch) {
    int p[kBatch];
    float g[kBatch];
    slots8<kBatch>(a.pos, a.topk_w, t, a.k, i0, a.S, p, g);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        Chunk<kBF16> raw[kBatch];
        rows8<kBF16, kBatch>(a.y, p, a.d, c, raw);
        add8<kBF16, kBatch>(raw, p, g, acc[j]);
      }
    }
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int q = 0; q < 8; ++q) s[0] = fmaf(acc[j][q], acc[j][q], s[0]);
  group_sum<L, 1>(s, lds, 0);
  const float r = inv_norm(s[0], a.d, a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[t] = r;
  s[0] = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * L + threadIdx.x) * 8;
    if (c < a.d) {
      float w[8], o[8];
      vec8(a.weight, c, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = acc[j][q] * r * w[q];
      if (a.gate) {
        vec8(a.gate, c, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] *= w[q];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = fmaf(a.res_scale, at8(h[j], q), o[q]);
      h[j] = pack8<kBF16>(o);
      store8<kBF16, true>(a.out, row + c, h[j]);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[0] = fmaf(at8(h[j], q), at8(h[j], q), s[0]);
    }
  }
  if (a.next_weight == nullptr) return;
  group_sum<L, 1>(s, lds, 1);
  const float rn = inv_norm(s[0], a.d, a.eps);
  if (a.next_rstd && threadIdx.x == 0) a.next_rstd[t] = rn;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * L + threadIdx.x) * 8;
    if (c < a.d) {
      float w[8], o[8];
      vec8(a.next_weight, c, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = at8(h[j], q) * rn * w[q];
      store8<kBF16, true>(a.next_x, row + c, pack8<kBF16>(o));
    }
  }
}

struct CombineNormGradArgs {
  const void* dout;
  const void* y;
  const int32_t* pos;   // null: row t of y is token t's
  const float* topk_w;  // or null
  const float* weight;
  const float* rstd;
  const float* gate;    // or null
  void* dy;             // or null
  float* dtopk_w;       // or null
  float* part;          // [gridDim.x][d] column sums of dout n, or null
  long long S;
  int T, d, k;
};

// Slots whose rows are in flight together in the backward pass: what 1024 threads
// have registers for beside the row.  (1463 x 11136, k = 2: float32 355 -> 84 us,
// bfloat16 145 -> 48; with k = 8, whose rows are then read twice, 429 -> 261 and
// 151 -> 173.)
constexpr int batch_of(bool bf16, int threads) { return threads < 1024 ? kBatch : bf16 ? 4 : 2; }

// One pass over the y rows where the slots are a batch (kOne): with a chunk's rows in registers
// its c is complete, so <u, r y_i> and <n, r y_i> are summed at once and
//    <dc, y_i> = <u, r y_i> - mean(n u) <n, r y_i>
// needs no second look at y.  (Terms of the result's size: <c, y_i> leaves the
// float32 range where a large y_i meets a small gate.)  More slots read y twice, the
// second time from a cache.
// Narrow bfloat16 rows keep to 128 registers: four workgroups of 256 a compute
// unit, which hide each other's loads (4099 x 2048, k = 8, of 286 MB: 75 -> 64.6
// us; 6 registers are spilled for it, 30 to 37 in two passes).  Wider rows do not fit there: held to 168 registers 8192 x 4096, k = 4
// takes 190 us rather than 154.
template <bool kBF16, int L, int V, bool kOne>
__global__ __launch_bounds__(L, kBF16&& V == 1 && L <= 256 ? 4 : 1) void combine_norm_backward_kernel(
    CombineNormGradArgs a) {
  constexpr int kB = batch_of(kBF16, L);
  constexpr int kPairs = 2 * kB;  // <u, r y_i> and <n, r y_i>
  constexpr int kSums = kOne ? 1 + kPairs : kB;
  constexpr int kW = L / kWave;
  __shared__ float lds[2 * kW * kSums];
  float acc[V][8];  // column sums over the workgroup's rows
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[j][q] = 0.0f;
  int turn = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const long long row = t * a.d;
    const float r = a.rstd[t];
    float cc[V][8], u[V][8];  // c, then n, then dc; u
    float s[1] = {0.0f}, e[kOne ? kPairs : 1];
#pragma unroll
    for (int n = 0; n < (kOne ? kPairs : 1); ++n) e[n] = 0.0f;
    int p[kB];
    float g[kB];
    if constexpr (kOne) slots8<kB>(a.pos, a.topk_w, t, a.k, 0, a.S, p, g);
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int q = 0; q < 8; ++q) cc[j][q] = u[j][q] = 0.0f;
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        const Chunk<kBF16> go = load8<kBF16>(a.dout, row + c);
        Chunk<kBF16> raw[kB];
        if constexpr (kOne) {
          rows8<kBF16, kB>(a.y, p, a.d, c, raw);
          add8<kBF16, kB>(raw, p, g, cc[j]);
        } else {
          for (int i0 = 0; i0 < a.k; i0 += kB) {
            slots8<kB>(a.pos, a.topk_w, t, a.k, i0, a.S, p, g);
            rows8<kBF16, kB>(a.y, p, a.d, c, raw);
            add8<kBF16, kB>(raw, p, g, cc[j]);
          }
        }
        float w[8], f[8];
        vec8(a.weight, c, w);
        if (a.gate) vec8(a.gate, c, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float o = at8(go, q), n = cc[j][q] * r;
          u[j][q] = w[q] * (a.gate ? o * f[q] : o);
          s[0] = fmaf(n, u[j][q], s[0]);
          acc[j][q] = fmaf(o, n, acc[j][q]);
          cc[j][q] = n;
        }
        if constexpr (kOne) {
          if (a.dtopk_w) {
#pragma unroll
            for (int b = 0; b < kB; ++b) {
              if (p[b] < 0) continue;
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float v = r * at8(raw[b], q);
                e[2 * b] = fmaf(u[j][q], v, e[2 * b]);
                e[2 * b + 1] = fmaf(cc[j][q], v, e[2 * b + 1]);
              }
            }
          }
        }
      }
    }
    if constexpr (kOne) {
      float* at = lds + turn * (kW * kSums);
      const int wave = threadIdx.x / kWave;
      s[0] = wave_sum(s[0]);
      if (lane_id() == 0) at[wave * kSums] = s[0];
      if (a.dtopk_w) {
        const int i = wave_sums<kPairs>(e);
        if (lane_id() < kPairs) at[wave * kSums + 1 + i] = e[0];
      }
      __syncthreads();
      s[0] = at[0];
#pragma unroll
      for (int w = 1; w < kW; ++w) s[0] += at[w * kSums];
    } else {
      group_sum<L, kSums>(s, lds, turn);
    }
    const float m = s[0] / (float)a.d;
    if constexpr (kOne) {
      if (a.dtopk_w && (int)threadIdx.x < a.k) {
        const float* at = lds + turn * (kW * kSums) + 1 + 2 * threadIdx.x;
        float uy = at[0], ny = at[1], v = 0.0f;
#pragma unroll
        for (int w = 1; w < kW; ++w) {
          uy += at[w * kSums];
          ny += at[w * kSums + 1];
        }
#pragma unroll
        for (int b = 0; b < kB; ++b)
          if ((int)threadIdx.x == b && p[b] >= 0) v = uy - m * ny;
        a.dtopk_w[t * a.k + threadIdx.x] = v;
      }
    }
    turn ^= 1;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < 8; ++q) cc[j][q] = r * (u[j][q] - cc[j][q] * m);  // dc
    for (int i0 = 0; i0 < a.k; i0 += kB) {
      if constexpr (!kOne) slots8<kB>(a.pos, a.topk_w, t, a.k, i0, a.S, p, g);
      float dot[kB];
#pragma unroll
      for (int b = 0; b < kB; ++b) dot[b] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (j * L + threadIdx.x) * 8;
        if (c >= a.d) continue;
        if constexpr (!kOne) {
          if (a.dtopk_w) {
            Chunk<kBF16> raw[kB];
            rows8<kBF16, kB>(a.y, p, a.d, c, raw);
#pragma unroll
            for (int b = 0; b < kB; ++b) {
              if (p[b] < 0) continue;
#pragma unroll
              for (int q = 0; q < 8; ++q) dot[b] = fmaf(cc[j][q], at8(raw[b], q), dot[b]);
            }
          }
        }
        if (a.dy) {
#pragma unroll
          for (int b = 0; b < kB; ++b) {
            if (p[b] < 0) continue;
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = g[b] * cc[j][q];
            store8<kBF16, true>(a.dy, (long long)p[b] * a.d + c, pack8<kBF16>(o));
          }
        }
      }
      if constexpr (!kOne) {
        if (a.dtopk_w) {
          group_sum<L, kSums>(dot, lds, turn);
          turn ^= 1;
          if ((int)threadIdx.x < kB && i0 + (int)threadIdx.x < a.k) {
            float v = 0.0f;
#pragma unroll
            for (int b = 0; b < kB; ++b)
              if ((int)threadIdx.x == b && p[b] >= 0) v = dot[b];
            a.dtopk_w[t * a.k + i0 + threadIdx.x] = v;
          }
        }
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * L + threadIdx.x) * 8;
      if (c < a.d) {
        float* p = a.part + (long long)blockIdx.x * a.d + c;
        *reinterpret_cast<f32x4_t*>(p) = f32x4_t{acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
        *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{acc[j][4], acc[j][5], acc[j][6], acc[j][7]};
      }
    }
  }
}

// ---- column sums: out0 = f0 * sum of n rows of part, out1 = f1 * that
// (f null: 1; out null: not wanted).  A workgroup takes 16 columns: 4 threads of
// 4 columns, 64 of them over the rows.
__global__ __launch_bounds__(256) void column_sum_kernel(const float* part, int n, int d,
                                                         const float* f0, float* out0,
                                                         const float* f1, float* out1) {
  __shared__ f32x4_t lds[64][4];
  const int cq = threadIdx.x % 4, rr = threadIdx.x / 4;
  const int c = blockIdx.x * 16 + cq * 4;  // d is a multiple of 128
  f32x4_t s = {0, 0, 0, 0};
#pragma unroll 8
  for (int i = rr; i < n; i += 64) s += *reinterpret_cast<const f32x4_t*>(part + (long long)i * d + c);
  lds[rr][cq] = s;
  __syncthreads();
  if (rr >= 8) return;
#pragma unroll
  for (int i = 8; i < 64; i += 8) s += lds[rr + i][cq];
  // (the eight partial sums are lanes 4 apart of the first half wave)
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += __shfl_xor(s[j], o, kWave);
  }
  if (rr > 0) return;
  if (out0) {
    f32x4_t f = {1, 1, 1, 1};
    if (f0) f = *reinterpret_cast<const f32x4_t*>(f0 + c);
    *reinterpret_cast<f32x4_t*>(out0 + c) = s * f;
  }
  if (out1) {
    f32x4_t f = {1, 1, 1, 1};
    if (f1) f = *reinterpret_cast<const f32x4_t*>(f1 + c);
    *reinterpret_cast<f32x4_t*>(out1 + c) = s * f;
  }
}

hipError_t column_sum(const float* part, int n, int d, const float* f0, float* out0,
                      const float* f1, float* out1, hipStream_t st) {
  hipLaunchKernelGGL(column_sum_kernel, dim3(d / 16), dim3(256), 0, st, part, n, d, f0, out0, f1,
                     out1);
  return hipGetLastError();
}

// Threads of a row's group and chunks a thread: a wave up to 1024 columns, 256
// threads up to 4096, 512 up to 8192, 1024 beyond.  (norm_backward at 8192 x
// 7168: 256 threads of four chunks 195 us, 512 of two 181, 1024 of one 184;
// combine_norm_backward at 8192 x 4096: 256 of two 154, 512 of one 186.)
template <typename F>
void with_group(int d, F&& f) {
  using std::integral_constant;
  const int chunks = d / 8;
  auto go = [&](auto L, auto V) { f(L, V); };
  if (chunks <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (chunks <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (chunks <= 256) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (chunks <= 512) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (chunks <= 1024) go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  else if (chunks <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else if (chunks <= 4096) go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  else go(integral_constant<int, 1024>{}, integral_constant<int, 8>{});
}

// Workgroups of a backward kernel: what fills the chip, and no more: each leaves
// a row of partial sums (norm_backward at 8192 x 7168: 512 workgroups 181 + 6 us
// of column sums, 1024 185 + 11).
int grad_blocks(const Shape& s) {
  const int most = s.d <= 1024 ? 2048 : s.d <= 4096 ? 1024 : s.d <= 8192 ? 512 : 256;
  return std::max(1, std::min(most, s.T));
}

}  // namespace

size_t norm_grad_ws_bytes(const Shape& s) {
  return align_up((size_t)grad_blocks(s) * s.d * sizeof(float));
}

hipError_t norm(const Shape& s, const void* h, const float* weight, float eps, void* x, float* rstd,
                hipStream_t st) {
  const NormArgs a{h, weight, x, rstd, s.d, eps};
  with_group(s.d, [&](auto L, auto V) {
    if (s.act == kBF16)
      hipLaunchKernelGGL((norm_kernel<true, L.value, V.value>), dim3(s.T), dim3(L.value), 0, st, a);
    else
      hipLaunchKernelGGL((norm_kernel<false, L.value, V.value>), dim3(s.T), dim3(L.value), 0, st, a);
  });
  return hipGetLastError();
}

hipError_t norm_backward(const Shape& s, const moe_norm_backward_args_t& g, void* ws,
                         hipStream_t st) {
  float* part = g.dweight ? static_cast<float*>(ws) : nullptr;
  const int blocks = grad_blocks(s);
  if (s.T > 0) {
    const NormGradArgs a{g.dx, g.h, g.weight, g.rstd, g.dout, g.res_scale, g.dh, part, s.T, s.d};
    with_group(s.d, [&](auto L, auto V) {
      if (s.act == kBF16)
        hipLaunchKernelGGL((norm_backward_kernel<true, L.value, V.value>), dim3(blocks),
                           dim3(L.value), 0, st, a);
      else
        hipLaunchKernelGGL((norm_backward_kernel<false, L.value, V.value>), dim3(blocks),
                           dim3(L.value), 0, st, a);
    });
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (g.dweight == nullptr) return hipSuccess;
  return column_sum(part, s.T > 0 ? blocks : 0, s.d, nullptr, g.dweight, nullptr, nullptr, st);
}

hipError_t combine_norm(const Shape& s, const moe_combine_norm_args_t& g, hipStream_t st) {
  const CombineNormArgs a{g.y,    g.slot_pos, g.topk_w,      g.h,      g.weight,
                          g.gate, g.out,      g.rstd,        g.next_weight, g.next_x,
                          g.next_rstd, s.S,   s.d,           s.k,      g.eps, g.res_scale};
  with_group(s.d, [&](auto L, auto V) {
    if (s.act == kBF16)
      hipLaunchKernelGGL((combine_norm_kernel<true, L.value, V.value>), dim3(s.T), dim3(L.value), 0,
                         st, a);
    else
      hipLaunchKernelGGL((combine_norm_kernel<false, L.value, V.value>), dim3(s.T), dim3(L.value),
                         0, st, a);
  });
  return hipGetLastError();
}

hipError_t combine_norm_backward(const Shape& s, const moe_combine_norm_backward_args_t& g,
                                 void* ws, hipStream_t st) {
  float* part = g.dweight || g.dgate ? static_cast<float*>(ws) : nullptr;
  const int blocks = grad_blocks(s);
  if (s.T > 0) {
    const CombineNormGradArgs a{g.dout, g.y,  g.slot_pos, g.topk_w, g.weight, g.rstd, g.gate,
                                g.dy,   g.dtopk_w, part,  s.S,      s.T,      s.d,    s.k};
    with_group(s.d, [&](auto L, auto V) {
      auto launch = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3(blocks), dim3(L.value), 0, st, a);
      };
      if (s.act == kBF16) {
        if (s.k <= batch_of(true, L.value)) launch(combine_norm_backward_kernel<true, L.value, V.value, true>);
        else launch(combine_norm_backward_kernel<true, L.value, V.value, false>);
      } else {
        if (s.k <= batch_of(false, L.value)) launch(combine_norm_backward_kernel<false, L.value, V.value, true>);
        else launch(combine_norm_backward_kernel<false, L.value, V.value, false>);
      }
    });
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (part == nullptr) return hipSuccess;
  return column_sum(part, s.T > 0 ? blocks : 0, s.d, g.gate, g.dweight, g.weight, g.dgate, st);
}

}  // namespace moe

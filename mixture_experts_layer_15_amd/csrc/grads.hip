// Global L2 norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors and values of g^2)
//   out  = g * (max_norm / norm)  if norm is finite and above max_norm, else g
//
// The squares are summed in float64 (a float32 value's square always fits),
// so neither large nor small gradients leave the range.  Both passes are
// HBM-bound.
//
// The tensors of a launch travel as a kernel argument (a table of addresses
// and sizes), so nothing is copied to the device and a captured call keeps
// its own table.  The values of all tensors are cut into chunks; a workgroup
// takes every gridDim.x-th chunk and finds its tensor by bisection.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 112;            // tensors of a launch (an argument of at most 4 KB)
constexpr int kChunk = 16384;          // values of a chunk
constexpr int kMaxBlocks = 2048;       // workgroups of a launch

struct Table {
  const void* src[kTable];
  void* dst[kTable];
  long long numel[kTable];
  int chunk_end[kTable];               // chunks of tensors 0 .. i
  uint8_t bf16[kTable];
  int n;
  int chunks;
};
static_assert(sizeof(Table) <= 3600, "kernel argument size");

__device__ __forceinline__ int find_tensor(const Table& t, int chunk) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (chunk < t.chunk_end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Values [b, e) of a tensor of 16-byte vectors of V: the first value at a
// 16-byte address and the whole vectors from there.
__device__ __forceinline__ void vector_range(uintptr_t addr, int size, long long n, int V,
                                             long long* head, long long* vecs) {
  const long long h = (long long)((16 - addr % 16) % 16) / size;
  *head = h < n ? h : n;
  *vecs = (n - *head) / V;
}

__device__ __forceinline__ void add_square(double& s, float v) { s = fma((double)v, (double)v, s); }

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < (int)blockDim.x / kWave; ++i) s += lds[i];
  return s;
}

// part[blockIdx.x] = the sum of squares of the workgroup's chunks; with norm,
// the only workgroup of the only launch writes the result.
__global__ __launch_bounds__(kThreads) void grad_squares(Table t, double* part, float* norm) {
  __shared__ double lds[kThreads / kWave];
  double s = 0.0;
  const int tid = threadIdx.x;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const long long b = (long long)(c - (i ? t.chunk_end[i - 1] : 0)) * kChunk;
    const long long n = min((long long)kChunk, t.numel[i] - b);
    long long head, vecs;
    if (t.bf16[i]) {
      const uint16_t* p = static_cast<const uint16_t*>(t.src[i]) + b;
      vector_range((uintptr_t)p, 2, n, 8, &head, &vecs);
      for (long long q = tid; q < head; q += kThreads) add_square(s, bf16_to_f32(p[q]));
      const u32x4_t* v = reinterpret_cast<const u32x4_t*>(p + head);
#pragma unroll 4
      for (long long q = tid; q < vecs; q += kThreads) {
        const u32x4_t r = v[q];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          add_square(s, bf16_to_f32(uint16_t(r[j])));
          add_square(s, bf16_to_f32(uint16_t(r[j] >> 16)));
        }
      }
      for (long long q = head + vecs * 8 + tid; q < n; q += kThreads) add_square(s, bf16_to_f32(p[q]));
    } else {
      const float* p = static_cast<const float*>(t.src[i]) + b;
      vector_range((uintptr_t)p, 4, n, 4, &head, &vecs);
      for (long long q = tid; q < head; q += kThreads) add_square(s, p[q]);
      const f32x4_t* v = reinterpret_cast<const f32x4_t*>(p + head);
#pragma unroll 4
      for (long long q = tid; q < vecs; q += kThreads) {
        const f32x4_t r = v[q];
#pragma unroll
        for (int j = 0; j < 4; ++j) add_square(s, r[j]);
      }
      for (long long q = head + vecs * 4 + tid; q < n; q += kThreads) add_square(s, p[q]);
    }
  }
  s = block_sum(s, lds);
  if (tid == 0) {
    if (norm) *norm = (float)sqrt(s);
    else part[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(1024) void grad_norm_finish(const double* part, int n, float* norm) {
  __shared__ double lds[1024 / kWave];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

// A product with the scale rounds to float32, then (bf16) to the nearest
// bfloat16.  Scale 1 leaves the value's bits alone, NaN payloads included.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t v, float scale) {
  return pack_bf16x2(bf16_to_f32(uint16_t(v)) * scale, bf16_to_f32(uint16_t(v >> 16)) * scale);
}

__global__ __launch_bounds__(kThreads) void grad_scale(Table t, const float* norm, float max_norm) {
  const float nv = *norm;
  const bool clip = nv > max_norm && nv < INFINITY;
  const float scale = clip ? max_norm / nv : 1.0f;
  const int tid = threadIdx.x;
  // from the end: the norm's pass has left the last chunks in the cache
  for (int c = t.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = find_tensor(t, c);
    if (!clip && t.src[i] == t.dst[i]) continue;  // in place and nothing to change
    const long long b = (long long)(c - (i ? t.chunk_end[i - 1] : 0)) * kChunk;
    const long long n = min((long long)kChunk, t.numel[i] - b);
    long long head, vecs;
    if (t.bf16[i]) {
      const uint16_t* p = static_cast<const uint16_t*>(t.src[i]) + b;
      uint16_t* o = static_cast<uint16_t*>(t.dst[i]) + b;
      vector_range((uintptr_t)p, 2, n, 8, &head, &vecs);
      if (((uintptr_t)p - (uintptr_t)o) % 16 != 0) vecs = 0;  // no common alignment
      auto one = [&](long long q) {
        o[q] = clip ? f32_to_bf16(bf16_to_f32(p[q]) * scale) : p[q];
      };
      for (long long q = tid; q < head; q += kThreads) one(q);
      const u32x4_t* v = reinterpret_cast<const u32x4_t*>(p + head);
      u32x4_t* w = reinterpret_cast<u32x4_t*>(o + head);
#pragma unroll 4
      for (long long q = tid; q < vecs; q += kThreads) {
        u32x4_t r = v[q];
        if (clip)
#pragma unroll
          for (int j = 0; j < 4; ++j) r[j] = scale_bf16x2(r[j], scale);
        w[q] = r;
      }
      for (long long q = head + vecs * 8 + tid; q < n; q += kThreads) one(q);
    } else {
      const float* p = static_cast<const float*>(t.src[i]) + b;
      float* o = static_cast<float*>(t.dst[i]) + b;
      vector_range((uintptr_t)p, 4, n, 4, &head, &vecs);
      if (((uintptr_t)p - (uintptr_t)o) % 16 != 0) vecs = 0;
      auto one = [&](long long q) { o[q] = clip ? p[q] * scale : p[q]; };
      for (long long q = tid; q < head; q += kThreads) one(q);
      const f32x4_t* v = reinterpret_cast<const f32x4_t*>(p + head);
      f32x4_t* w = reinterpret_cast<f32x4_t*>(o + head);
#pragma unroll 4
      for (long long q = tid; q < vecs; q += kThreads) {
        f32x4_t r = v[q];
        if (clip)
#pragma unroll
          for (int j = 0; j < 4; ++j) r[j] *= scale;
        w[q] = r;
      }
      for (long long q = head + vecs * 4 + tid; q < n; q += kThreads) one(q);
    }
  }
}

long long chunks_of(const moe_grad_t& g) { return (g.numel + kChunk - 1) / kChunk; }

// Calls f(table) for one launch after another; empty tensors take no place.
// A table holds at most 2^30 chunks.
template <class F>
void for_tables(const moe_grad_t* g, int n, F f) {
  Table t;
  t.n = 0;
  t.chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (g[i].numel == 0) continue;
    const long long c = chunks_of(g[i]);
    if (t.n == kTable || t.chunks + c > (1LL << 30)) {
      f(t);
      t.n = 0;
      t.chunks = 0;
    }
    t.src[t.n] = g[i].grad;
    t.dst[t.n] = g[i].out;
    t.numel[t.n] = g[i].numel;
    t.bf16[t.n] = g[i].dtype == MOE_BF16;
    t.chunks += (int)c;
    t.chunk_end[t.n] = t.chunks;
    ++t.n;
  }
  if (t.n) f(t);
}

int blocks_of(const Table& t) { return std::min(t.chunks, kMaxBlocks); }

}  // namespace

// Launches and workgroups of a list, as for_tables cuts it.
struct Totals {
  int launches = 0;
  long long blocks = 0;
};

static Totals totals_of(const moe_grad_t* g, int n) {
  Totals r;
  long long chunks = 0;
  int in = 0;
  auto close = [&] {
    if (in == 0) return;
    ++r.launches;
    r.blocks += std::min<long long>(chunks, kMaxBlocks);
  };
  for (int i = 0; i < n; ++i) {
    if (g[i].numel == 0) continue;
    const long long c = chunks_of(g[i]);
    if (in == kTable || chunks + c > (1LL << 30)) {
      close();
      in = 0;
      chunks = 0;
    }
    ++in;
    chunks += c;
  }
  close();
  return r;
}

size_t grad_ws_bytes(const moe_grad_t* g, int n) {
  return align_up((size_t)std::max<long long>(totals_of(g, n).blocks, 1) * sizeof(double));
}

hipError_t grad_norm(const moe_grad_t* g, int n, float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  int used = 0;
  const Totals total = totals_of(g, n);
  const bool solo = total.launches == 1 && total.blocks == 1;
  for_tables(g, n, [&](const Table& t) {
    const int nb = blocks_of(t);
    hipLaunchKernelGGL(grad_squares, dim3(nb), dim3(kThreads), 0, st, t, part + used,
                       solo ? norm : nullptr);
    used += nb;
  });
  if (!solo)
    hipLaunchKernelGGL(grad_norm_finish, dim3(1), dim3(1024), 0, st, part, used, norm);
  return hipGetLastError();
}

hipError_t grad_clip(const moe_grad_t* g, int n, const float* norm, float max_norm,
                     hipStream_t st) {
  hipError_t e = hipSuccess;  // of an empty list
  for_tables(g, n, [&](const Table& t) {
    hipLaunchKernelGGL(grad_scale, dim3(blocks_of(t)), dim3(kThreads), 0, st, t, norm, max_norm);
    e = hipGetLastError();
  });
  return e;
}

}  // namespace moe

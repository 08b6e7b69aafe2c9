// Combine: gate-weighted sum of each token's expert outputs, back in token
// order, without atomics.
//
// "Expert Parallelism for MoE Models" (apxml), section "Mechanics of Token
// Routing and All-to-All Communication": after the expert computes, its output
// is sent back to the token.  out[t] = sum over i of the kept slots t*k + i of
// y[slot_pos[t*k + i]] (times the gate when y is unweighted), accumulated in
// float32 in increasing i and rounded once.  A token with no kept slot gets 0.
//
// One workgroup per token row; each thread owns 8 consecutive columns (one
// 16-byte bf16 chunk, or two 16-byte float32 chunks), so every y row is read
// with full-width coalesced loads.  With k <= 8 a token's slot positions and
// gates are loaded once for all its columns, and a token without a local slot
// only writes zeros.  The pass is HBM-bound; bf16 rows are read and written
// with nontemporal accesses (each byte is touched once: measured 55 -> 48 us
// on the Qwen3 prefill's 268 MB of expert outputs).
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMaxThreads = 256;  // 8 columns per thread; 256 or 128 threads

// Accumulate the rows of slots t*k + i0 .. + kBatch - 1 (those with pos >= 0)
// into acc, in increasing i; every row load of the batch is issued first.
template <bool kBF16, int kBatch>
__device__ __forceinline__ void combine_batch(const void* y, const int* pos, const float* gw,
                                              int d, int c0, float* acc) {
  u32x4_t raw[kBatch][kBF16 ? 1 : 2];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (pos[b] < 0) continue;
    if constexpr (kBF16) {
      raw[b][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(
          static_cast<const uint16_t*>(y) + (long long)pos[b] * d + c0));
    } else {
      const float* yr = static_cast<const float*>(y) + (long long)pos[b] * d + c0;
      raw[b][0] = *reinterpret_cast<const u32x4_t*>(yr);
      raw[b][1] = *reinterpret_cast<const u32x4_t*>(yr + 4);
    }
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (pos[b] < 0) continue;
    if constexpr (kBF16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t u = raw[b][0][q];
        acc[2 * q] = fmaf(bf16_to_f32(uint16_t(u & 0xffff)), gw[b], acc[2 * q]);
        acc[2 * q + 1] = fmaf(bf16_to_f32(uint16_t(u >> 16)), gw[b], acc[2 * q + 1]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = fmaf(__uint_as_float(raw[b][q >> 2][q & 3]), gw[b], acc[q]);
    }
  }
}

template <bool kBF16>
__device__ __forceinline__ void combine_store(void* out, long long t, int d, int c0,
                                              const float* acc) {
  if constexpr (kBF16) {
    __builtin_nontemporal_store(
        u32x4_t{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])},
        reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + t * d + c0));
  } else {
    float* orow = static_cast<float*>(out) + t * d + c0;
    *reinterpret_cast<f32x4_t*>(orow) = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
    *reinterpret_cast<f32x4_t*>(orow + 4) = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
  }
}

template <bool kBF16>
__global__ __launch_bounds__(kMaxThreads) void combine_kernel(const void* y, const int32_t* slot_pos,
                                                           const float* topk_w, void* out, int d,
                                                           int k) {
  const long long t = blockIdx.x;
  constexpr int kBatch = 8;  // slots whose rows are loaded together
  if (k <= kBatch) {
    // the token's slot positions and gates, loaded once for all its columns
    int pos[kBatch];
    float gw[kBatch];
    bool any = false;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      pos[b] = b < k ? slot_pos[t * k + b] : -1;
      gw[b] = (b < k && topk_w) ? topk_w[t * k + b] : 1.0f;
      any = any || pos[b] >= 0;
    }
    for (int c0 = threadIdx.x * 8; c0 < d; c0 += blockDim.x * 8) {
      float acc[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = 0.f;
      if (any) combine_batch<kBF16, kBatch>(y, pos, gw, d, c0, acc);
      combine_store<kBF16>(out, t, d, c0, acc);
    }
    return;
  }
  for (int c0 = threadIdx.x * 8; c0 < d; c0 += blockDim.x * 8) {
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
    for (int i0 = 0; i0 < k; i0 += kBatch) {
      int pos[kBatch];
      float gw[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const long long s = t * k + i0 + b;
        pos[b] = i0 + b < k ? slot_pos[s] : -1;
        gw[b] = (i0 + b < k && topk_w) ? topk_w[s] : 1.0f;
      }
      combine_batch<kBF16, kBatch>(y, pos, gw, d, c0, acc);
    }
    combine_store<kBF16>(out, t, d, c0, acc);
  }
}

// ---- backward:  dy[pos] = w dout[t],  dw[t][i] = <dout[t], y[pos]>
//
// L lanes per slot (a wave, less where a row has fewer 16-byte chunks): they
// read their token's dout row (the slots of a token are neighbours, so all but
// the first find it in a cache) and their y row, four chunks of a lane at a
// time, write their dy row, and sum the product in float32 with a fixed
// butterfly.  Every y and dy byte is touched once: HBM-bound (8192 tokens of
// 2048, k = 8, bf16: 105 us, 5.4 TB/s; a 2 GiB copy reaches 4.8 TB/s).
struct CombineGradArgs {
  const void* dout;
  const void* y;       // null: no dw
  const int32_t* pos;
  const float* w;      // null: 1
  void* dy;            // null: no dy
  float* dw;           // null: no dw
  long long S;
  int d, k;
};

template <bool kBF16, int L>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(CombineGradArgs a) {
  constexpr int kSize = kBF16 ? 2 : 4;
  constexpr int V = 16 / kSize;  // values of a chunk
  constexpr int U = 4;           // chunks of a lane in flight
  const int g = threadIdx.x % L;
  const long long block = (long long)blockIdx.y * gridDim.x + blockIdx.x;
  const long long s = block * (kMaxThreads / L) + threadIdx.x / L;
  if (s >= a.S) return;  // whole groups
  const int p = a.pos[s];
  if (p < 0 || p >= a.S) {
    if (a.dw && g == 0) a.dw[s] = 0.0f;
    return;
  }
  const float w = a.w ? a.w[s] : 1.0f;
  const unsigned char* din = static_cast<const unsigned char*>(a.dout) + s / a.k * a.d * kSize;
  const unsigned char* yin = static_cast<const unsigned char*>(a.y) + (long long)p * a.d * kSize;
  unsigned char* dyo = static_cast<unsigned char*>(a.dy) + (long long)p * a.d * kSize;
  float dot = 0.0f;
  for (int c0 = g * V; c0 < a.d; c0 += U * L * V) {
    u32x4_t gv[U], yv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * L * V;
      gv[u] = yv[u] = u32x4_t{0, 0, 0, 0};
      if (c < a.d) {
        gv[u] = *reinterpret_cast<const u32x4_t*>(din + c * kSize);
        if (a.dw)
          yv[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(yin + c * kSize));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * L * V;
      u32x4_t o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (kBF16) {
          const float lo = bf16_to_f32(uint16_t(gv[u][q])), hi = bf16_to_f32(uint16_t(gv[u][q] >> 16));
          dot = fmaf(lo, bf16_to_f32(uint16_t(yv[u][q])), dot);
          dot = fmaf(hi, bf16_to_f32(uint16_t(yv[u][q] >> 16)), dot);
          o[q] = pack_bf16x2(w * lo, w * hi);
        } else {
          const float x = __uint_as_float(gv[u][q]);
          dot = fmaf(x, __uint_as_float(yv[u][q]), dot);
          o[q] = __float_as_uint(w * x);
        }
      }
      if (a.dy && c < a.d)
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(dyo + c * kSize));
    }
  }
  if (a.dw) {
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) dot += __shfl_xor(dot, o, kWave);
    if (g == 0) a.dw[s] = dot;
  }
}

template <bool kBF16, int L>
void launch_combine_backward(const CombineGradArgs& a, hipStream_t st) {
  constexpr int per = kMaxThreads / L;
  const long long blocks = (a.S + per - 1) / per;
  // one dimension of a launch has fewer than 2^32 threads, 2^31 slots need more
  const long long nx = std::min(blocks, 1LL << 22), ny = (blocks + nx - 1) / nx;
  hipLaunchKernelGGL((combine_backward_kernel<kBF16, L>), dim3((unsigned)nx, (unsigned)ny),
                     dim3(kMaxThreads), 0, st, a);
}

}  // namespace

hipError_t combine_backward(const Shape& s, const void* dout, const void* y,
                            const int32_t* slot_pos, const float* topk_w, void* dy,
                            float* dtopk_w, hipStream_t st) {
  const CombineGradArgs a{dout, y, slot_pos, topk_w, dy, dtopk_w, s.S, s.d, s.k};
  const int chunks = s.d * act_bytes(s) / 16;  // of a row: at least 16
  if (s.act == kBF16) {
    if (chunks >= 64) launch_combine_backward<true, 64>(a, st);
    else if (chunks >= 32) launch_combine_backward<true, 32>(a, st);
    else launch_combine_backward<true, 16>(a, st);
  } else {
    if (chunks >= 64) launch_combine_backward<false, 64>(a, st);
    else launch_combine_backward<false, 32>(a, st);
  }
  return hipGetLastError();
}

hipError_t combine(const Shape& s, const void* y, const int32_t* slot_pos, const float* topk_w,
                   void* out, hipStream_t st) {
  if (s.T == 0) return hipSuccess;
  // whole passes over the row: 256 threads when d is a multiple of 2048, else
  // 128 (d / 8 is a multiple of 16)
  const int threads = (s.d % 2048) == 0 ? 256 : 128;
  if (s.act == kBF16)
    hipLaunchKernelGGL(combine_kernel<true>, dim3(s.T), dim3(threads), 0, st, y, slot_pos, topk_w,
                       out, s.d, s.k);
  else
    hipLaunchKernelGGL(combine_kernel<false>, dim3(s.T), dim3(threads), 0, st, y, slot_pos,
                       topk_w, out, s.d, s.k);
  return hipGetLastError();
}

}  // namespace moe

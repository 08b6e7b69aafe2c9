// The router's backward pass: from the gradient of the logits (balance.hip)
// to the router matrix, the bias and the tokens.
//
//   dW_r[c][e] = sum_t x[t][c] dL[t][e]
//   dx[t][c]   = sum_e dL[t][e] W_r[c][e]
//   db[e]      = sum_t dL[t][e]
//
// bf16 activations: dL (float32) is split into bfloat16 planes whose sum is
// the value (gate_grad).  The router matrix' gradient is float32, so it takes
// all three planes: the products with the bfloat16 tokens are exact and only
// the float32 sums round.  The tokens' gradient is rounded to bfloat16 at the
// end, so two planes (16 bits, 2^-17 off) do for it.
// float32 activations: both products on the float32 matrix instructions.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kXcds = 8;
constexpr int kThreads = 256;

// Consecutive workgroups run on consecutive XCDs: gives each XCD one run of
// consecutive items, so that items that share operands share an L2.
// Launched with xcd_grid(items) workgroups; -1: nothing to do.
__device__ __forceinline__ int xcd_item(int items) {
  const int per = (items + kXcds - 1) / kXcds;
  const int i = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  return (int)(blockIdx.x / kXcds) < per && i < items ? i : -1;
}
int xcd_grid(int items) { return (items + kXcds - 1) / kXcds * kXcds; }

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Barrier that orders LDS accesses of the wave's own instruction stream only:
// the loads of the next stage stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 bytes per lane, global -> LDS: lane i's land at lds + 16 i.
__device__ __forceinline__ void dma16(const void* src, unsigned char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
#else
  (void)src;
  (void)lds;
#endif
}

// LDS address of a shared-memory pointer.
__device__ __forceinline__ uint32_t lds_addr(const unsigned char* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) unsigned char*)p;
}

// Transposing LDS reads (ds_read_b64_tr_b16) of one 16-deep step: of 16
// lanes, lane j gives the address of four 16-bit values of row j / 4, columns
// 4 (j % 4) .. + 3, and gets column j of the four rows.  Two reads, four rows
// apart, make the eight K values of an MFMA operand.  One statement issues
// all reads of a step and waits for them: the builtin would make the compiler
// wait for the next stage's global loads as well (they write LDS).
//   x: MB blocks at ax[m];  p: three planes of NB blocks at ap[n]
template <int MB, int NB>
struct StepRegs {
  u32x2_t x[MB][2];
  u32x2_t p[3][NB][2];
};

#define MOE_TR(D, A, OFF) "ds_read_b64_tr_b16 %" #D ", %" #A " offset:" #OFF "\n\t"

// rows of 256 bytes of both operands; a plane is 8192 bytes
__device__ __forceinline__ void read_step(StepRegs<2, 2>& r, const uint32_t (&ax)[2],
                                          const uint32_t (&ap)[2]) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile(
      MOE_TR(0, 16, 0) MOE_TR(1, 16, 1024) MOE_TR(2, 17, 0) MOE_TR(3, 17, 1024)
      MOE_TR(4, 18, 0) MOE_TR(5, 18, 1024) MOE_TR(6, 19, 0) MOE_TR(7, 19, 1024)
      MOE_TR(8, 18, 8192) MOE_TR(9, 18, 9216) MOE_TR(10, 19, 8192) MOE_TR(11, 19, 9216)
      MOE_TR(12, 18, 16384) MOE_TR(13, 18, 17408) MOE_TR(14, 19, 16384) MOE_TR(15, 19, 17408)
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r.x[0][0]), "=&v"(r.x[0][1]), "=&v"(r.x[1][0]), "=&v"(r.x[1][1]),
        "=&v"(r.p[0][0][0]), "=&v"(r.p[0][0][1]), "=&v"(r.p[0][1][0]), "=&v"(r.p[0][1][1]),
        "=&v"(r.p[1][0][0]), "=&v"(r.p[1][0][1]), "=&v"(r.p[1][1][0]), "=&v"(r.p[1][1][1]),
        "=&v"(r.p[2][0][0]), "=&v"(r.p[2][0][1]), "=&v"(r.p[2][1][0]), "=&v"(r.p[2][1][1])
      : "v"(ax[0]), "v"(ax[1]), "v"(ap[0]), "v"(ap[1])
      : "memory");
#endif
}

// x rows of 256 bytes, plane rows of 128; a plane is 4096 bytes
__device__ __forceinline__ void read_step(StepRegs<1, 2>& r, const uint32_t (&ax)[1],
                                          const uint32_t (&ap)[2]) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile(
      MOE_TR(0, 14, 0) MOE_TR(1, 14, 1024)
      MOE_TR(2, 15, 0) MOE_TR(3, 15, 512) MOE_TR(4, 16, 0) MOE_TR(5, 16, 512)
      MOE_TR(6, 15, 4096) MOE_TR(7, 15, 4608) MOE_TR(8, 16, 4096) MOE_TR(9, 16, 4608)
      MOE_TR(10, 15, 8192) MOE_TR(11, 15, 8704) MOE_TR(12, 16, 8192) MOE_TR(13, 16, 8704)
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r.x[0][0]), "=&v"(r.x[0][1]),
        "=&v"(r.p[0][0][0]), "=&v"(r.p[0][0][1]), "=&v"(r.p[0][1][0]), "=&v"(r.p[0][1][1]),
        "=&v"(r.p[1][0][0]), "=&v"(r.p[1][0][1]), "=&v"(r.p[1][1][0]), "=&v"(r.p[1][1][1]),
        "=&v"(r.p[2][0][0]), "=&v"(r.p[2][0][1]), "=&v"(r.p[2][1][0]), "=&v"(r.p[2][1][1])
      : "v"(ax[0]), "v"(ap[0]), "v"(ap[1])
      : "memory");
#endif
}

// x rows of 256 bytes, plane rows of 64; a plane is 2048 bytes
__device__ __forceinline__ void read_step(StepRegs<1, 1>& r, const uint32_t (&ax)[1],
                                          const uint32_t (&ap)[1]) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile(
      MOE_TR(0, 8, 0) MOE_TR(1, 8, 1024) MOE_TR(2, 9, 0) MOE_TR(3, 9, 256)
      MOE_TR(4, 9, 2048) MOE_TR(5, 9, 2304) MOE_TR(6, 9, 4096) MOE_TR(7, 9, 4352)
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r.x[0][0]), "=&v"(r.x[0][1]), "=&v"(r.p[0][0][0]), "=&v"(r.p[0][0][1]),
        "=&v"(r.p[1][0][0]), "=&v"(r.p[1][0][1]), "=&v"(r.p[2][0][0]), "=&v"(r.p[2][0][1])
      : "v"(ax[0]), "v"(ap[0])
      : "memory");
#endif
}
#undef MOE_TR

__device__ __forceinline__ bf16x8_t operand(const u32x2_t (&v)[2]) {
  return __builtin_bit_cast(bf16x8_t, u32x4_t{v[0][0], v[0][1], v[1][0], v[1][1]});
}

// ---- dW_r, bf16
// Tile: BC columns of x by BE experts, the sum over a range of tokens.  Both
// operands have the summed index (the token) as their slow dimension, so they
// are staged as they lie and the transposing read forms the operands.  A
// staged row is cut into blocks of 64 bytes (32 columns, one MFMA block);
// block b of row t sits at b ^ swz(t), so that the four rows which a group of
// 16 lanes reads together lie in different banks (256 bytes a sweep).
constexpr int kKT = 32;          // tokens per stage
constexpr int kSegment = 16384;  // tokens whose mask bits are held in LDS

template <int kRowBytes>
__device__ __forceinline__ int tr_swz(int t) {
  constexpr int R = kRowBytes >= 256 ? 1 : 256 / kRowBytes;  // rows per bank sweep
  constexpr int N = kRowBytes >= 256 ? 4 : kRowBytes / 64;
  return (t / R) % N;
}

struct DwArgs {
  const uint16_t* x;       // [T][d]
  const uint16_t* planes;  // [3][T][Ep]
  const uint8_t* mask;     // [T] or null
  const unsigned char* zero;
  float* out;              // [splits][d][E]
  long long T;
  int d, E, Ep;
  int c_tiles, e_tiles, splits;
  long long t_per_split;   // a multiple of kKT
};

template <int BC, int BE, int WC, int WE, bool kMask>
__global__ __launch_bounds__(kThreads) void router_dw_bf16(DwArgs a) {
  constexpr int MB = BC / 32 / WC, NB = BE / 32 / WE;
  static_assert(WC * WE == 4 && MB >= 1 && NB >= 1, "four waves");
  static_assert(BC == 128 && BE == (MB == 2 ? 128 : 32 * NB), "row sizes that read_step knows");
  constexpr int kRowX = BC * 2, kRowP = BE * 2;
  constexpr int kStageX = kKT * kRowX, kStageP = kKT * kRowP;
  constexpr int kStage = kStageX + 3 * kStageP;
  constexpr int kInstr = kStage / 1024;  // 1 KB loads of a stage
  constexpr int kPerWave = (kInstr + 3) / 4;
  static_assert(kStageX % 1024 == 0 && kStageP % 1024 == 0, "whole loads");
  __shared__ __align__(1024) unsigned char stage[2][kStage];
  __shared__ uint64_t keep[kMask ? kSegment / 64 : 1];
  const int item = xcd_item(a.splits * a.e_tiles * a.c_tiles);
  if (item < 0) return;  // the whole workgroup
  const int ct = item % a.c_tiles;
  const int et = item / a.c_tiles % a.e_tiles;
  const int split = item / (a.c_tiles * a.e_tiles);
  const int c0 = ct * BC, e0 = et * BE;
  const long long t0 = split * a.t_per_split;
  const long long t1 = min(t0 + a.t_per_split, a.T);
  const int tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l = tid % kWave;

  // one 1 KB load of the stage whose first token is `t` into buffer `b`
  auto load = [&](int n, long long t, int b) {
    const bool isx = n * 1024 < kStageX;
    unsigned char* dst = &stage[b][n * 1024];
    if (isx) {
      const int q = n * 64 + l;
      const int r = q / (kRowX / 16), pc = q % (kRowX / 16);
      const int c = pc ^ (tr_swz<kRowX>(r) << 2);
      bool live = t + r < t1;
      if constexpr (kMask) {
        const int i = (int)((t + r - t0) % kSegment);
        live = live && (keep[i / 64] >> (i % 64) & 1);
      }
      const void* src = live ? (const void*)(a.x + (t + r) * a.d + c0 + c * 8) : (const void*)a.zero;
      dma16(src, dst);
    } else {
      const int m = n * 1024 - kStageX;
      const int pl = m / kStageP;
      const int q = (m % kStageP) / 16 + l;
      const int r = q / (kRowP / 16), pc = q % (kRowP / 16);
      const int c = pc ^ (tr_swz<kRowP>(r) << 2);
      const bool live = t + r < t1 && e0 + c * 8 < a.Ep;
      const void* src = live ? (const void*)(a.planes + (pl * a.T + t + r) * a.Ep + e0 + c * 8)
                             : (const void*)a.zero;
      dma16(src, dst);
    }
  };
  auto load_stage = [&](long long t, int b) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int n = w + 4 * i;
      if (n < kInstr) load(n, t, b);
    }
  };

  // operand read offsets: lane l covers column l % 32 of a block, tokens
  // 8 (l / 32) + 0 .. 7 of each 16-deep step (two reads of four)
  const int wc = w % WC, we = w / WC;
  const int j = l % 16;
  const int row = 8 * (l / 32) + j / 4;
  const int in_block = ((l % 32) / 16) * 32 + (j % 4) * 8;
  int offx[MB], offp[NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
    offx[m] = row * kRowX + (((wc * MB + m) ^ tr_swz<kRowX>(j / 4)) * 64) + in_block;
#pragma unroll
  for (int n = 0; n < NB; ++n)
    offp[n] = kStageX + row * kRowP + (((we * NB + n) ^ tr_swz<kRowP>(j / 4)) * 64) + in_block;

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x16_t{};

  for (long long s0 = t0; s0 < t1; s0 += kSegment) {
    const long long s1 = min(s0 + kSegment, t1);
    if constexpr (kMask) {
      __syncthreads();
      for (int i = w; i < kSegment / 64 && s0 + i * 64 < s1; i += 4) {
        const long long t = s0 + i * 64 + l;
        const unsigned long long m = __ballot(t < s1 && a.mask[min(t, a.T - 1)] != 0);
        if (l == 0) keep[i] = m;
      }
      __syncthreads();
    }
    load_stage(s0, 0);
    int b = 0;
    for (long long t = s0; t < s1; t += kKT, b ^= 1) {
      if (t + kKT < s1) {
        load_stage(t + kKT, b ^ 1);
        // at most the next stage's loads still in flight
        if (w + 4 * (kPerWave - 1) < kInstr) wait_vm<kPerWave>();
        else wait_vm<kPerWave - 1>();
      } else {
        wait_vm<0>();
      }
      lds_barrier();
      const uint32_t st = lds_addr(stage[b]);
#pragma unroll
      for (int ks = 0; ks < kKT / 16; ++ks) {
        uint32_t ax[MB], ap[NB];
#pragma unroll
        for (int m = 0; m < MB; ++m) ax[m] = st + offx[m] + ks * 16 * kRowX;
#pragma unroll
        for (int n = 0; n < NB; ++n) ap[n] = st + offp[n] + ks * 16 * kRowP;
        StepRegs<MB, NB> r;
        read_step(r, ax, ap);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MB; ++m)
              acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(r.x[m]), operand(r.p[pl][n]),
                                                                  acc[m][n], 0, 0, 0);
      }
      // every wave's reads of this buffer have returned before it is filled
      // again
      lds_barrier();
    }
  }
  // lane l holds expert l % 32 of a block, columns 8 (q / 4) + 4 (l / 32) + q % 4
  float* out = a.out + (size_t)split * a.d * a.E;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int e = e0 + (we * NB + n) * 32 + l % 32;
      if (e >= a.E) continue;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int c = c0 + (wc * MB + m) * 32 + 8 * (q / 4) + 4 * (l / 32) + q % 4;
        out[(size_t)c * a.E + e] = acc[m][n][q];
      }
    }
}

// ---- dx, bf16
// Tile: 128 columns by 128 tokens, the sum over the experts (at most 512) in
// stages of 32.  The router matrix is the A operand with its rows staged in
// an order that leaves a lane 16 consecutive columns of one token.  A staged
// row is 64 bytes; chunk c of row r sits at c ^ (r / 4) % 4 (four rows make a
// bank sweep).
struct DxArgs {
  const uint16_t* planes;  // [2 of 3][T][Ep]
  const uint16_t* w;       // [d][Ep]
  uint16_t* dx;            // [T][d]
  long long T;
  int d, Ep;
  int c_tiles, t_tiles;
};

constexpr int kDxTile = 128;

// LDS row r of a 32-row block holds matrix row dx_feat(r): the MFMA result
// register q of lane half h is row 8 (q / 4) + 4 h + q % 4, and column
// 16 h + q this way.
__device__ __forceinline__ int dx_feat(int r) { return ((r >> 2) & 1) * 16 + (r >> 3) * 4 + (r & 3); }

__global__ __launch_bounds__(kThreads) void router_dx_bf16(DxArgs a) {
  constexpr int kPart = kDxTile * 64;  // bytes of one staged matrix
  constexpr int kStage = 3 * kPart;
  constexpr int kPerWave = kStage / 1024 / 4;
  __shared__ __align__(1024) unsigned char stage[2][kStage];
  const int item = xcd_item(a.c_tiles * a.t_tiles);
  if (item < 0) return;
  const int ct = item % a.c_tiles;
  const long long t0 = (long long)(item / a.c_tiles) * kDxTile;
  const int c0 = ct * kDxTile;
  const int tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l = tid % kWave;

  const uint16_t* src[kPerWave];
#pragma unroll
  for (int i = 0; i < kPerWave; ++i) {
    const int n = w + 4 * i;        // 1 KB: 16 rows
    const int part = n * 1024 / kPart;
    const int r = (n * 1024 % kPart) / 64 + l / 4;
    const int c = (l % 4) ^ ((r / 4) % 4);
    if (part == 0)
      src[i] = a.w + (size_t)(c0 + (r & ~31) + dx_feat(r & 31)) * a.Ep + c * 8;
    else
      src[i] = a.planes + ((part - 1) * a.T + min(t0 + r, a.T - 1)) * a.Ep + c * 8;
  }
  auto load_stage = [&](int k0, int b) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) dma16(src[i] + k0, &stage[b][(w + 4 * i) * 1024]);
  };
  const int wc = w % 2, wt = w / 2;
  // lane l: row l % 32 of a block, chunk 2 ks + l / 32
  auto off = [&](int r, int ks) { return r * 64 + (((2 * ks + l / 32) ^ ((r / 4) % 4)) << 4); };
  f32x16_t acc[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < 2; ++n) acc[m][n] = f32x16_t{};
  load_stage(0, 0);
  int b = 0;
  for (int k0 = 0; k0 < a.Ep; k0 += 32, b ^= 1) {
    if (k0 + 32 < a.Ep) {
      load_stage(k0 + 32, b ^ 1);
      wait_vm<kPerWave>();
    } else {
      wait_vm<0>();
    }
    lds_barrier();
    const unsigned char* st = stage[b];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      bf16x8_t wa[2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
        wa[m] = *reinterpret_cast<const bf16x8_t*>(st + off(wc * 64 + m * 32 + l % 32, ks));
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const bf16x8_t pb = *reinterpret_cast<const bf16x8_t*>(
              st + (1 + pl) * kPart + off(wt * 64 + n * 32 + l % 32, ks));
#pragma unroll
          for (int m = 0; m < 2; ++m)
            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wa[m], pb, acc[m][n], 0, 0, 0);
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    lds_barrier();
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const long long t = t0 + wt * 64 + n * 32 + l % 32;
    if (t >= a.T) continue;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint16_t* o = a.dx + t * a.d + c0 + wc * 64 + m * 32 + 16 * (l / 32);
      const f32x16_t& v = acc[m][n];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4_t*>(o + 8 * h) =
            u32x4_t{pack_bf16x2(v[8 * h], v[8 * h + 1]), pack_bf16x2(v[8 * h + 2], v[8 * h + 3]),
                    pack_bf16x2(v[8 * h + 4], v[8 * h + 5]),
                    pack_bf16x2(v[8 * h + 6], v[8 * h + 7])};
    }
  }
}

// The router matrix [d][E] with rows of Ep values (zeros behind E) for
// router_dx_bf16, whose loads are 16-byte aligned; one workgroup per 8 rows.
__global__ __launch_bounds__(kThreads) void router_pad_rows(const uint16_t* w, uint16_t* wp, int E,
                                                            int Ep) {
  const size_t r0 = (size_t)blockIdx.x * 8;
  for (int i = threadIdx.x; i < 8 * Ep; i += kThreads) {
    const int r = i / Ep, e = i % Ep;
    wp[(r0 + r) * Ep + e] = e < E ? w[(r0 + r) * E + e] : uint16_t(0);
  }
}

// ---- float32: 64 x 64 tiles, each wave a 32 x 32 block of
// v_mfma_f32_32x32x2_f32, K-major LDS stages 32 deep.
//   kDx:  rows = tokens, columns = x columns, sum over the experts
//   else: rows = x columns, columns = experts, sum over a range of tokens
struct F32Args {
  const float* x;
  const float* w;
  const float* dl;
  const uint8_t* mask;
  float* out;
  long long T;
  int d, E;
  int m_tiles, n_tiles;
  long long t_per_split;
};

template <bool kDx>
__global__ __launch_bounds__(kThreads) void router_grad_f32(F32Args a) {
  constexpr int BK = 32, B = 64, P = B + 1;
  __shared__ float As[BK][P], Bs[BK][P];
  const int tid = threadIdx.x;
  const int w = tid / kWave, l = tid % kWave;
  const long long mt = blockIdx.x % a.m_tiles;
  const int nt = blockIdx.x / a.m_tiles;
  const long long m0 = mt * B;
  const int n0 = nt * B;
  const int split = blockIdx.y;
  const long long k0 = kDx ? 0 : split * a.t_per_split;
  const long long k1 = kDx ? a.E : min(k0 + a.t_per_split, a.T);
  f32x16_t acc = f32x16_t{};
  const int wm = (w % 2) * 32, wn = (w / 2) * 32;
  for (long long kb = k0; kb < k1; kb += BK) {
    __syncthreads();
    if constexpr (kDx) {
      // experts are consecutive in both operands: thread i on expert i % 32
      const int k = tid % BK;
      for (int r = tid / BK; r < B; r += kThreads / BK) {
        const bool in = kb + k < k1;
        As[k][r] = in && m0 + r < a.T ? a.dl[(m0 + r) * a.E + kb + k] : 0.0f;
        Bs[k][r] = in ? a.w[(size_t)(n0 + r) * a.E + kb + k] : 0.0f;
      }
    } else {
      const int c = tid % B;
      for (int k = tid / B; k < BK; k += kThreads / B) {
        const long long t = kb + k;
        const bool in = t < k1;
        const bool live = in && (!a.mask || a.mask[t] != 0);
        As[k][c] = live ? a.x[t * a.d + m0 + c] : 0.0f;
        Bs[k][c] = in && n0 + c < a.E ? a.dl[t * a.E + n0 + c] : 0.0f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; kk += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(As[kk + l / 32][wm + l % 32],
                                                 Bs[kk + l / 32][wn + l % 32], acc, 0, 0, 0);
  }
  const int n = n0 + wn + l % 32;
  const int N = kDx ? a.d : a.E;
  const long long M = kDx ? a.T : a.d;
  float* out = a.out + (kDx ? 0 : (size_t)split * a.d * a.E);
  if (n >= N) return;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const long long m = m0 + wm + 8 * (q / 4) + 4 * (l / 32) + q % 4;
    if (m < M) out[m * N + n] = acc[q];
  }
}

// ---- sums of the partial results, in order: the splits of dW_r (d E values,
// a multiple of four) by the first w_blocks workgroups, the row blocks' column
// sums by the others.
struct SumArgs {
  const float* part;  // [splits][n]
  float* dw;          // [n]
  long long n;
  int splits;
  int w_blocks;
  const float* bias_part;  // [nb][E]
  float* dbias;
  int nb, E;
};

constexpr int kSumThreads = 512;
constexpr int kSumCols = 16;

__global__ __launch_bounds__(kSumThreads) void router_grad_sum(SumArgs a) {
  if ((int)blockIdx.x < a.w_blocks) {
    const long long i = ((long long)blockIdx.x * kSumThreads + threadIdx.x) * 4;
    if (i >= a.n) return;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < a.splits; ++p)
      s += *reinterpret_cast<const f32x4_t*>(a.part + (size_t)p * a.n + i);
    *reinterpret_cast<f32x4_t*>(a.dw + i) = s;
    return;
  }
  // 16 experts, 32 partials abreast
  constexpr int kRows = kSumThreads / kSumCols;
  __shared__ double sp[kSumThreads / kWave][kSumCols];
  const int j = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
  const int w = threadIdx.x / kWave, l = threadIdx.x % kWave;
  const int e = ((int)blockIdx.x - a.w_blocks) * kSumCols + j;
  double s = 0.0;
  if (e < a.E) {
#pragma unroll 16
    for (int b = r; b < a.nb; b += kRows) s += a.bias_part[(size_t)b * a.E + e];
  }
#pragma unroll
  for (int o = kSumCols; o < kWave; o *= 2) s += __shfl_xor(s, o, kWave);
  if (l < kSumCols) sp[w][l] = s;
  __syncthreads();
  if (r == 0 && e < a.E) {
    s = 0.0;
    for (int i = 0; i < kSumThreads / kWave; ++i) s += sp[i][j];
    a.dbias[e] = (float)s;
  }
}

int padded_experts(const Shape& s) { return (s.E + 31) / 32 * 32; }

// Tile of the bf16 dW_r kernel for E experts.
int dw_tile_e(const Shape& s) { return s.E <= 32 ? 32 : s.E <= 64 ? 64 : 128; }
int dw_tile_c() { return 128; }

// Parts of the token range: about two workgroups per compute unit, at least
// 128 tokens each, and partial sums (written and read) no larger than x.
int dw_splits(const Shape& s) {
  const int be = s.act == kBF16 ? dw_tile_e(s) : 64;
  const int bc = s.act == kBF16 ? dw_tile_c() : 64;
  const long long tiles = (long long)(s.d / bc) * ((s.E + be - 1) / be);
  long long n = (512 + tiles - 1) / tiles;
  n = std::min<long long>(n, (s.T + 127) / 128);
  n = std::min<long long>(n, std::max<long long>(s.T / (4LL * s.E), 4));
  return (int)std::max<long long>(std::min<long long>(n, 64), 1);
}

struct GradLayout {
  size_t zero, planes, wpad, dl, bias, dw, total;
};

GradLayout grad_layout(const Shape& s) {
  GradLayout L{};
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  const int Ep = padded_experts(s);
  L.zero = take(kZeroLineBytes);
  if (s.act == kBF16) {
    L.planes = take((size_t)3 * s.T * Ep * 2);
    L.wpad = take(Ep != s.E ? (size_t)s.d * Ep * 2 : 0);
  } else {
    L.dl = take((size_t)s.T * s.E * 4);
  }
  L.bias = take((size_t)gate_grad_blocks(s) * s.E * 4);
  const int ns = dw_splits(s);
  L.dw = take(ns > 1 ? (size_t)ns * s.d * s.E * 4 : 0);
  L.total = o;
  return L;
}

template <int BC, int BE, int WC, int WE>
void launch_dw(const DwArgs& a, hipStream_t st) {
  const dim3 grid(xcd_grid(a.splits * a.e_tiles * a.c_tiles));
  if (a.mask)
    hipLaunchKernelGGL((router_dw_bf16<BC, BE, WC, WE, true>), grid, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((router_dw_bf16<BC, BE, WC, WE, false>), grid, dim3(kThreads), 0, st, a);
}

}  // namespace

size_t route_backward_ws_bytes(const Shape& s) { return grad_layout(s).total; }

hipError_t route_backward(const Shape& s, const RouteGradArgs& g, void* ws, hipStream_t st) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  const GradLayout lay = grad_layout(s);
  const int Ep = padded_experts(s);
  const int ns = dw_splits(s);
  const bool bf16 = s.act == kBF16;
  float* bias_part = reinterpret_cast<float*>(base + lay.bias);
  uint16_t* planes = reinterpret_cast<uint16_t*>(base + lay.planes);
  float* dl = g.dlogits;
  if (!bf16 && !dl && (g.dw || g.dx)) dl = reinterpret_cast<float*>(base + lay.dl);
  float* part = ns > 1 ? reinterpret_cast<float*>(base + lay.dw) : g.dw;

  if (s.T > 0) {
    GateGradArgs ga = g.gate;
    ga.dlogits = dl;
    ga.planes = planes;
    ga.nplanes = !bf16 ? 0 : g.dw ? 3 : g.dx ? 2 : 0;
    ga.zero_line = base + lay.zero;
    ga.bias_part = g.dbias ? bias_part : nullptr;
    hipError_t e = gate_grad(s, ga, Ep, st);
    if (e != hipSuccess) return e;
  }
  if (g.dw && s.T > 0 && bf16) {
    DwArgs a{};
    a.x = static_cast<const uint16_t*>(g.x);
    a.planes = planes;
    a.mask = g.gate.mask;
    a.zero = base + lay.zero;
    a.out = part;
    a.T = s.T;
    a.d = s.d;
    a.E = s.E;
    a.Ep = Ep;
    a.c_tiles = s.d / dw_tile_c();
    a.e_tiles = (s.E + dw_tile_e(s) - 1) / dw_tile_e(s);
    a.splits = ns;
    a.t_per_split = ((s.T + ns - 1) / ns + kKT - 1) / kKT * kKT;
    if (dw_tile_e(s) == 32)
      launch_dw<128, 32, 4, 1>(a, st);
    else if (dw_tile_e(s) == 64)
      launch_dw<128, 64, 4, 1>(a, st);
    else
      launch_dw<128, 128, 2, 2>(a, st);
  }
  if (g.dw && s.T > 0 && !bf16) {
    F32Args a{};
    a.x = static_cast<const float*>(g.x);
    a.dl = dl;
    a.mask = g.gate.mask;
    a.out = part;
    a.T = s.T;
    a.d = s.d;
    a.E = s.E;
    a.m_tiles = s.d / 64;
    a.n_tiles = (s.E + 63) / 64;
    a.t_per_split = ((s.T + ns - 1) / ns + 31) / 32 * 32;
    hipLaunchKernelGGL(router_grad_f32<false>, dim3(a.m_tiles * a.n_tiles, ns), dim3(kThreads), 0,
                       st, a);
  }
  const bool sum_w = g.dw && (ns > 1 || s.T == 0);
  if (sum_w || g.dbias) {
    SumArgs a{};
    a.part = part;
    a.dw = g.dw;
    a.n = (long long)s.d * s.E;
    a.splits = s.T == 0 ? 0 : ns;
    a.w_blocks = sum_w ? (int)((a.n / 4 + kSumThreads - 1) / kSumThreads) : 0;
    a.bias_part = bias_part;
    a.dbias = g.dbias;
    a.nb = s.T == 0 ? 0 : gate_grad_blocks(s);
    a.E = s.E;
    hipLaunchKernelGGL(router_grad_sum, dim3(a.w_blocks + (g.dbias ? (s.E + kSumCols - 1) / kSumCols : 0)),
                       dim3(kSumThreads), 0, st, a);
  }
  if (g.dx && s.T > 0 && bf16) {
    const uint16_t* w = static_cast<const uint16_t*>(g.w_router);
    if (Ep != s.E) {
      uint16_t* wp = reinterpret_cast<uint16_t*>(base + lay.wpad);
      hipLaunchKernelGGL(router_pad_rows, dim3(s.d / 8), dim3(kThreads), 0, st, w, wp, s.E, Ep);
      w = wp;
    }
    DxArgs a{};
    a.planes = planes;
    a.w = w;
    a.dx = static_cast<uint16_t*>(g.dx);
    a.T = s.T;
    a.d = s.d;
    a.Ep = Ep;
    a.c_tiles = s.d / kDxTile;
    a.t_tiles = (s.T + kDxTile - 1) / kDxTile;
    hipLaunchKernelGGL(router_dx_bf16, dim3(xcd_grid(a.c_tiles * a.t_tiles)), dim3(kThreads), 0, st,
                       a);
  }
  if (g.dx && s.T > 0 && !bf16) {
    F32Args a{};
    a.w = static_cast<const float*>(g.w_router);
    a.dl = dl;
    a.out = static_cast<float*>(g.dx);
    a.T = s.T;
    a.d = s.d;
    a.E = s.E;
    a.m_tiles = (s.T + 63) / 64;
    a.n_tiles = s.d / 64;
    hipLaunchKernelGGL(router_grad_f32<true>, dim3(a.m_tiles * a.n_tiles), dim3(kThreads), 0, st,
                       a);
  }
  return hipGetLastError();
}

}  // namespace moe

// The router's backward pass: from the gradient of the logits (balance.hip)
// to the router matrix, the bias and the tokens.
//
//   dW_r[c][e] = sum_t x[t][c] dL[t][e]
//   dx[t][c]   = sum_e dL[t][e] W_r[c][e]
//   db[e]      = sum_t dL[t][e]
//
// bf16 activations: for the router matrix' gradient, which is float32, dL
// (float32) is split into three bfloat16 planes whose sum is the value
// (gate_grad): the products with the bfloat16 tokens are exact and only the
// float32 sums round.  The tokens' gradient is rounded to bfloat16 at the end,
// so two planes do for it: every value of dL with 16 bits (2^-17 off, where the
// result is rounded by up to 2^-8), whatever else is in its row, and the router
// matrix as it is.  (One product in float16, of rows of both scaled by powers of
// two, took 279 us a call against 301 us on 16384 tokens of 7168 x 256, but lost
// what lies far below a row's largest value, in dL and in the matrix.)
// float32 activations: the same kernels on the float32 matrix instructions,
// with dL as it is.
#include <algorithm>
#include <type_traits>

#include "moe_device.h"
#include "moe_internal.h"
#include "route_plan.h"

namespace moe {
namespace {

constexpr int kXcds = 8;

// Consecutive workgroups run on consecutive XCDs: gives each XCD one run of
// consecutive items, so that items that share operands share an L2.  Launched
// with xcd_grid(items) workgroups, of which `block` is one; -1: nothing to do.
__device__ __forceinline__ int xcd_item(int items, int block) {
  const int per = (items + kXcds - 1) / kXcds;
  const int i = block % kXcds * per + block / kXcds;
  return block / kXcds < per && i < items ? i : -1;
}
int xcd_grid(int items) { return (items + kXcds - 1) / kXcds * kXcds; }

// At most N vector-memory operations of this wave (loads to LDS and stores,
// counted in order) still in flight.  The empty statements keep the compiler
// from moving a store or an LDS read across the count that assumes it done.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

// This wave's LDS reads have returned.
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
}

// Barrier that orders LDS accesses of the wave's own instruction stream only:
// the loads of the next stage stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS address of a shared-memory pointer.
__device__ __forceinline__ uint32_t lds_addr(const unsigned char* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) unsigned char*)p;
}

// 16 bytes per lane, global -> LDS: lane i's land at lds + 16 i.  Written as
// an instruction: with the builtin the compiler lets every transposing LDS
// read wait for all loads in flight.  It has no register result; the kernel
// waits by wait_vm and a barrier before it reads what arrives.
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  uint32_t m0;  // (the instruction takes its LDS address from M0, which is put back)
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "v"(src), "s"(lds)
      : "memory");
#else
  (void)src;
  (void)lds;
#endif
}

// Transposing LDS read (ds_read_b64_tr_b16): of 16 lanes, lane j gives the
// address of four 16-bit values of row j / 4, columns 4 (j % 4) .. + 3, and
// gets column j of the four rows.
__device__ __forceinline__ u32x2_t read_tr(uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef short s16x4_t __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(
      u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                   (__attribute__((address_space(3))) s16x4_t*)(uintptr_t)lds));
#else
  (void)lds;
  return u32x2_t{};
#endif
}

// 4 bytes per lane, global -> LDS: lane i's land at lds + 4 i.
__device__ __forceinline__ void dma4(const void* src, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  uint32_t m0;  // (the instruction takes its LDS address from M0, which is put back)
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "v"(src), "s"(lds)
      : "memory");
#else
  (void)src;
  (void)lds;
#endif
}

// ---- dW_r
// Tile: BC columns of x by BE experts, the sum over a range of tokens.  Both
// operands have the summed index (the token) as their slow dimension, so they
// are staged as they lie and the transposing read forms the operands.  A
// staged bf16 row is cut into blocks of 64 bytes (32 columns, one MFMA block);
// block b of row t sits at b ^ swz(t), so that the four rows which a group of
// 16 lanes reads together lie in different banks (256 bytes a sweep).
//
// A wave has MB x NB blocks of 32 x 32.  The three planes of dL share the
// operands of x, so a wave is taller in columns of x than in experts: LDS
// bandwidth bounds it otherwise.  The waves are WC x WE, times KG groups that
// take every KG-th step of 16 tokens and are added at the end.
template <bool kF32, int kRowBytes>
__device__ __forceinline__ int tr_swz(int t) {
  if constexpr (kF32) return 0;  // plain reads: a lane a value, consecutive lanes
  constexpr int R = kRowBytes >= 256 ? 1 : 256 / kRowBytes;  // rows per bank sweep
  constexpr int N = kRowBytes >= 256 ? 4 : kRowBytes / 64;
  return (t / R) % N;
}

struct DwArgs {
  const unsigned char* x;       // [T][d]
  const unsigned char* planes;  // bf16: [3][T][Ep]; float32: [T][Ep]
  const uint8_t* mask;          // [T] or null
  const unsigned char* zero;
  float* out;                   // [splits][d][E]
  long long T;
  int d, E, Ep;
  int c_tiles, e_tiles, splits;
  long long t_per_split;        // a multiple of 64
};

template <bool kF32_, int MB_, int NB_, int WC_, int WE_, int KG_, int KT_, int NST_>
struct DwCfg {
  static constexpr bool kF32 = kF32_;
  static constexpr int MB = MB_, NB = NB_, WC = WC_, WE = WE_, KG = KG_, KT = KT_, NST = NST_;
  static constexpr int kSize = kF32 ? 4 : 2;    // bytes of a value
  static constexpr int kPlanes = kF32 ? 1 : 3;
  static constexpr int kWaves = WC * WE * KG;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int BC = 32 * MB * WC, BE = 32 * NB * WE;
  static constexpr int kRowX = BC * kSize, kRowP = BE * kSize;
  static constexpr int kStageX = KT * kRowX, kStageP = KT * kRowP;
  static constexpr int kStage = kStageX + kPlanes * kStageP;
  static constexpr int kInstr = kStage / 1024;  // 1 KB loads of a stage
  static constexpr int kPerWave = (kInstr + kWaves - 1) / kWaves;
  static constexpr int kSteps = KT / 16 / KG;   // steps of a wave per stage
  static constexpr int kLds = NST * kStage;
  static_assert(kStageX % 1024 == 0 && kStageP % 1024 == 0, "whole loads");
  static_assert(KT % (16 * KG) == 0 && 64 % KT == 0, "whole steps");
  static_assert((NST - 1) * kPerWave < 64, "vmcnt range");
  static_assert(kLds + kSegment / 8 <= 160 * 1024, "LDS budget");
  // the sum over the K groups passes one block row of every wave through LDS
  static_assert(KG == 1 || WC * WE * NB * 4096 <= kLds, "room for the sums");
};

template <class C, bool kMask>
__device__ __forceinline__ void dw_tile(const DwArgs& a, int block, unsigned char* smem) {
  constexpr int MB = C::MB, NB = C::NB;
  uint64_t* keep = reinterpret_cast<uint64_t*>(smem + C::kLds);  // kMask: kSegment bits
  const int item = xcd_item(a.splits * a.e_tiles * a.c_tiles, block);
  if (item < 0) return;  // the whole workgroup
  // the expert tiles of a column tile are neighbours: they share x
  const int et = item % a.e_tiles;
  const int ct = item / a.e_tiles % a.c_tiles;
  const int split = item / (a.c_tiles * a.e_tiles);
  const int c0 = ct * C::BC, e0 = et * C::BE;
  const long long t0 = split * a.t_per_split;
  const long long t1 = min(t0 + a.t_per_split, a.T);
  const int tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l = tid % kWave;
  const uint32_t lds0 = lds_addr(smem);

  // this wave's loads of a stage: source of token 0 of the range, bytes per
  // token, and the token within the stage
  const unsigned char* src[C::kPerWave];
  int row[C::kPerWave];
#pragma unroll
  for (int i = 0; i < C::kPerWave; ++i) {
    const int n = w + C::kWaves * i;
    constexpr int kPer16 = 16 / C::kSize;  // values of a load
    if (n * 1024 < C::kStageX) {
      const int q = n * 64 + l;
      const int r = q / (C::kRowX / 16), pc = q % (C::kRowX / 16);
      const int c = c0 + (pc ^ (tr_swz<C::kF32, C::kRowX>(r) << 2)) * kPer16;
      row[i] = r;
      src[i] = c < a.d ? a.x + ((t0 + r) * a.d + c) * C::kSize : nullptr;
    } else {
      const int m = n * 1024 - C::kStageX;
      const int pl = m / C::kStageP;
      const int q = (m % C::kStageP) / 16 + l;
      const int r = q / (C::kRowP / 16), pc = q % (C::kRowP / 16);
      const int e = e0 + (pc ^ (tr_swz<C::kF32, C::kRowP>(r) << 2)) * kPer16;
      row[i] = r;
      src[i] = e < a.Ep ? a.planes + ((pl * a.T + t0 + r) * a.Ep + e) * C::kSize : nullptr;
    }
  }
  auto load_stage = [&](long long t, int b) {  // t: tokens from t0
#pragma unroll
    for (int i = 0; i < C::kPerWave; ++i) {
      const int n = w + C::kWaves * i;
      if (C::kInstr % C::kWaves != 0 && n >= C::kInstr) continue;
      const bool isx = n * 1024 < C::kStageX;
      const unsigned char* p = src[i] + t * (isx ? a.d : a.Ep) * C::kSize;
      bool live = src[i] != nullptr && t0 + t + row[i] < t1;
      if (kMask && isx) {
        const int k = (int)((t + row[i]) % kSegment);
        live = live && (keep[k / 64] >> (k % 64) & 1);
      }
      dma16(live ? p : a.zero, lds0 + b * C::kStage + n * 1024);
    }
  };

  // operand read offsets: lane l covers column l % 32 of a block; bf16: tokens
  // 8 (l / 32) + 0 .. 7 of each 16-deep step (two reads of four), float32:
  // token 2 i + l / 32 of the i-th of its eight products
  const int kg = w / (C::WC * C::WE), wc = w % C::WC, we = w / C::WC % C::WE;
  const int j = l % 16;
  const int r0 = C::kF32 ? l / 32 + 16 * kg : 8 * (l / 32) + j / 4 + 16 * kg;
  const int in_block = C::kF32 ? (l % 32) * 4 : ((l % 32) / 16) * 32 + (j % 4) * 8;
  constexpr int kBlock = 32 * C::kSize;
  uint32_t offx[MB], offp[NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
    offx[m] = r0 * C::kRowX + ((wc * MB + m) ^ tr_swz<C::kF32, C::kRowX>(j / 4)) * kBlock + in_block;
#pragma unroll
  for (int n = 0; n < NB; ++n)
    offp[n] = C::kStageX + r0 * C::kRowP +
              ((we * NB + n) ^ tr_swz<C::kF32, C::kRowP>(j / 4)) * kBlock + in_block;

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x16_t{};

  auto operand = [](uint32_t at, int row4) {  // row4: bytes of four rows
    const u32x2_t lo = read_tr(at), hi = read_tr(at + row4);
    return __builtin_bit_cast(bf16x8_t, u32x4_t{lo[0], lo[1], hi[0], hi[1]});
  };
  for (long long s0 = 0; s0 < t1 - t0; s0 += kSegment) {
    const int len = (int)min((long long)kSegment, t1 - t0 - s0);
    if constexpr (kMask) {
      __syncthreads();
      for (int i = w; i * 64 < len; i += C::kWaves) {
        const long long t = t0 + s0 + i * 64 + l;
        const unsigned long long m = __ballot(i * 64 + l < len && a.mask[min(t, a.T - 1)] != 0);
        if (l == 0) keep[i] = m;
      }
      __syncthreads();
    }
    const int stages = (len + C::KT - 1) / C::KT;
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i)
      if (i < stages) load_stage(s0 + i * C::KT, i);
    int b = 0;
    for (int s = 0; s < stages; ++s) {
      // stage s has landed: at most those behind it are in flight
      if (s + C::NST - 1 <= stages) {
        constexpr int kBehind = C::NST - 2;
        if (C::kInstr % C::kWaves == 0 || w < C::kInstr % C::kWaves) wait_vm<kBehind * C::kPerWave>();
        else wait_vm<kBehind * (C::kPerWave - 1)>();
      } else {
        wait_vm<0>();
      }
      lds_barrier();  // ... for every wave, and nobody reads stage s - 1 any more
      if (s + C::NST - 1 < stages)
        load_stage(s0 + (long long)(s + C::NST - 1) * C::KT, b == 0 ? C::NST - 1 : b - 1);
      const unsigned char* st = smem + b * C::kStage;
      const uint32_t sa = lds0 + b * C::kStage;
#pragma unroll
      for (int ks = 0; ks < C::kSteps; ++ks) {
        const int kx = ks * 16 * C::KG * C::kRowX, kp = ks * 16 * C::KG * C::kRowP;
        if constexpr (C::kF32) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float xa[MB], pb[NB];
#pragma unroll
            for (int m = 0; m < MB; ++m)
              xa[m] = *reinterpret_cast<const float*>(st + offx[m] + kx + 2 * i * C::kRowX);
#pragma unroll
            for (int n = 0; n < NB; ++n)
              pb[n] = *reinterpret_cast<const float*>(st + offp[n] + kp + 2 * i * C::kRowP);
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
              for (int n = 0; n < NB; ++n)
                acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x2f32(xa[m], pb[n], acc[m][n], 0, 0, 0);
          }
        } else {
          bf16x8_t xa[MB];
#pragma unroll
          for (int m = 0; m < MB; ++m) xa[m] = operand(sa + offx[m] + kx, 4 * C::kRowX);
#pragma unroll
          for (int pl = 0; pl < 3; ++pl)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              const bf16x8_t pb = operand(sa + offp[n] + pl * C::kStageP + kp, 4 * C::kRowP);
#pragma unroll
              for (int m = 0; m < MB; ++m)
                acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[m], pb, acc[m][n], 0, 0, 0);
            }
        }
      }
      wait_lds();
      b = b + 1 == C::NST ? 0 : b + 1;
    }
    lds_barrier();
  }

  if constexpr (C::KG > 1) {
    // the K groups' sums, in order, one block row at a time
    f32x4_t* buf = reinterpret_cast<f32x4_t*>(smem) + (w % (C::WC * C::WE)) * NB * 4 * kWave + l;
    for (int grp = 1; grp < C::KG; ++grp)
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        __syncthreads();
        if (kg == grp) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              buf[(n * 4 + q) * kWave] = f32x4_t{acc[m][n][4 * q], acc[m][n][4 * q + 1],
                                                 acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
        }
        __syncthreads();
        if (kg == 0) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4_t v = buf[(n * 4 + q) * kWave];
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][n][4 * q + i] += v[i];
            }
        }
      }
    if (kg != 0) return;
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
        if (C::BC <= 128 || c < a.d) out[(size_t)c * a.E + e] = acc[m][n][q];
      }
    }
}

template <class C, bool kMask>
__global__ __launch_bounds__(C::kThreads, 2) void router_dw(DwArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  dw_tile<C, kMask>(a, blockIdx.x, smem);
}

// ---- dx
// The sum is short (the experts, at most 512), the output long: each wave
// keeps its columns' share of the router matrix in registers as MFMA operands
// (MB blocks of 32 columns, KS steps of 16 experts, in float32 of 8: 4 MB KS
// registers) and runs over the tokens, whose rows of dL pass through LDS,
// 32 NB tokens a stage, in two buffers.  The waves of a workgroup have
// neighbouring columns and share the stage.  The matrix is the A operand, with
// its rows in an order that suits the stores.
// A staged row (one token) of P bytes: 16-byte chunk c of row t
// sits at c ^ swz(t) within its aligned group of 16 chunks (8, 4 where P is
// no multiple of 256, 128), so that 16 consecutive rows at one logical chunk
// lie in different banks.
struct DxArgs {
  const unsigned char* rows;    // dL: bf16 the first two planes of [3][T][Ep], float32 [T][Ep]
  const int* live;              // [T], 0: a masked token, whose row of dx is zeros; or null
  const unsigned char* w;       // [d][w_pitch], experts behind E not read
  unsigned char* dx;            // [T][d]
  long long T;
  int d, E, w_pitch;
  int c_groups, t_ranges;       // workgroups: column groups x token ranges
  int steps_per_range;          // stages
};

// The MFMA result has row 8 (q / 4) + 4 h + q % 4 in register q of lane half
// h.  Row r of block m of a wave's MB is column dx_feat(m, r) of them.  kQuad:
// half h has the columns 16 MB h + 16 m + q, so that a lane's registers are
// 16 MB consecutive columns of its token.  Else each 16-byte store of the two
// halves covers 32 consecutive bytes: float32 the columns as they come, bf16
// column 16 (q / 8) + 8 h + q % 8 of the block.
template <bool kF32, int MB, bool kQuad>
__device__ __forceinline__ int dx_feat(int m, int r) {
  const int h = (r >> 2) & 1, q = (r >> 3) * 4 + (r & 3);
  if constexpr (kQuad) return 16 * MB * h + 16 * m + q;
  if constexpr (kF32) return 32 * m + r;
  return 32 * m + 16 * (q >> 3) + 8 * h + (q & 7);
}

// 4 x 4 transposition of 16-byte values within every four lanes: value r of
// lane i goes to value i of lane r.
__device__ __forceinline__ void quad_transpose(u32x4_t (&v)[4], int l) {
  auto step = [&](auto ctrl, int bit) {
    constexpr int kCtrl = decltype(ctrl)::value;
    const bool up = l & bit;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r & bit) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = v[r][q], y = v[r | bit][q];
        const uint32_t fx = __builtin_amdgcn_update_dpp(0u, x, kCtrl, 0xF, 0xF, false);
        const uint32_t fy = __builtin_amdgcn_update_dpp(0u, y, kCtrl, 0xF, 0xF, false);
        v[r][q] = up ? fy : x;
        v[r | bit][q] = up ? y : fx;
      }
    }
  };
  step(std::integral_constant<int, 0xB1>{}, 1);  // lane ^ 1
  step(std::integral_constant<int, 0x4E>{}, 2);  // lane ^ 2
}

template <int KS>
__device__ __forceinline__ int dx_swz(int t) {
  constexpr int P = KS * 32;
  return P % 256 == 0 ? t & 15 : P % 128 == 0 ? (t >> 1) & 7 : (t >> 2) & 3;
}

template <bool kF32, int MB, int KS, int NB, int NW>
__device__ __forceinline__ void dx_tile(const DxArgs& a, int block, unsigned char* smem) {
  constexpr int kSize = kF32 ? 4 : 2;        // bytes of a value
  constexpr int kPlanes = kF32 ? 1 : 2;
  constexpr int kTokens = 32 * NB;
  constexpr int P = KS * 32;                 // bytes of a staged row
  constexpr int kPlane = kTokens * P;
  constexpr int kStage = kPlanes * kPlane;
  constexpr int kInstr = kStage / 1024;      // 1 KB loads of a stage
  constexpr int kPerWave = (kInstr + NW - 1) / NW;
  static_assert(kStage % 1024 == 0, "whole loads");
  constexpr int kStores = MB * NB * kSize;   // 16-byte stores of a lane per stage
  // Four 16-byte values at a time are transposed within four lanes before
  // the store, where there are as many.
  constexpr bool kQuad = MB * kSize % 4 == 0;
  const int item = xcd_item(a.c_groups * a.t_ranges, block);
  if (item < 0) return;  // the whole workgroup
  // the column groups of a token range run on one XCD (they share its rows)
  const int cg = item % a.c_groups;
  const int range = item / a.c_groups;
  const int tid = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l = tid % kWave;
  const int h = l / 32;
  const int c0 = (cg * NW + w) * MB * 32;    // this wave's columns (may be behind d)
  const long long steps = (a.T + kTokens - 1) / kTokens;
  const long long s0 = (long long)range * a.steps_per_range;
  const int ns = (int)min((long long)a.steps_per_range, steps - s0);
  if (ns <= 0) return;  // the whole workgroup

  // loads of a stage: 1 KB is 1024 / P rows (or a part of one)
  const uint32_t lds0 = lds_addr(smem);
  auto load_stage = [&](int s, int b) {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int n = w * kPerWave + i;
      if (kInstr % NW != 0 && n >= kInstr) break;
      const int q = n * 64 + l;               // 16-byte chunk of the stage
      const int row = q / (P / 16), pc = q % (P / 16);
      const int pl = row / kTokens, r = row % kTokens;
      const int c = pc ^ dx_swz<KS>(r);
      const long long t = min((s0 + s) * kTokens + r, a.T - 1);
      dma16(a.rows + (pl * a.T + t) * P + c * 16, lds0 + b * kStage + n * 1024);
    }
    // the tokens' marks go the same way: a load into registers would be waited
    // for with every store before it
    if (a.live && w == 0 && l < kTokens)
      dma4(a.live + min((s0 + s) * kTokens + l, a.T - 1), lds0 + 2 * kStage + b * kTokens * 4);
  };
  load_stage(0, 0);

  // lane l: matrix row dx_feat(m, l % 32), the 16 bytes h of each
  // step's 32 (float32: the step's product i takes value i of both halves)
  u32x4_t wf[MB][KS];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int c = min(c0 + dx_feat<kF32, MB, kQuad>(m, l % 32), a.d - 1);
    const unsigned char* row = a.w + (size_t)c * a.w_pitch * kSize + 16 * h;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      wf[m][ks] = u32x4_t{0, 0, 0, 0};
      if (32 * ks + 16 * h < a.E * kSize)
        wf[m][ks] = *reinterpret_cast<const u32x4_t*>(row + 32 * ks);
    }
  }
  // operand read: lane l has token l % 32 of a block, chunk 2 ks + h
  constexpr int kGroup = P % 256 == 0 ? 8 : P % 128 == 0 ? 4 : 2;  // steps of a swizzle group
  uint32_t base[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int r = n * 32 + l % 32;
    base[n] = r * P + ((h ^ dx_swz<KS>(r)) << 4);
  }
  const bool all_cols = c0 + MB * 32 <= a.d;
  int b = 0;
  for (int s = 0; s < ns; ++s, b ^= 1) {
    // the stage's loads; all stores of the last stage may be in flight, where
    // all were made (it had no token behind T: only a range's end has)
    if (s == 0 || !all_cols) wait_vm<0>();
    else wait_vm<kStores>();
    lds_barrier();            // ... of every wave, and nobody reads the other buffer any more
    if (s + 1 < ns) load_stage(s + 1, b ^ 1);
    f32x16_t acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n) acc[m][n] = f32x16_t{};
    const unsigned char* st = smem + b * kStage;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int pl = 0; pl < kPlanes; ++pl) {
        u32x4_t pb[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n)
          pb[n] = *reinterpret_cast<const u32x4_t*>(
              st + pl * kPlane + (base[n] ^ ((ks % kGroup) << 5)) + ks / kGroup * kGroup * 32);
        if constexpr (kF32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
              for (int m = 0; m < MB; ++m)
                acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                    __uint_as_float(wf[m][ks][i]), __uint_as_float(pb[n][i]), acc[m][n], 0, 0, 0);
        } else {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < MB; ++m)
              acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  __builtin_bit_cast(bf16x8_t, wf[m][ks]), __builtin_bit_cast(bf16x8_t, pb[n]),
                  acc[m][n], 0, 0, 0);
        }
      }
    // A masked token's row of dL is zeros, which an infinity or NaN of the
    // matrix turns into NaN: its row of dx is not taken from the product.
    const int* live = reinterpret_cast<const int*>(smem + 2 * kStage) + b * kTokens;
    bool drop[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) drop[n] = a.live && live[n * 32 + l % 32] == 0;
    wait_lds();
    // kQuad: lane l has 16 MB columns of token l % 32, from column 16 MB h, as
    // kVals 16-byte values.  Transposed within four lanes, these store 64
    // consecutive bytes of one token, in four stores of the lanes' four
    // tokens: whole pieces of a line, which may stream past the caches (16384
    // tokens of 7168 x 8: the whole call 134 us, with 32-byte pieces, 128 us
    // with 64-byte ones, 106 us streaming; 32-byte pieces streaming are five
    // times slower).
    constexpr int kVals = MB * kSize;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      u32x4_t o[kVals];
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const f32x16_t& v = acc[m][n];
#pragma unroll
        for (int i = 0; i < kSize; ++i) {
          if constexpr (kF32) {
            o[m * kSize + i] = u32x4_t{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                       __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
          } else {
            o[m * kSize + i] =
                u32x4_t{pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                        pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7])};
          }
        }
      }
      if (drop[n])
#pragma unroll
        for (int i = 0; i < kVals; ++i) o[i] = u32x4_t{0, 0, 0, 0};
      const long long tb = (s0 + s) * kTokens + n * 32;
      if constexpr (kQuad) {
        const long long t = tb + (l % 32 & ~3);
#pragma unroll
        for (int c = 0; c < kVals; c += 4) {
          u32x4_t q4[4] = {o[c], o[c + 1], o[c + 2], o[c + 3]};
          quad_transpose(q4, l);
          unsigned char* to = a.dx + (t * a.d + c0 + 16 * MB * h) * kSize + (c + l % 4) * 16;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (t + r < a.T && c0 < a.d)
              __builtin_nontemporal_store(
                  q4[r], reinterpret_cast<u32x4_t*>(to + (long long)r * a.d * kSize));
        }
      } else {
        const long long t = tb + l % 32;
        if (t < a.T && c0 < a.d) {
          unsigned char* to = a.dx + (t * a.d + c0) * kSize + 16 * h;
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < kSize; ++i)
              *reinterpret_cast<u32x4_t*>(to + 32 * m * kSize + 32 * i) = o[m * kSize + i];
        }
      }
    }
  }
}

template <bool kF32, int MB, int KS, int NB, int NW, int kMinWaves>
__global__ __launch_bounds__(NW* kWave, kMinWaves) void router_dx(DxArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  dx_tile<kF32, MB, KS, NB, NW>(a, blockIdx.x, smem);
}

// Both products of few tokens in one launch: the first dw_blocks workgroups
// (a multiple of the XCDs) are those of dW_r, the others of dx.
template <class C, bool kMask, int KS>
__global__ __launch_bounds__(512, 2) void router_products(DwArgs w, DxArgs x, int dw_blocks) {
  static_assert(C::kThreads == 512, "both have eight waves");
  extern __shared__ __align__(1024) unsigned char smem[];
  if ((int)blockIdx.x < dw_blocks)
    dw_tile<C, kMask>(w, blockIdx.x, smem);
  else
    dx_tile<C::kF32, 1, KS, 1, 8>(x, (int)blockIdx.x - dw_blocks, smem);
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

DwPlan plan_of(const Shape& s) { return dw_plan(s.T, s.d, s.E, s.act == kBF16); }

struct GradLayout {
  size_t zero, planes, live, wpad, bias, dw, total;
};

GradLayout grad_layout(const Shape& s) {
  GradLayout L{};
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  const int Ep = padded_experts(s.E);
  L.zero = take(kZeroLineBytes);
  if (s.act == kBF16) {
    L.planes = take((size_t)3 * s.T * Ep * 2);
    L.wpad = take(s.E % 8 != 0 ? (size_t)s.d * Ep * 2 : 0);
  } else {
    L.planes = take((size_t)s.T * Ep * 4);
    L.wpad = take(s.E % 4 != 0 ? (size_t)s.d * Ep * 4 : 0);
  }
  L.live = take((size_t)s.T * 4);
  L.bias = take((size_t)gate_grad_blocks(s) * s.E * 4);
  const int ns = plan_of(s).splits;
  L.dw = take(ns > 1 ? (size_t)ns * s.d * s.E * 4 : 0);
  L.total = o;
  return L;
}

template <class C>
void place_dw(DwArgs& a) {
  a.c_tiles = (a.d + C::BC - 1) / C::BC;
  a.e_tiles = (a.E + C::BE - 1) / C::BE;
  a.t_per_split = dw_tokens_per_split(a.T, a.splits);
}
template <class C>
int dw_lds(const DwArgs& a) {
  return C::kLds + (a.mask ? kSegment / 8 : 0);
}

template <class C, bool kMask>
hipError_t launch_dw_as(const DwArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  const int lds = dw_lds<C>(a);
  const hipError_t e = set_lds_attr(reinterpret_cast<const void*>(&router_dw<C, kMask>), lds, done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((router_dw<C, kMask>), dim3(xcd_grid(a.splits * a.e_tiles * a.c_tiles)),
                     dim3(C::kThreads), lds, st, a);
  return hipGetLastError();
}
template <class C>
hipError_t launch_dw(DwArgs a, hipStream_t st) {
  place_dw<C>(a);
  return a.mask ? launch_dw_as<C, true>(a, st) : launch_dw_as<C, false>(a, st);
}

// Column groups and token ranges of dx, for `slots` workgroups at once.
void place_dx(DxArgs& a, int cols, int tokens, int slots) {
  a.c_groups = (a.d + cols - 1) / cols;
  const long long steps = (a.T + tokens - 1) / tokens;
  const int ranges = std::max(slots / a.c_groups, 1);
  a.steps_per_range = (int)std::max<long long>((steps + ranges - 1) / ranges, 1);
  a.t_ranges = (int)((steps + a.steps_per_range - 1) / a.steps_per_range);
}
constexpr int dx_lds(bool f32, int KS, int NB) {
  return 2 * 32 * NB * ((f32 ? 1 : 2) * KS * 32 + 4);
}

template <bool kF32, int MB, int KS, int NB, int NW, int kMinWaves>
hipError_t launch_dx_as(DxArgs a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int kLds = dx_lds(kF32, KS, NB);
  static_assert(kLds <= 160 * 1024, "LDS budget");
  const void* kern = reinterpret_cast<const void*>(&router_dx<kF32, MB, KS, NB, NW, kMinWaves>);
  const hipError_t e = set_lds_attr(kern, kLds, done);
  if (e != hipSuccess) return e;
  // as many workgroups as fit the compute units at once
  place_dx(a, MB * 32 * NW, 32 * NB, 256 * 4 * kMinWaves / NW);
  hipLaunchKernelGGL((router_dx<kF32, MB, KS, NB, NW, kMinWaves>),
                     dim3(xcd_grid(a.c_groups * a.t_ranges)), dim3(NW * kWave), kLds, st, a);
  return hipGetLastError();
}

// The variant for KS steps: a wave's share of the matrix takes 4 MB KS
// registers, a stage 32 NB x 32 KS bytes of LDS a plane.  (From 256 experts on,
// 64 tokens a stage leave no registers for the transposition of the stores, or
// no LDS.)  For few tokens one of 128 columns and 32 tokens a workgroup (one
// token of 4096 x 128, float32: 6.2 us, 23.8 us wide).
template <bool kF32, int MB, int KS, int NB, int NW, int kMinWaves>
hipError_t launch_dx_for(const DxArgs& a, bool few, hipStream_t st) {
  if (few) return launch_dx_as<kF32, 1, KS, 1, 4, 1>(a, st);
  return launch_dx_as<kF32, MB, KS, NB, NW, kMinWaves>(a, st);
}

hipError_t launch_dx(const DxArgs& a, int Ep, bool f32, bool few, hipStream_t st) {
  if (f32) switch (Ep) {
      case 32: return launch_dx_for<true, 2, 4, 2, 4, 2>(a, few, st);
      case 64: return launch_dx_for<true, 2, 8, 2, 4, 2>(a, few, st);
      case 128: return launch_dx_for<true, 2, 16, 1, 8, 2>(a, few, st);
      case 192: return launch_dx_for<true, 2, 24, 2, 4, 1>(a, few, st);
      case 256: return launch_dx_for<true, 2, 32, 2, 4, 1>(a, few, st);
      case 320: return launch_dx_as<true, 1, 40, 1, 4, 1>(a, st);
      case 384: return launch_dx_as<true, 1, 48, 1, 4, 1>(a, st);
      case 448: return launch_dx_as<true, 1, 56, 1, 4, 1>(a, st);
      default: return launch_dx_as<true, 1, 64, 1, 4, 1>(a, st);
    }
  switch (Ep) {
    case 32: return launch_dx_for<false, 2, 2, 2, 4, 2>(a, few, st);
    case 64: return launch_dx_for<false, 2, 4, 2, 4, 2>(a, few, st);
    case 128: return launch_dx_for<false, 2, 8, 2, 4, 2>(a, few, st);
    case 192: return launch_dx_for<false, 2, 12, 2, 8, 2>(a, few, st);
    case 256: return launch_dx_for<false, 2, 16, 1, 8, 2>(a, few, st);
    case 320: return launch_dx_for<false, 2, 20, 1, 4, 1>(a, few, st);
    case 384: return launch_dx_for<false, 2, 24, 1, 4, 1>(a, few, st);
    case 448: return launch_dx_for<false, 2, 28, 1, 4, 1>(a, few, st);
    default: return launch_dx_for<false, 2, 32, 1, 4, 1>(a, few, st);
  }
}

// dW_r and dx of few tokens in one launch.
template <class C, int KS, bool kMask>
hipError_t launch_products_as(const DwArgs& w, DxArgs x, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int kDx = dx_lds(C::kF32, KS, 1);
  const int lds = std::max(dw_lds<C>(w), kDx);
  const void* kern = reinterpret_cast<const void*>(&router_products<C, kMask, KS>);
  const hipError_t e = set_lds_attr(kern, lds, done);
  if (e != hipSuccess) return e;
  place_dx(x, 256, 32, 256);
  const int dw_blocks = xcd_grid(w.splits * w.e_tiles * w.c_tiles);
  hipLaunchKernelGGL((router_products<C, kMask, KS>),
                     dim3(dw_blocks + xcd_grid(x.c_groups * x.t_ranges)), dim3(512), lds, st, w, x,
                     dw_blocks);
  return hipGetLastError();
}
template <class C, int KS>
hipError_t launch_products_for(DwArgs w, const DxArgs& x, hipStream_t st) {
  place_dw<C>(w);
  return w.mask ? launch_products_as<C, KS, true>(w, x, st)
                : launch_products_as<C, KS, false>(w, x, st);
}

template <bool kF32>
using Dw32 = DwCfg<kF32, 1, 1, 4, 1, 2, 64, 3>;
template <bool kF32>
using Dw64 = DwCfg<kF32, 2, 1, 2, 2, 2, 32, kF32 ? 5 : 6>;
template <bool kF32>
using Dw128 = DwCfg<kF32, 2, 2, 2, 2, 2, 32, 4>;

// (the tile of dW_r follows from the experts, as in dw_plan; kB: steps of 64
// experts)
template <bool kF32, int kB>
hipError_t launch_products(const DwArgs& w, const DxArgs& x, int Ep, hipStream_t st) {
  switch (Ep) {
    case 32: return launch_products_for<Dw32<kF32>, kB / 2>(w, x, st);
    case 64: return launch_products_for<Dw64<kF32>, kB>(w, x, st);
    case 128: return launch_products_for<Dw128<kF32>, 2 * kB>(w, x, st);
    case 192: return launch_products_for<Dw128<kF32>, 3 * kB>(w, x, st);
    case 256: return launch_products_for<Dw128<kF32>, 4 * kB>(w, x, st);
  }
  if constexpr (!kF32) switch (Ep) {
      case 320: return launch_products_for<Dw128<kF32>, 5 * kB>(w, x, st);
      case 384: return launch_products_for<Dw128<kF32>, 6 * kB>(w, x, st);
      case 448: return launch_products_for<Dw128<kF32>, 7 * kB>(w, x, st);
      case 512: return launch_products_for<Dw128<kF32>, 8 * kB>(w, x, st);
    }
  return hipErrorInvalidValue;  // (not reached: see route_backward)
}

}  // namespace

size_t route_backward_ws_bytes(const Shape& s) { return grad_layout(s).total; }

hipError_t route_backward(const Shape& s, const RouteGradArgs& g, void* ws, hipStream_t st) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  const GradLayout lay = grad_layout(s);
  const int Ep = padded_experts(s.E);
  const DwPlan plan = plan_of(s);
  const int ns = plan.splits;
  const bool f32 = s.act != kBF16;
  const bool products = s.T > 0 && (g.dw || g.dx);
  // one row block's column sums are the bias' gradient
  const bool sum_b = g.dbias && (s.T == 0 || gate_grad_blocks(s) > 1);
  float* bias_part = sum_b ? reinterpret_cast<float*>(base + lay.bias) : g.dbias;
  float* part = ns > 1 ? reinterpret_cast<float*>(base + lay.dw) : g.dw;
  // what the products read, bf16: the planes; float32: rows of Ep values (the
  // caller's, if they are as long)
  unsigned char* planes = base + lay.planes;
  if (f32 && g.dlogits && Ep == s.E) planes = reinterpret_cast<unsigned char*>(g.dlogits);

  if (s.T > 0) {
    GateGradArgs ga = g.gate;
    ga.dlogits = g.dlogits;
    if (products && f32 && planes != reinterpret_cast<unsigned char*>(g.dlogits))
      ga.dl_rows = reinterpret_cast<float*>(planes);
    if (products && !f32) {
      ga.planes = reinterpret_cast<uint16_t*>(planes);
      ga.nplanes = g.dw ? 3 : 2;
    }
    if (g.dx && g.gate.mask) ga.live = reinterpret_cast<int*>(base + lay.live);
    ga.zero_line = base + lay.zero;
    ga.bias_part = bias_part;
    // rows of the matrix that 16-byte loads cannot take are copied with Ep
    // values each, by workgroups of the same launch
    if (g.dx && s.E % (f32 ? 4 : 8) != 0) {
      ga.pad_src = g.w_router;
      ga.pad_dst = base + lay.wpad;
    }
    const hipError_t e = gate_grad(s, ga, Ep, st);
    if (e != hipSuccess) return e;
  }
  DwArgs wa{};
  if (g.dw && s.T > 0) {
    wa.x = static_cast<const unsigned char*>(g.x);
    wa.planes = planes;
    wa.mask = g.gate.mask;
    wa.zero = base + lay.zero;
    wa.out = part;
    wa.T = s.T;
    wa.d = s.d;
    wa.E = s.E;
    wa.Ep = Ep;
    wa.splits = ns;
  }
  DxArgs xa{};
  if (g.dx && s.T > 0) {
    const bool padded = s.E % (f32 ? 4 : 8) != 0;
    xa.rows = planes;
    xa.live = g.gate.mask ? reinterpret_cast<const int*>(base + lay.live) : nullptr;
    xa.w = padded ? base + lay.wpad : static_cast<const unsigned char*>(g.w_router);
    xa.w_pitch = padded ? Ep : s.E;
    xa.E = xa.w_pitch;
    xa.dx = static_cast<unsigned char*>(g.dx);
    xa.T = s.T;
    xa.d = s.d;
  }
  const bool few = few_tokens(s.T, s.d);
  const bool both = products && g.dw && g.dx && products_in_one_launch(s.T, s.d, s.E, !f32);
  hipError_t e = hipSuccess;
  if (both) {
    e = f32 ? launch_products<true, 8>(wa, xa, Ep, st) : launch_products<false, 4>(wa, xa, Ep, st);
  } else if (g.dw && s.T > 0) {
    if (f32)
      e = plan.be == 32   ? launch_dw<Dw32<true>>(wa, st)
          : plan.be == 64 ? launch_dw<Dw64<true>>(wa, st)
                          : launch_dw<Dw128<true>>(wa, st);
    else if (plan.bc == 256)
      e = plan.be == 32   ? launch_dw<DwCfg<false, 2, 1, 4, 1, 2, 64, 3>>(wa, st)
          : plan.be == 64 ? launch_dw<DwCfg<false, 2, 2, 4, 1, 2, 32, 4>>(wa, st)
                          : launch_dw<DwCfg<false, 4, 2, 2, 2, 2, 32, 3>>(wa, st);
    else
      e = plan.be == 32   ? launch_dw<Dw32<false>>(wa, st)
          : plan.be == 64 ? launch_dw<Dw64<false>>(wa, st)
                          : launch_dw<Dw128<false>>(wa, st);
  }
  if (e != hipSuccess) return e;
  const bool sum_w = g.dw && (ns > 1 || s.T == 0);
  if (sum_w || sum_b) {
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
    hipLaunchKernelGGL(router_grad_sum,
                       dim3(a.w_blocks + (sum_b ? (s.E + kSumCols - 1) / kSumCols : 0)),
                       dim3(kSumThreads), 0, st, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (g.dx && s.T > 0 && !both) e = launch_dx(xa, Ep, f32, few, st);
  return e;
}

}  // namespace moe

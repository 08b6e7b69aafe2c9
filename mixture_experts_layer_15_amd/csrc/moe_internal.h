// Internal host-side interface between the C ABI (moe_api.cpp) and the
// kernel launchers (*.hip).  Not installed; callers use include/moe.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "moe.h"

namespace moe {

enum Fmt : int { kF32 = 0, kBF16 = 1, kFP8 = 2, kFP4 = 3 };

constexpr int kMaxExperts = 512;      // E limit (router top-k and permutation LDS tables)
constexpr int kPermuteChunk = 2048;   // slots per workgroup in the permutation kernels

// Validated problem shape.  S = T*k slots.
struct Shape {
  int T, d, E, k, F, e0, El;
  int act, weight;
  int blocked;  // expert weights in the blocked layout of pack_weights
  long long S;
};

inline size_t align_up(size_t v, size_t a = 256) { return (v + a - 1) / a * a; }

// hipFuncSetAttribute for the dynamic LDS size of `kern`, once per device
// (devices 0..63 remembered in an atomic bit set; the call is idempotent, so
// two threads that both make it race harmlessly).
inline hipError_t set_lds_attr(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}
inline int act_bytes(const Shape& s) { return s.act == kF32 ? 4 : 2; }

// ---- route.hip
// K splits of the router GEMM used by moe_forward, and the scratch they need.
int router_splits(const Shape& s);
size_t route_ws_bytes(const Shape& s);
// w_router != null: logits = x W_r + bias are published to `logits` and
// selected on; scratch holds route_ws_bytes (the transposed router matrix and
// K-split partials).  w_router == null: `logits_in` holds the final logits
// (scratch may be null).
hipError_t route(const Shape& s, const void* x, const void* w_router, const float* bias,
                 const float* logits_in, float* logits, int32_t* topk_idx, float* topk_w,
                 void* scratch, hipStream_t st);
bool use_router_gemm(const Shape& s);

// prod [ks][T][E] = x W_r (float32 accumulation, K cut into
// ks = router_gemm_splits(s) parts, one plane each) from the router matrix
// stored [E][d]
int router_gemm_splits(const Shape& s);
hipError_t router_gemm(const Shape& s, const void* x, const void* w_router_t, float* prod,
                       hipStream_t st);

// ---- ffn.hip (tile schedule shared with the permutation)
struct FfnSchedule {
  int4* tiles;   // (local expert, first row, expert's end row, 0) of every M tile
  int* ntiles;   // number of M tiles
  int bm;        // M tile height
};
FfnSchedule ffn_schedule_view(const Shape& s, void* ffn_ws);
size_t ffn_ws_bytes(const Shape& s);
// schedule_ready: the tile schedule in ffn_ws was already written (by the
// permutation); stage_events: null or 3 events recorded after the schedule,
// the gate/up GEMM and the down GEMM.
hipError_t expert_ffn(const Shape& s, const void* x, const int32_t* sorted_slot,
                      const int32_t* offsets, const void* w_gate, const void* w_up,
                      const void* w_down, const void* s_gate, const void* s_up,
                      const void* s_down, const float* topk_w, void* y, void* ws,
                      hipStream_t st, bool schedule_ready = false,
                      hipEvent_t const* stage_events = nullptr);

// ---- permute.hip
size_t permute_ws_bytes(const Shape& s);
// When `sched` is non-null and the single-workgroup path runs, the expert
// tile schedule is written too and *sched_written is set.
hipError_t permute(const Shape& s, const int32_t* topk_idx, int32_t* counts, int32_t* offsets,
                   int32_t* sorted_slot, int32_t* slot_pos, void* ws, hipStream_t st,
                   const FfnSchedule* sched = nullptr, bool* sched_written = nullptr);

// ---- combine.hip
hipError_t combine(const Shape& s, const void* y, const int32_t* slot_pos, const float* topk_w,
                   void* out, hipStream_t st);

// The combine's backward pass (y, dy, topk_w, dtopk_w may be null).
hipError_t combine_backward(const Shape& s, const void* dout, const void* y,
                            const int32_t* slot_pos, const float* topk_w, void* dy,
                            float* dtopk_w, hipStream_t st);

// ---- balance.hip
size_t balance_ws_bytes(const Shape& s);
hipError_t balance_loss(const Shape& s, const float* logits, const int32_t* topk_idx,
                        const uint8_t* mask, int32_t* counts, int32_t* n_tokens,
                        float* prob_mean, float* losses, void* ws, hipStream_t st);

// Gradient of gates (dtopk_w) and losses (dlosses) with respect to the logits.
constexpr int kZeroLineBytes = 512;
struct GateGradArgs {
  const float* logits;     // read where dlosses is given
  const int32_t* idx;      // idx, topk_w: read where dtopk_w is given
  const float* topk_w;
  const float* dtopk_w;    // [T][k] or null
  const uint8_t* mask;     // [T] or null
  const int32_t* counts;   // counts, n_tokens: read where dlosses is given
  const int32_t* n_tokens;
  const float* dlosses;    // [2] or null
  float* dlogits;          // [T][E] or null
  uint16_t* planes;        // [nplanes][T][Ep] bfloat16 planes whose sum is the gradient, or null
  int nplanes;             // 2 or 3
  float* dl_rows;          // [T][Ep] the gradient, columns from E on zero, or null
  int* live;               // [T] the mask as integers, or null (without a mask)
  const void* pad_src;     // a matrix [d][E] of act values that is copied to
  void* pad_dst;           // [d][Ep] (zeros behind E), or null
  void* zero_line;         // kZeroLineBytes that the kernel clears
  float* bias_part;        // [gate_grad_blocks][E] column sums per workgroup, or null
};
int gate_grad_blocks(const Shape& s);
hipError_t gate_grad(const Shape& s, const GateGradArgs& a, int Ep, hipStream_t st);

// ---- route_grad.hip
struct RouteGradArgs {
  GateGradArgs gate;       // the inputs
  const void* x;           // read where dw is given
  const void* w_router;    // read where dx is given
  float* dlogits;          // each output may be null
  void* dx;
  float* dw;
  float* dbias;
};
size_t route_backward_ws_bytes(const Shape& s);
hipError_t route_backward(const Shape& s, const RouteGradArgs& g, void* ws, hipStream_t st);

// ---- grads.hip
size_t grad_ws_bytes(const moe_grad_t* g, int n);
hipError_t grad_norm(const moe_grad_t* g, int n, float* norm, void* ws, hipStream_t st);
hipError_t grad_clip(const moe_grad_t* g, int n, const float* norm, float max_norm,
                     hipStream_t st);

// Blocked layout of one stored expert weight matrix [Nout][K] (any weight
// format but float32): [Nout/32][K/64][32 rows][64 K values], each 32 x 64
// unit being the LDS image the expert GEMMs stage for that block (rows in
// the MFMA feature order, 16-byte chunks XOR-swizzled).  Same size as the
// row-major matrix.
hipError_t pack_weights(const Shape& s, int which, const void* src, void* dst, hipStream_t st);

// ---- eplb.hip
// The placement plan of moe_eplb_plan (arguments already checked).
int eplb_plan(const int64_t* load, int E, int G, int R, int32_t* replicas, int32_t* phys_to_log,
              int32_t* log_to_phys, double* rank_load);
hipError_t eplb_remap(int T, int k, int E, int G, const int32_t* topk_idx,
                      const int32_t* replicas, const int32_t* log_to_phys, int32_t* topk_phys,
                      hipStream_t st);

}  // namespace moe

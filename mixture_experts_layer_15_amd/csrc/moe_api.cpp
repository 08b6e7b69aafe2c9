// C ABI of the MoE layer (declared in include/moe.h): argument checks,
// workspace sizing and launch sequencing.  Every check runs on the host
// before anything is enqueued; no call allocates, frees or synchronises.
#include "moe.h"

#include <algorithm>
#include <cmath>
#include <new>

#include "moe_internal.h"

namespace {

using moe::Shape;

bool supported_pair(int act, int weight) {
  return (act == MOE_F32 && weight == MOE_F32) || (act == MOE_BF16 && weight == MOE_BF16) ||
         (act == MOE_BF16 && weight == MOE_FP8_E4M3) || (act == MOE_BF16 && weight == MOE_MXFP4);
}

// Shape checks shared by every call.  Returns MOE_OK and fills `s` on success.
moe_status_t check_problem(const moe_problem_t* p, Shape* s) {
  if (p == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (p->T < 0 || p->d <= 0 || p->E <= 0 || p->F <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->k < 1 || p->k > p->E) return MOE_ERR_INVALID_ARGUMENT;
  if (p->expert_begin < 0 || p->num_local < 1) return MOE_ERR_INVALID_ARGUMENT;
  if ((long long)p->expert_begin + p->num_local > p->E) return MOE_ERR_INVALID_ARGUMENT;
  if (p->d % 128 != 0 || p->F % 128 != 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->act < MOE_F32 || p->act > MOE_MXFP4 || p->weight < MOE_F32 || p->weight > MOE_MXFP4)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->weight_layout != MOE_LAYOUT_ROWS && p->weight_layout != MOE_LAYOUT_BLOCKED)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!supported_pair(p->act, p->weight)) return MOE_ERR_UNSUPPORTED;
  if (p->weight_layout == MOE_LAYOUT_BLOCKED && p->weight == MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (p->E > moe::kMaxExperts || p->d > 65536 || p->F > 65536) return MOE_ERR_UNSUPPORTED;
  const long long S = (long long)p->T * p->k;
  if (S >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  // the expert GEMMs address x and one expert's weight matrix with 32-bit
  // offsets
  const long long ab = p->act == MOE_F32 ? 4 : 2;
  const long long wbits = p->weight == MOE_F32 ? 32 : p->weight == MOE_BF16 ? 16
                        : p->weight == MOE_FP8_E4M3 ? 8 : 4;
  if ((long long)p->T * p->d * ab >= (1LL << 32) || (long long)p->F * p->d * wbits / 8 >= (1LL << 32))
    return MOE_ERR_UNSUPPORTED;
  s->T = p->T;
  s->d = p->d;
  s->E = p->E;
  s->k = p->k;
  s->F = p->F;
  s->e0 = p->expert_begin;
  s->El = p->num_local;
  s->act = p->act;
  s->weight = p->weight;
  s->blocked = p->weight_layout == MOE_LAYOUT_BLOCKED;
  s->S = S;
  return MOE_OK;
}

bool few_tokens(const Shape& s) { return s.T <= MOE_FEW_MAX_TOKENS && s.S <= MOE_FEW_MAX_SLOTS; }

moe_status_t from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <class... P>
bool all_aligned16(P... p) {
  return (... && aligned16(p));
}

// A gradient list: sizes, types, addresses, and (for clipping) outputs that
// are the tensor itself or overlap no tensor and no other output.
moe_status_t check_grads(const moe_grad_t* g, int32_t n, bool outputs) {
  if (n < 0 || (n > 0 && g == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (n > MOE_GRAD_MAX_TENSORS) return MOE_ERR_UNSUPPORTED;
  struct Range {
    uintptr_t b, e;
    int i;
  };
  Range out[MOE_GRAD_MAX_TENSORS];
  int used = 0;
  for (int i = 0; i < n; ++i) {
    if (g[i].numel < 0) return MOE_ERR_INVALID_ARGUMENT;
    if (g[i].dtype != MOE_F32 && g[i].dtype != MOE_BF16)
      return g[i].dtype > MOE_BF16 && g[i].dtype <= MOE_MXFP4 ? MOE_ERR_UNSUPPORTED
                                                              : MOE_ERR_INVALID_ARGUMENT;
    if (g[i].numel >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
    if (g[i].numel == 0) continue;
    const uintptr_t size = g[i].dtype == MOE_F32 ? 4 : 2;
    const uintptr_t b = reinterpret_cast<uintptr_t>(g[i].grad);
    if (g[i].grad == nullptr || b % size != 0) return MOE_ERR_INVALID_ARGUMENT;
    if (!outputs) continue;
    const uintptr_t o = reinterpret_cast<uintptr_t>(g[i].out);
    if (g[i].out == nullptr || o % size != 0) return MOE_ERR_INVALID_ARGUMENT;
    out[used++] = Range{o, o + size * (uintptr_t)g[i].numel, i};
  }
  if (used == 0) return MOE_OK;
  std::sort(out, out + used, [](const Range& a, const Range& b) { return a.b < b.b; });
  for (int q = 1; q < used; ++q)
    if (out[q].b < out[q - 1].e) return MOE_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < n; ++i) {
    if (g[i].numel == 0) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(g[i].grad);
    const uintptr_t e = b + (g[i].dtype == MOE_F32 ? 4 : 2) * (uintptr_t)g[i].numel;
    // the outputs are disjoint: those that reach into [b, e) end behind b
    int q = (int)(std::upper_bound(out, out + used, b,
                                   [](uintptr_t v, const Range& r) { return v < r.e; }) - out);
    for (; q < used && out[q].b < e; ++q)
      if (out[q].i != i || g[i].out != g[i].grad) return MOE_ERR_INVALID_ARGUMENT;
  }
  return MOE_OK;
}

// Whether the norm's word lies in a tensor of the list (`outputs`: in one that
// clipping writes, which other workgroups would still read it from).
bool norm_in_list(const moe_grad_t* g, int32_t n, const float* norm, bool outputs) {
  const uintptr_t v = reinterpret_cast<uintptr_t>(norm);
  for (int i = 0; i < n; ++i) {
    if (g[i].numel == 0) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(outputs ? g[i].out : g[i].grad);
    const uintptr_t e = b + (g[i].dtype == MOE_F32 ? 4 : 2) * (uintptr_t)g[i].numel;
    if (v < e && v + sizeof(float) > b) return true;
  }
  return false;
}

// Arguments of moe_mx_quantize and moe_mx_dequantize; *none: no values.
moe_status_t check_convert(int32_t batch, int32_t rows, int32_t cols, int32_t dtype,
                           const void* values, const void* codes, const void* scales,
                           int32_t scale_layout, bool* none) {
  if (batch < 0 || rows < 0 || cols <= 0 || cols % 32 != 0) return MOE_ERR_INVALID_ARGUMENT;
  if (scale_layout != MOE_MX_SCALES_ROW && scale_layout != MOE_MX_SCALES_BLOCK)
    return MOE_ERR_INVALID_ARGUMENT;
  if (dtype != MOE_F32 && dtype != MOE_BF16)
    return dtype > MOE_BF16 && dtype <= MOE_MXFP4 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARGUMENT;
  if (cols > 65536 || (long long)batch * rows >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (!all_aligned16(values, codes, scales)) return MOE_ERR_INVALID_ARGUMENT;
  *none = batch == 0 || rows == 0;
  if (!*none && (values == nullptr || codes == nullptr || scales == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// Device-memory layout of the moe_forward workspace.
struct ForwardLayout {
  size_t logits, idx, w, counts, offsets, sorted, pos, y, router, permute, ffn, total;
};

ForwardLayout forward_layout(const Shape& s) {
  ForwardLayout L{};
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += moe::align_up(bytes);
    return at;
  };
  L.logits = take((size_t)s.T * s.E * sizeof(float));
  L.idx = take((size_t)s.S * sizeof(int32_t));
  L.w = take((size_t)s.S * sizeof(float));
  L.counts = take((size_t)s.El * sizeof(int32_t));
  L.offsets = take((size_t)(s.El + 1) * sizeof(int32_t));
  L.sorted = take((size_t)s.S * sizeof(int32_t));
  L.pos = take((size_t)s.S * sizeof(int32_t));
  L.y = take((size_t)s.S * s.d * moe::act_bytes(s));
  L.router = take(moe::route_ws_bytes(s));
  L.permute = take(moe::permute_ws_bytes(s));
  L.ffn = take(moe::ffn_ws_bytes(s));
  L.total = o;
  return L;
}

}  // namespace

extern "C" {

size_t moe_workspace_size(const moe_problem_t* p, int32_t call) {
  Shape s;
  if (check_problem(p, &s) != MOE_OK) return 0;
  switch (call) {
    case MOE_CALL_PERMUTE:
      return moe::permute_ws_bytes(s);
    case MOE_CALL_EXPERT_FFN:
      return moe::ffn_ws_bytes(s);
    case MOE_CALL_FORWARD:
      return forward_layout(s).total;
    case MOE_CALL_ROUTE:
      return moe::route_ws_bytes(s);
    case MOE_CALL_BALANCE_LOSS:
      return moe::balance_ws_bytes(s);
    case MOE_CALL_ROUTE_BACKWARD:
      return moe::route_backward_ws_bytes(s);
    case MOE_CALL_NORM_BACKWARD:
    case MOE_CALL_COMBINE_NORM_BACKWARD:
      return moe::norm_grad_ws_bytes(s);
    case MOE_CALL_EXPERT_FFN_MX:
      return s.weight == MOE_MXFP4 ? moe::mx_ffn_ws_bytes(s) : 0;
    case MOE_CALL_FORWARD_FEW:
      return few_tokens(s) ? moe::few_ws_bytes(s) : 0;
    default:
      return 0;
  }
}

const char* moe_status_string(moe_status_t s) {
  switch (s) {
    case MOE_OK:
      return "MOE_OK";
    case MOE_ERR_INVALID_ARGUMENT:
      return "MOE_ERR_INVALID_ARGUMENT";
    case MOE_ERR_UNSUPPORTED:
      return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_WORKSPACE_TOO_SMALL:
      return "MOE_ERR_WORKSPACE_TOO_SMALL";
    case MOE_ERR_HIP:
      return "MOE_ERR_HIP";
  }
  return "MOE_ERR_UNKNOWN";
}

moe_status_t moe_route(const moe_problem_t* p, const void* x, const void* w_router,
                       const float* router_bias, float* logits, int32_t* topk_idx,
                       float* topk_w, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (topk_idx == nullptr || topk_w == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (w_router != nullptr && x == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (logits == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (w_router != nullptr) {
    const size_t need = moe::route_ws_bytes(s);
    if (need > 0 && ws == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (s.T == 0) return MOE_OK;
  const float* lin = w_router == nullptr ? logits : nullptr;
  return from_hip(moe::route(s, x, w_router, router_bias, lin, logits, topk_idx, topk_w, ws,
                             static_cast<hipStream_t>(stream)));
}

moe_status_t moe_permute(const moe_problem_t* p, const int32_t* topk_idx, int32_t* counts,
                         int32_t* offsets, int32_t* sorted_slot, int32_t* slot_pos, void* ws,
                         size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (topk_idx == nullptr || counts == nullptr || offsets == nullptr || sorted_slot == nullptr ||
      slot_pos == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = moe::permute_ws_bytes(s);
  if (need > 0 && ws == nullptr) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (s.T == 0) return MOE_OK;
  return from_hip(moe::permute(s, topk_idx, counts, offsets, sorted_slot, slot_pos, ws,
                               static_cast<hipStream_t>(stream)));
}

moe_status_t moe_expert_ffn(const moe_problem_t* p, const void* x, const int32_t* sorted_slot,
                            const int32_t* offsets, const void* w_gate, const void* w_up,
                            const void* w_down, const void* s_gate, const void* s_up,
                            const void* s_down, const float* topk_w, void* y, void* ws,
                            size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (x == nullptr || sorted_slot == nullptr || offsets == nullptr || w_gate == nullptr ||
      w_up == nullptr || w_down == nullptr || y == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if ((s.weight == MOE_FP8_E4M3 || s.weight == MOE_MXFP4) &&
      (s_gate == nullptr || s_up == nullptr || s_down == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = moe::ffn_ws_bytes(s);
  if (ws == nullptr || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (s.T == 0) return MOE_OK;
  return from_hip(moe::expert_ffn(s, x, sorted_slot, offsets, w_gate, w_up, w_down, s_gate, s_up,
                                  s_down, topk_w, y, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine(const moe_problem_t* p, const void* y, const int32_t* slot_pos,
                         const float* topk_w, void* out, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (y == nullptr || slot_pos == nullptr || out == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (s.T == 0) return MOE_OK;
  return from_hip(moe::combine(s, y, slot_pos, topk_w, out, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_forward(const moe_problem_t* p, const moe_forward_args_t* a, void* ws,
                         size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (a == nullptr || a->x == nullptr || a->w_gate == nullptr || a->w_up == nullptr ||
      a->w_down == nullptr || a->out == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (a->w_router == nullptr && a->logits == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if ((s.weight == MOE_FP8_E4M3 || s.weight == MOE_MXFP4) &&
      (a->s_gate == nullptr || a->s_up == nullptr || a->s_down == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  const ForwardLayout L = forward_layout(s);
  if (ws == nullptr || ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (s.T == 0) return MOE_OK;
  hipStream_t strm = static_cast<hipStream_t>(stream);
  unsigned char* base = static_cast<unsigned char*>(ws);
  auto pick = [base](void* user, size_t off) { return user ? user : static_cast<void*>(base + off); };
  float* logits = static_cast<float*>(pick(a->logits, L.logits));
  int32_t* idx = static_cast<int32_t*>(pick(a->topk_idx, L.idx));
  float* gw = static_cast<float*>(pick(a->topk_w, L.w));
  int32_t* counts = static_cast<int32_t*>(pick(a->counts, L.counts));
  int32_t* offsets = static_cast<int32_t*>(pick(a->offsets, L.offsets));
  int32_t* sorted = static_cast<int32_t*>(pick(a->sorted_slot, L.sorted));
  int32_t* pos = static_cast<int32_t*>(pick(a->slot_pos, L.pos));
  void* y = base + L.y;

  const float* lin = a->w_router == nullptr ? a->logits : nullptr;
  float* lout = a->w_router == nullptr ? nullptr : logits;
  hipEvent_t ev[MOE_FORWARD_EVENTS];
  if (a->events)
    for (int i = 0; i < MOE_FORWARD_EVENTS; ++i) ev[i] = static_cast<hipEvent_t>(a->events[i]);
  auto mark = [&](int i) { return a->events ? hipEventRecord(ev[i], strm) : hipSuccess; };
  hipError_t e = mark(0);
  if (e == hipSuccess)
    e = moe::route(s, a->x, a->w_router, a->router_bias, lin, lout, idx, gw, base + L.router,
                   strm);
  if (e == hipSuccess) e = mark(1);
  const moe::FfnSchedule sched = moe::ffn_schedule_view(s, base + L.ffn);
  bool sched_ready = false;
  if (e == hipSuccess)
    e = moe::permute(s, idx, counts, offsets, sorted, pos, base + L.permute, strm, &sched,
                     &sched_ready);
  if (e == hipSuccess) e = mark(2);
  if (e == hipSuccess)
    e = moe::expert_ffn(s, a->x, sorted, offsets, a->w_gate, a->w_up, a->w_down, a->s_gate,
                        a->s_up, a->s_down, gw, y, base + L.ffn, strm, sched_ready,
                        a->events ? ev + 3 : nullptr);
  if (e == hipSuccess) e = moe::combine(s, y, pos, nullptr, a->out, strm);
  if (e == hipSuccess) e = mark(6);
  return from_hip(e);
}

moe_status_t moe_forward_few(const moe_problem_t* p, const moe_forward_args_t* a, void* ws,
                             size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (a == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (!few_tokens(s)) return MOE_ERR_UNSUPPORTED;
  if (a->counts != nullptr || a->offsets != nullptr || a->sorted_slot != nullptr ||
      a->slot_pos != nullptr || a->events != nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!all_aligned16(a->x, a->w_router, a->router_bias, a->w_gate, a->w_up, a->w_down, a->s_gate,
                     a->s_up, a->s_down, a->out, a->logits, a->topk_idx, a->topk_w, ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (a->w_gate == nullptr || a->w_up == nullptr || a->w_down == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if ((s.weight == MOE_FP8_E4M3 || s.weight == MOE_MXFP4) &&
      (a->s_gate == nullptr || a->s_up == nullptr || a->s_down == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0 && (a->x == nullptr || a->out == nullptr ||
                  (a->w_router == nullptr && a->logits == nullptr)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0 && (a->out == a->x || (a->logits != nullptr && a->logits == a->topk_w)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws == nullptr || ws_bytes < moe::few_ws_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (s.T == 0) return MOE_OK;
  return from_hip(moe::forward_few(s, *a, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_balance_loss(const moe_problem_t* p, const float* logits, const int32_t* topk_idx,
                              const uint8_t* token_mask, int32_t* counts, int32_t* n_tokens,
                              float* prob_mean, float* losses, void* ws, size_t ws_bytes,
                              void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (counts == nullptr || n_tokens == nullptr || prob_mean == nullptr || losses == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0 && (logits == nullptr || topk_idx == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (!all_aligned16(logits, topk_idx, token_mask, counts, n_tokens, prob_mean, losses, ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws == nullptr || ws_bytes < moe::balance_ws_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return from_hip(moe::balance_loss(s, logits, topk_idx, token_mask, counts, n_tokens, prob_mean,
                                    losses, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_route_backward(const moe_problem_t* p, const moe_route_backward_args_t* a,
                                void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (a == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  // (arrays of no tokens may be null)
  if (s.T > 0 && a->dtopk_w == nullptr && a->dlosses == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0 && a->dlogits == nullptr && a->dx == nullptr && a->dw_router == nullptr &&
      a->dbias == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (a->dlogits != nullptr && a->dlogits == a->logits) return MOE_ERR_INVALID_ARGUMENT;
  if (a->dx != nullptr && a->dx == a->x) return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0) {
    if (a->dtopk_w != nullptr && (a->topk_idx == nullptr || a->topk_w == nullptr))
      return MOE_ERR_INVALID_ARGUMENT;
    if (a->dlosses != nullptr &&
        (a->logits == nullptr || a->counts == nullptr || a->n_tokens == nullptr))
      return MOE_ERR_INVALID_ARGUMENT;
    if (a->dw_router != nullptr && a->x == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (a->dx != nullptr && a->w_router == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  }
  if (!all_aligned16(a->x, a->w_router, a->logits, a->topk_idx, a->topk_w, a->dtopk_w,
                     a->token_mask, a->counts, a->n_tokens, a->dlosses, a->dlogits, a->dx,
                     a->dw_router, a->dbias, ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws == nullptr || ws_bytes < moe::route_backward_ws_bytes(s))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  moe::RouteGradArgs g{};
  g.gate.logits = a->logits;
  g.gate.idx = a->topk_idx;
  g.gate.topk_w = a->topk_w;
  g.gate.dtopk_w = a->dtopk_w;
  g.gate.mask = a->token_mask;
  g.gate.counts = a->counts;
  g.gate.n_tokens = a->n_tokens;
  g.gate.dlosses = a->dlosses;
  g.x = a->x;
  g.w_router = a->w_router;
  g.dlogits = a->dlogits;
  g.dx = a->dx;
  g.dw = a->dw_router;
  g.dbias = a->dbias;
  return from_hip(moe::route_backward(s, g, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine_backward(const moe_problem_t* p, const void* dout, const void* y,
                                  const int32_t* slot_pos, const float* topk_w, void* dy,
                                  float* dtopk_w, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (s.T == 0) return MOE_OK;
  if (dout == nullptr || slot_pos == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (dy == nullptr && dtopk_w == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (dtopk_w != nullptr && y == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (dy != nullptr && (dy == y || dy == dout)) return MOE_ERR_INVALID_ARGUMENT;
  if (!all_aligned16(dout, y, slot_pos, topk_w, dy, dtopk_w)) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::combine_backward(s, dout, y, slot_pos, topk_w, dy, dtopk_w,
                                        static_cast<hipStream_t>(stream)));
}

size_t moe_grad_workspace_size(const moe_grad_t* g, int32_t n) {
  return check_grads(g, n, false) == MOE_OK ? moe::grad_ws_bytes(g, n) : 0;
}

moe_status_t moe_grad_norm(const moe_grad_t* g, int32_t n, float* norm, void* ws, size_t ws_bytes,
                           void* stream) {
  const moe_status_t st = check_grads(g, n, false);
  if (st != MOE_OK) return st;
  if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4 != 0 || !aligned16(ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws == nullptr || ws_bytes < moe::grad_ws_bytes(g, n)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (norm_in_list(g, n, norm, false)) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::grad_norm(g, n, norm, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_grad_clip(const moe_grad_t* g, int32_t n, const float* norm, float max_norm,
                           void* stream) {
  const moe_status_t st = check_grads(g, n, true);
  if (st != MOE_OK) return st;
  if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4 != 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!(max_norm > 0.0f) || norm_in_list(g, n, norm, true)) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::grad_clip(g, n, norm, max_norm, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_norm(const moe_problem_t* p, const void* h, const float* weight, float eps,
                      void* x, float* rstd, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (!(eps > 0.0f) || !all_aligned16(h, weight, x, rstd)) return MOE_ERR_INVALID_ARGUMENT;
  if (s.T == 0) return MOE_OK;
  if (h == nullptr || weight == nullptr || x == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::norm(s, h, weight, eps, x, rstd, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_norm_backward(const moe_problem_t* p, const moe_norm_backward_args_t* a, void* ws,
                               size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (a == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (!all_aligned16(a->dx, a->h, a->weight, a->rstd, a->dout, a->dh, a->dweight, ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0) {
    if (a->dx == nullptr || a->h == nullptr || a->weight == nullptr || a->rstd == nullptr)
      return MOE_ERR_INVALID_ARGUMENT;
    if ((a->dh == nullptr && a->dweight == nullptr) || a->dh == a->h)
      return MOE_ERR_INVALID_ARGUMENT;
  }
  if (ws == nullptr || ws_bytes < moe::norm_grad_ws_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return from_hip(moe::norm_backward(s, *a, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine_norm(const moe_problem_t* p, const moe_combine_norm_args_t* a,
                              void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (a == nullptr || !(a->eps > 0.0f)) return MOE_ERR_INVALID_ARGUMENT;
  if (!all_aligned16(a->y, a->slot_pos, a->topk_w, a->h, a->weight, a->gate, a->out, a->rstd,
                     a->next_weight, a->next_x, a->next_rstd))
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T == 0) return MOE_OK;
  if (a->y == nullptr || a->h == nullptr || a->weight == nullptr || a->out == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (a->slot_pos == nullptr && s.k != 1) return MOE_ERR_INVALID_ARGUMENT;
  if (a->next_weight == nullptr ? a->next_x != nullptr || a->next_rstd != nullptr
                                : a->next_x == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (a->out == a->y || a->next_x == a->out || (a->next_x != nullptr && a->next_x == a->y) ||
      (a->rstd != nullptr && a->rstd == a->next_rstd))
    return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::combine_norm(s, *a, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine_norm_backward(const moe_problem_t* p,
                                       const moe_combine_norm_backward_args_t* a, void* ws,
                                       size_t ws_bytes, void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (a == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (!all_aligned16(a->dout, a->y, a->slot_pos, a->topk_w, a->weight, a->rstd, a->gate, a->dy,
                     a->dtopk_w, a->dweight, a->dgate, ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0) {
    if (a->dout == nullptr || a->y == nullptr || a->weight == nullptr || a->rstd == nullptr)
      return MOE_ERR_INVALID_ARGUMENT;
    if (a->dy == nullptr && a->dtopk_w == nullptr && a->dweight == nullptr && a->dgate == nullptr)
      return MOE_ERR_INVALID_ARGUMENT;
    if (a->slot_pos == nullptr && (s.k != 1 || a->dtopk_w != nullptr))
      return MOE_ERR_INVALID_ARGUMENT;
    if (a->dy != nullptr && (a->dy == a->y || a->dy == a->dout)) return MOE_ERR_INVALID_ARGUMENT;
  }
  if (ws == nullptr || ws_bytes < moe::norm_grad_ws_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return from_hip(moe::combine_norm_backward(s, *a, ws, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_mx_quantize(int32_t batch, int32_t rows, int32_t cols, int32_t dtype,
                             const void* src, void* codes, void* scales, int32_t scale_layout,
                             void* stream) {
  bool none = false;
  const moe_status_t st =
      check_convert(batch, rows, cols, dtype, src, codes, scales, scale_layout, &none);
  if (st != MOE_OK || none) return st;
  if (codes == src || scales == src || codes == scales) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::mx_quantize(batch, rows, cols, dtype == MOE_BF16, src,
                                   static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                   scale_layout, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_mx_dequantize(int32_t batch, int32_t rows, int32_t cols, int32_t dtype,
                               const void* codes, const void* scales, void* dst,
                               int32_t scale_layout, void* stream) {
  bool none = false;
  const moe_status_t st =
      check_convert(batch, rows, cols, dtype, dst, codes, scales, scale_layout, &none);
  if (st != MOE_OK || none) return st;
  if (dst == codes || dst == scales) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::mx_dequantize(batch, rows, cols, dtype == MOE_BF16,
                                     static_cast<const uint8_t*>(codes),
                                     static_cast<const uint8_t*>(scales), dst, scale_layout,
                                     static_cast<hipStream_t>(stream)));
}

moe_status_t moe_expert_ffn_mx(const moe_problem_t* p, const void* x_codes, const void* x_scales,
                               const int32_t* sorted_slot, const int32_t* offsets,
                               const void* w_gate, const void* w_up, const void* w_down,
                               const void* s_gate, const void* s_up, const void* s_down,
                               const float* topk_w, void* y, void* ws, size_t ws_bytes,
                               void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (s.weight != MOE_MXFP4) return MOE_ERR_UNSUPPORTED;
  if (!all_aligned16(x_codes, x_scales, sorted_slot, offsets, w_gate, w_up, w_down, s_gate, s_up,
                     s_down, topk_w, y, ws))
    return MOE_ERR_INVALID_ARGUMENT;
  if (w_gate == nullptr || w_up == nullptr || w_down == nullptr || s_gate == nullptr ||
      s_up == nullptr || s_down == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (s.T > 0 && (x_codes == nullptr || x_scales == nullptr || sorted_slot == nullptr ||
                  offsets == nullptr || y == nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws == nullptr || ws_bytes < moe::mx_ffn_ws_bytes(s)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (s.T == 0) return MOE_OK;
  return from_hip(moe::expert_ffn_mx(s, static_cast<const uint8_t*>(x_codes),
                                     static_cast<const uint8_t*>(x_scales), sorted_slot, offsets,
                                     w_gate, w_up, w_down, s_gate, s_up, s_down, topk_w, y, ws,
                                     static_cast<hipStream_t>(stream)));
}

moe_status_t moe_pack_weights(const moe_problem_t* p, int32_t which, const void* src, void* dst,
                              void* stream) {
  Shape s;
  moe_status_t st = check_problem(p, &s);
  if (st != MOE_OK) return st;
  if (which != 0 && which != 1) return MOE_ERR_INVALID_ARGUMENT;
  if (s.weight == MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (src == nullptr || dst == nullptr || src == dst) return MOE_ERR_INVALID_ARGUMENT;
  return from_hip(moe::pack_weights(s, which, src, dst, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_eplb_plan(const int64_t* load, int32_t E, int32_t G, int32_t R,
                           int32_t* replicas, int32_t* phys_to_log, int32_t* log_to_phys,
                           double* rank_load) {
  if (load == nullptr || replicas == nullptr || phys_to_log == nullptr || log_to_phys == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (E < 1 || G < 1 || R < 0 || (long long)R > (long long)E * (G - 1))
    return MOE_ERR_INVALID_ARGUMENT;
  if (((long long)E + R) % G != 0) return MOE_ERR_INVALID_ARGUMENT;
  if ((long long)E + R > moe::kMaxExperts) return MOE_ERR_UNSUPPORTED;
  for (int e = 0; e < E; ++e)
    if (load[e] < 0 || load[e] >= (1LL << 40)) return MOE_ERR_INVALID_ARGUMENT;
  try {
    moe::eplb_plan(load, E, G, R, replicas, phys_to_log, log_to_phys, rank_load);
  } catch (const std::bad_alloc&) {
    return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

moe_status_t moe_eplb_remap(int32_t T, int32_t k, int32_t E, int32_t G, const int32_t* topk_idx,
                            const int32_t* replicas, const int32_t* log_to_phys,
                            int32_t* topk_phys, void* stream) {
  if (T < 0 || k < 1 || E < 1 || G < 1) return MOE_ERR_INVALID_ARGUMENT;
  if ((long long)T * k >= (1LL << 31) || (long long)E * G >= (1LL << 31))
    return MOE_ERR_UNSUPPORTED;
  if (topk_idx == nullptr || replicas == nullptr || log_to_phys == nullptr || topk_phys == nullptr)
    return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0) return MOE_OK;
  return from_hip(moe::eplb_remap(T, k, E, G, topk_idx, replicas, log_to_phys, topk_phys,
                                  static_cast<hipStream_t>(stream)));
}

}  // extern "C"

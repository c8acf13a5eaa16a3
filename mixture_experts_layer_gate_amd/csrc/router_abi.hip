// C entry points of the scored router, its losses and gradients, and the
// dropout beside the combine: argument validation, workspace and launches.
// Declarations and the contract of each entry point are in include/moe.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe.h"
#include "abi_host.h"
#include "kernels.h"
#include "router.h"

namespace moe {
namespace {

int check_opts(const moe_dims_t* dm, const moe_route_opts_t* op, SelectOpts* o) {
  if (!op) return MOE_ERR_INVALID;
  if (op->score != MOE_SCORE_SOFTMAX && op->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID;
  if (op->group_rule != MOE_GROUP_MAX && op->group_rule != MOE_GROUP_TOP2) return MOE_ERR_INVALID;
  if (op->renormalise != 0 && op->renormalise != 1) return MOE_ERR_INVALID;
  if (op->groups < 1 || op->groups > kMaxGroups || dm->E % op->groups != 0) return MOE_ERR_INVALID;
  if (op->topk_groups < 1 || op->topk_groups > op->groups) return MOE_ERR_INVALID;
  if (int64_t(op->topk_groups) * (dm->E / op->groups) < dm->k) return MOE_ERR_INVALID;
  if (!isfinite(op->scale)) return MOE_ERR_INVALID;
  o->sigmoid = op->score == MOE_SCORE_SIGMOID;
  // every group kept is no grouping
  o->groups = op->topk_groups == op->groups ? 1 : op->groups;
  o->topk_groups = o->groups == 1 ? 1 : op->topk_groups;
  o->top2 = op->group_rule == MOE_GROUP_TOP2;
  o->renorm = op->renormalise;
  o->scale = op->scale;
  o->per = dm->E / o->groups;
  o->lpg_log2 = 0;
  while ((2 << o->lpg_log2) * o->groups <= 64) ++o->lpg_log2;
  o->inv_per = 1.0f / static_cast<float>(o->per);
  return MOE_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return MOE_ERR_INVALID;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

int check_seqs(const int32_t* seq_offsets, int32_t n_seq) {
  if (n_seq < 1 || (!seq_offsets && n_seq != 1) || !ok4_or_null(seq_offsets)) return MOE_ERR_INVALID;
  return n_seq > kMaxSeqs ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

struct BalanceWs {
  int parts;
  float* p;
  int32_t* f;
  double* z;
  double* term;
  uint32_t* done;
};
size_t balance_ws(const moe_dims_t* dm, int n_seq, void* ws, BalanceWs* out) {
  Carver c(ws);
  BalanceWs r{};
  r.parts = balance_parts(dm->T, n_seq, dm->E);
  const size_t np = size_t(n_seq) * r.parts;
  r.p = c.take<float>(sizeof(float) * np * dm->E);
  r.f = c.take<int32_t>(sizeof(int32_t) * np * dm->E);
  r.z = c.take<double>(sizeof(double) * np);
  r.term = c.take<double>(sizeof(double) * n_seq * (balance_blocks(dm->E) + 1));
  r.done = c.take<uint32_t>(sizeof(uint32_t));
  if (out) *out = r;
  return c.off;
}

int check_drop(double p, const uint64_t* rng, DropArgs* a) {
  if (!(p >= 0.0 && p <= 1.0) || !ok8(rng)) return MOE_ERR_INVALID;
  a->rng = rng;
  a->thr = static_cast<uint32_t>(lrint(p * 65536.0));
  a->scale = a->thr < 65536 ? static_cast<float>(65536.0 / (65536.0 - a->thr)) : 0.0f;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_route_select(const moe_dims_t* dm, const moe_route_opts_t* opts, const float* logits,
                     const float* balance_bias, int32_t* topk_idx, float* topk_w, void* stream) {
  if (int st = check_dims(dm)) return st;
  SelectOpts o{};
  if (int st = check_opts(dm, opts, &o)) return st;
  if (!ok4_or_null(balance_bias)) return MOE_ERR_INVALID;
  if (dm->T == 0) return MOE_OK;
  if (!ok4(logits) || !ok4(topk_idx) || !ok4(topk_w)) return MOE_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_SELECT, s);
  return hip_status(launch_select(o, logits, balance_bias, dm->T, dm->E, dm->k, topk_idx, topk_w, s));
}

int moe_route_scored(const moe_dims_t* dm, const moe_route_opts_t* opts, const void* x, const void* wg,
                     const float* bias, const float* balance_bias, float* logits, int32_t* topk_idx, float* topk_w,
                     void* stream) {
  if (int st = check_dims(dm)) return st;
  SelectOpts o{};
  if (int st = check_opts(dm, opts, &o)) return st;
  if (dm->T == 0) return MOE_OK;
  if (!ok16(x) || !ok16(wg) || !ok4_or_null(bias) || !ok4_or_null(balance_bias) || !ok4(logits) || !ok4(topk_idx) ||
      !ok4(topk_w))
    return MOE_ERR_INVALID;
  if (dm->d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  {
    StageScope sc(MOE_STAGE_GATE, s);
    if (int st = hip_status(launch_gate_logits(dm->dtype, x, wg, bias, logits, dm->T, dm->d, dm->E, s))) return st;
  }
  StageScope sc(MOE_STAGE_SELECT, s);
  return hip_status(launch_select(o, logits, balance_bias, dm->T, dm->E, dm->k, topk_idx, topk_w, s));
}

size_t moe_balance_workspace_bytes(const moe_dims_t* dm, int32_t n_seq) {
  if (check_dims(dm) != MOE_OK || n_seq < 1 || n_seq > kMaxSeqs) return 0;
  return balance_ws(dm, n_seq, nullptr, nullptr);
}

int moe_balance_loss(const moe_dims_t* dm, const moe_route_opts_t* opts, const float* logits, const int32_t* topk_idx,
                     const int32_t* seq_offsets, int32_t n_seq, float* losses, int32_t* load, void* ws,
                     size_t ws_bytes, void* stream) {
  if (int st = check_dims(dm)) return st;
  SelectOpts o{};
  if (int st = check_opts(dm, opts, &o)) return st;
  if (int st = check_seqs(seq_offsets, n_seq)) return st;
  if (!ok4(losses) || !ok4(load)) return MOE_ERR_INVALID;
  if (dm->T > 0 && (!ok4(logits) || !ok4(topk_idx))) return MOE_ERR_INVALID;
  if (int st = check_ws(ws, ws_bytes, balance_ws(dm, n_seq, nullptr, nullptr))) return st;
  BalanceWs b{};
  balance_ws(dm, n_seq, ws, &b);
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_BALANCE, s);
  return hip_status(launch_balance(o, logits, topk_idx, seq_offsets, n_seq, dm->T, dm->E, dm->k, b.parts, b.p, b.f, b.z,
                                   b.term, b.done, losses, load, s));
}

int moe_route_select_backward(const moe_dims_t* dm, const moe_route_opts_t* opts, const float* logits,
                              const int32_t* topk_idx, const float* topk_w, const float* dtopk_w,
                              const float* dlosses, const int32_t* load, const int32_t* seq_offsets, int32_t n_seq,
                              float* dlogits, void* stream) {
  if (int st = check_dims(dm)) return st;
  SelectOpts o{};
  if (int st = check_opts(dm, opts, &o)) return st;
  if (!ok4_or_null(topk_idx) || !ok4_or_null(topk_w) || !ok4_or_null(dtopk_w) || !ok4_or_null(dlosses) ||
      !ok4_or_null(load))
    return MOE_ERR_INVALID;
  if (dlosses) {
    if (!load) return MOE_ERR_INVALID;
    if (int st = check_seqs(seq_offsets, n_seq)) return st;
  }
  if (dm->T == 0) return MOE_OK;
  if (!ok4(logits) || !ok4(dlogits)) return MOE_ERR_INVALID;
  if (dtopk_w && (!topk_idx || !topk_w)) return MOE_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_SELECT_BWD, s);
  return hip_status(launch_select_backward(o, logits, topk_idx, topk_w, dtopk_w, dlosses, load, seq_offsets,
                                           dlosses ? n_seq : 1, dm->T, dm->E, dm->k, dlogits, s));
}

size_t moe_gate_backward_workspace_bytes(const moe_dims_t* dm) {
  if (check_dims(dm) != MOE_OK || !gate_backward_fits(dm->T, dm->d)) return 0;
  return gate_backward_ws(dm->T, dm->d, dm->E);
}

int moe_gate_backward(const moe_dims_t* dm, const void* x, const void* wg, const float* dlogits, const void* dx_in,
                      void* dx, float* dwg, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_dims(dm)) return st;
  if (!ok16(wg) || !ok16(dwg) || !ok4(dbias)) return MOE_ERR_INVALID;
  if (dm->T > 0 && (!ok16(x) || !ok4(dlogits) || !ok16(dx) || (dx_in && !ok16(dx_in)))) return MOE_ERR_INVALID;
  if (dm->dtype != MOE_DTYPE_BF16 || dm->d % 8 != 0 || !gate_backward_fits(dm->T, dm->d)) return MOE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_GATE_BWD, s);
  if (dm->T == 0) {
    if (int st = hip_status(launch_fill_zero(dwg, dm->E * dm->d, s))) return st;
    return hip_status(launch_fill_zero(dbias, dm->E, s));
  }
  if (int st = check_ws(ws, ws_bytes, gate_backward_ws(dm->T, dm->d, dm->E))) return st;
  return hip_status(launch_gate_backward(x, wg, dlogits, dx_in, dx, dwg, dbias, dm->T, dm->d, dm->E, ws, s));
}

int moe_combine_dropout(const moe_dims_t* dm, double p, const uint64_t* rng, const void* y_sorted,
                        const int32_t* inv_perm, const float* topk_w, const void* residual, void* out, void* stream) {
  if (int st = check_dims(dm)) return st;
  DropArgs a{};
  if (int st = check_drop(p, rng, &a)) return st;
  if (dm->T == 0) return MOE_OK;
  if (!ok16(y_sorted) || !ok4(inv_perm) || !ok4(topk_w) || (residual && !ok16(residual)) || !ok16(out))
    return MOE_ERR_INVALID;
  if (dm->d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_COMBINE_DROP, s);
  return hip_status(
      launch_combine_dropout(dm->dtype, a, y_sorted, inv_perm, topk_w, residual, out, dm->T, dm->d, dm->k, s));
}

int moe_dropout_backward(const moe_dims_t* dm, double p, const uint64_t* rng, const void* dout, void* dy,
                         void* stream) {
  if (int st = check_dims(dm)) return st;
  DropArgs a{};
  if (int st = check_drop(p, rng, &a)) return st;
  if (dm->T == 0) return MOE_OK;
  if (!ok16(dout) || !ok16(dy)) return MOE_ERR_INVALID;
  if (dm->d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_DROP_BWD, s);
  return hip_status(launch_dropout_backward(dm->dtype, a, dout, dy, dm->T, dm->d, s));
}

}  // extern "C"

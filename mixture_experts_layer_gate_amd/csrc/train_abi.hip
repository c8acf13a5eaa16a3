// C entry points of the norm, the gradients' 2-norm and the AdamW update:
// argument validation, workspace and launches. Declarations and the contract of
// each entry point are in include/moe.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <new>

#include "moe.h"
#include "abi_host.h"
#include "kernels.h"
#include "train.h"

namespace moe {
namespace {

constexpr int32_t kMostTensors = 1 << 20;

bool ok_dtype(int64_t t) { return t == MOE_DTYPE_F32 || t == MOE_DTYPE_BF16; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ok_elements(const void* p, int64_t dtype) { return p && aligned(p, dtype == MOE_DTYPE_F32 ? 4 : 2); }
int64_t size_of(int64_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// How a list is cut, from its elements and the bytes that a call moves
// (each(t): those of an element).
struct Cut {
  int chunk;
  bool stream;
};
template <typename Item, typename Fn>
Cut cut_of(const Item* t, int32_t count, int chunk, Fn&& each) {
  double n = 0, bytes = 0;
  for (int32_t i = 0; i < count; ++i) {
    n += static_cast<double>(t[i].n);
    bytes += static_cast<double>(t[i].n) * static_cast<double>(each(i));
  }
  return {n <= kListSmall ? kRound : chunk, bytes >= kListStream};
}
int64_t chunks_of(int64_t n, int chunk) { return (n + chunk - 1) / chunk; }

int check_norm(const moe_dims_t* dm, const moe_norm_opts_t* op) {
  if (int st = check_dims(dm)) return st;
  if (!op) return MOE_ERR_INVALID;
  if (op->kind != MOE_NORM_RMS && op->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID;
  if (!ok_dtype(op->param_dtype)) return MOE_ERR_INVALID;
  if (!(op->eps >= 0x1p-100f && op->eps <= 0x1p100f)) return MOE_ERR_INVALID;
  return dm->d % 8 != 0 || dm->d > kNormMaxCols ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool ok16_or_null(const void* p) { return !p || ok16(p); }

// Parts of the weight gradients: dweight's, then dbias's (layer norm). Where columns
// are summed beside the rows there are none, and a row's width of each is asked for all
// the same (so that every call has its check); rows over 8192 columns keep a number to
// each row there (norm_grad_shifts).
size_t norm_ws(const moe_dims_t* dm, bool layer, void* ws, float** w, float** b, float** shift) {
  const int parts = norm_grad_parts(dm->dtype, dm->T, dm->d);
  Carver c(ws);
  float* first = c.take<float>(sizeof(float) * (parts ? parts : 1) * dm->d);
  float* second = layer || !parts ? c.take<float>(sizeof(float) * (parts ? parts : 1) * dm->d) : nullptr;
  const bool shifts = norm_grad_shifts(dm->dtype, layer, dm->T, dm->d);
  if (w) *w = first;
  if (b) *b = second;
  if (shift) *shift = shifts ? first : nullptr;
  const size_t rows = shifts ? align_up(sizeof(float) * static_cast<size_t>(dm->T)) : 0;
  return rows > c.off ? rows : c.off;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, kAlign)) return MOE_ERR_INVALID;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

int check_grads(const moe_grad_t* g, int32_t count) {
  if (count < 0 || (count > 0 && !g)) return MOE_ERR_INVALID;
  if (count > kMostTensors) return MOE_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].n < 0 || !ok_dtype(g[i].dtype)) return MOE_ERR_INVALID;
    if (g[i].n > 0 && !ok_elements(g[i].grad, g[i].dtype)) return MOE_ERR_INVALID;
    if (g[i].n > kListElements) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

// Workgroups of one launch of square sums, and the parts of a list: its launches
// take up to kGradTensors tensors each.
int square_grid(int64_t chunks) { return static_cast<int>(chunks < kNormGrid ? chunks : kNormGrid); }

template <typename Fn>
int each_grad_table(const moe_grad_t* g, int32_t count, const Cut& cut, Fn&& fn) {
  GradTable t;
  t.count = 0;
  t.chunks = 0;
  t.chunk = cut.chunk;
  for (int32_t i = 0; i <= count; ++i) {
    if (i == count || t.count == kGradTensors) {
      if (t.count > 0)
        if (int st = fn(t)) return st;
      t.count = 0;
      t.chunks = 0;
      if (i == count) break;
    }
    if (g[i].n == 0) continue;
    const bool bf16 = g[i].dtype == MOE_DTYPE_BF16;
    t.t[t.count++] = {g[i].grad, g[i].n, t.chunks, (bf16 ? 1u : 0u) | (aligned(g[i].grad, 16) ? 2u : 0u)};
    t.chunks += static_cast<uint32_t>(chunks_of(g[i].n, cut.chunk));
  }
  return MOE_OK;
}

Cut grad_cut(const moe_grad_t* g, int32_t count) {
  return cut_of(g, count, kListChunk, [&](int32_t i) { return size_of(g[i].dtype); });
}

int64_t grad_parts(const moe_grad_t* g, int32_t count) {
  int64_t parts = 0;
  each_grad_table(g, count, grad_cut(g, count), [&](const GradTable& t) {
    parts += square_grid(t.chunks);
    return 0;
  });
  return parts;
}

// Whether a buffer that is written appears twice: an open-addressed table of the
// addresses seen.
struct Seen {
  const void** slot = nullptr;
  size_t mask = 0;
  ~Seen() { delete[] slot; }
  bool make(size_t entries) {
    size_t n = 16;
    while (n < 2 * entries) n *= 2;
    slot = new (std::nothrow) const void*[n]();
    mask = n - 1;
    return slot != nullptr;
  }
  // the slot of p: its own, or an empty one
  const void*& at(const void* p) {
    size_t h = (reinterpret_cast<uintptr_t>(p) * 0x9E3779B97F4A7C15ull) >> 20;
    while (slot[h & mask] && slot[h & mask] != p) ++h;
    return slot[h & mask];
  }
  bool has(const void* p) { return at(p) != nullptr; }
  bool again(const void* p) {
    const void*& s = at(p);
    if (s) return true;
    s = p;
    return false;
  }
};

int check_tensors(const moe_adam_tensor_t* t, int32_t count, int bits, bool with_params) {
  if (count < 0 || (count > 0 && !t)) return MOE_ERR_INVALID;
  if (count > kMostTensors) return MOE_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adam_tensor_t& a = t[i];
    if (a.n < 0) return MOE_ERR_INVALID;
    if (a.n > kAdamElements) return MOE_ERR_UNSUPPORTED;
    if (with_params && !ok_dtype(a.dtype)) return MOE_ERR_INVALID;
    if (a.n == 0) continue;
    if (with_params) {
      if (!ok_elements(a.param, a.dtype)) return MOE_ERR_INVALID;
      if (a.master && (a.dtype != MOE_DTYPE_BF16 || !aligned(a.master, 4))) return MOE_ERR_INVALID;
    }
    if (bits == 32 ? !ok4(a.m) || !ok4(a.v) : !a.m || !a.v || !a.m_scale || !a.v_scale) return MOE_ERR_INVALID;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_forward(const moe_dims_t* dm, const moe_norm_opts_t* op, const void* x, const void* residual,
                     const void* weight, const void* bias, void* sum, void* y, float* mean, float* rstd,
                     void* stream) {
  if (int st = check_norm(dm, op)) return st;
  const bool layer = op->kind == MOE_NORM_LAYER;
  if (!ok16_or_null(weight) || !ok16_or_null(bias) || !ok4_or_null(mean) || !ok4_or_null(rstd)) return MOE_ERR_INVALID;
  if (!layer && (bias || mean)) return MOE_ERR_INVALID;
  if (dm->T == 0) return MOE_OK;
  if (!ok16(x) || !ok16(y) || !ok16_or_null(residual) || !ok16_or_null(sum)) return MOE_ERR_INVALID;
  if (sum && sum == y) return MOE_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_NORM, s);
  const NormArgs a = {x, residual, weight, bias, sum, y, mean, rstd, dm->T, static_cast<int>(dm->d),
                      op->param_dtype == MOE_DTYPE_BF16, op->eps};
  return hip_status(launch_norm(dm->dtype, layer, a, s));
}

size_t moe_norm_backward_workspace_bytes(const moe_dims_t* dm, const moe_norm_opts_t* op) {
  if (check_norm(dm, op) != MOE_OK) return 0;
  return norm_ws(dm, op->kind == MOE_NORM_LAYER, nullptr, nullptr, nullptr, nullptr);
}

int moe_norm_backward(const moe_dims_t* dm, const moe_norm_opts_t* op, const void* dy, const void* xs,
                      const void* weight, const float* mean, const float* rstd, const void* dx_in, void* dx,
                      float* dweight, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_norm(dm, op)) return st;
  const bool layer = op->kind == MOE_NORM_LAYER;
  if (!ok16_or_null(weight) || !ok16_or_null(dweight) || !ok16_or_null(dbias)) return MOE_ERR_INVALID;
  if (!layer && (dbias || mean)) return MOE_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dm->T == 0) {
    StageScope sc(MOE_STAGE_NORM_BWD, s);
    if (dweight)
      if (int st = hip_status(launch_fill_zero(dweight, dm->d, s))) return st;
    return dbias ? hip_status(launch_fill_zero(dbias, dm->d, s)) : MOE_OK;
  }
  if (!ok16(dy) || !ok16(xs) || !ok16(dx) || !ok16_or_null(dx_in) || !ok4(rstd) || (layer && !ok4(mean)))
    return MOE_ERR_INVALID;
  float *pw = nullptr, *pb = nullptr, *shift = nullptr;
  if (dweight || dbias) {
    if (int st = check_ws(ws, ws_bytes, norm_ws(dm, layer, nullptr, nullptr, nullptr, nullptr))) return st;
    norm_ws(dm, layer, ws, &pw, &pb, &shift);
  }
  StageScope sc(MOE_STAGE_NORM_BWD, s);
  const NormGradArgs a = {dy, xs, weight, mean, rstd, dx_in, dx, dweight ? pw : nullptr, dbias ? pb : nullptr,
                          dweight ? shift : nullptr, dm->T, static_cast<int>(dm->d), op->param_dtype == MOE_DTYPE_BF16};
  return hip_status(launch_norm_grad(dm->dtype, layer, a, dweight, dbias, s));
}

size_t moe_grad_norm_workspace_bytes(const moe_grad_t* grads, int32_t count) {
  if (check_grads(grads, count) != MOE_OK) return 0;
  const size_t n = align_up(sizeof(double) * static_cast<size_t>(grad_parts(grads, count)));
  return n ? n : kAlign;
}

int moe_grad_norm(const moe_grad_t* grads, int32_t count, double grad_scale, double max_norm, float* out, void* ws,
                  size_t ws_bytes, void* stream) {
  if (int st = check_grads(grads, count)) return st;
  if (!isfinite(grad_scale) || !(max_norm >= 0.0) || !ok4(out)) return MOE_ERR_INVALID;
  if (int st = check_ws(ws, ws_bytes, sizeof(double) * static_cast<size_t>(grad_parts(grads, count)))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_GRAD_NORM, s);
  double* parts = static_cast<double*>(ws);
  int64_t done = 0;
  const Cut cut = grad_cut(grads, count);
  if (int st = each_grad_table(grads, count, cut, [&](const GradTable& t) {
        const int grid = square_grid(t.chunks);
        const int e = hip_status(launch_square_sums(t, cut.stream, grid, parts + done, s));
        done += grid;
        return e;
      }))
    return st;
  return hip_status(launch_grad_norm(parts, static_cast<int>(done), grad_scale, max_norm, out, s));
}

int moe_adam_step(const moe_adam_opts_t* op, const moe_adam_tensor_t* tensors, const moe_grad_t* grads, int32_t count,
                  const double* lr_step, const float* gscale, const uint64_t* rng, void* stream) {
  if (!op || (op->state_bits != 32 && op->state_bits != 8)) return MOE_ERR_INVALID;
  if (op->stochastic != 0 && op->stochastic != 1) return MOE_ERR_INVALID;
  if (!(op->beta1 >= 0.0 && op->beta1 < 1.0) || !(op->beta2 >= 0.0 && op->beta2 < 1.0)) return MOE_ERR_INVALID;
  if (!(op->eps >= 0x1p-100 && op->eps <= 0x1p100) || !isfinite(op->weight_decay)) return MOE_ERR_INVALID;
  if (lr_step ? !ok8(lr_step) : !isfinite(op->lr) || op->step < 1) return MOE_ERR_INVALID;
  if (!ok4_or_null(gscale) || (rng && !ok8(rng))) return MOE_ERR_INVALID;
  if (!rng && (op->state_bits == 8 || op->stochastic)) return MOE_ERR_INVALID;
  if (int st = check_tensors(tensors, count, op->state_bits, true)) return st;
  if (int st = check_grads(grads, count)) return st;
  Seen seen;
  if (!seen.make(5 * static_cast<size_t>(count) + 1)) return MOE_ERR_HIP;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adam_tensor_t& a = tensors[i];
    if (grads[i].n != a.n) return MOE_ERR_INVALID;
    if (a.n == 0) continue;
    if (seen.again(a.param) || (a.master && seen.again(a.master)) || seen.again(a.m) || seen.again(a.v))
      return MOE_ERR_INVALID;
    if (op->state_bits == 8 && (seen.again(a.m_scale) || seen.again(a.v_scale))) return MOE_ERR_INVALID;
  }
  for (int32_t i = 0; i < count; ++i)
    if (grads[i].n && seen.has(grads[i].grad)) return MOE_ERR_INVALID;

  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_ADAM, s);
  AdamTable t;
  t.count = 0;
  t.chunks = 0;
  t.stochastic = op->stochastic;
  t.lr_step = lr_step;
  t.gscale = gscale;
  t.rng = rng;
  AdamScalars& k = t.k;
  k = {};
  k.beta1 = op->beta1, k.beta2 = op->beta2, k.weight_decay = op->weight_decay;
  k.b1 = static_cast<float>(op->beta1), k.c1 = static_cast<float>(1.0 - op->beta1);
  k.b2 = static_cast<float>(op->beta2), k.c2 = static_cast<float>(1.0 - op->beta2);
  k.eps = static_cast<float>(op->eps);
  if (!lr_step) adam_scalars(k, op->lr, static_cast<double>(op->step));
  const uintptr_t code_align = op->state_bits == 8 ? 8 : 16;
  const Cut cut = cut_of(tensors, count, op->state_bits == 8 ? kCodeChunk : kRound, [&](int32_t i) {
    return 2 * size_of(tensors[i].dtype) + size_of(grads[i].dtype) + (op->state_bits == 8 ? 4 : 16) +
           (tensors[i].master ? 8 : 0);
  });
  t.chunk = cut.chunk;
  int64_t base = 0;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adam_tensor_t& a = tensors[i];
    if (a.n > 0) {
      const int64_t c = chunks_of(a.n, cut.chunk);
      if (t.count == kAdamTensors || (t.count > 0 && t.chunks + c > kListChunks)) {
        if (int st = hip_status(launch_adam(op->state_bits, t, cut.stream, s))) return st;
        t.count = 0;
        t.chunks = 0;
      }
      uint32_t flags = 0;
      if (a.dtype == MOE_DTYPE_BF16) flags |= kAdamParamBf16;
      if (grads[i].dtype == MOE_DTYPE_BF16) flags |= kAdamGradBf16;
      if (aligned(a.param, 16) && aligned(a.master, 16) && aligned(grads[i].grad, 16) && aligned(a.m, code_align) &&
          aligned(a.v, code_align))
        flags |= kAdamAligned;
      t.t[t.count++] = {a.param, a.master, grads[i].grad, a.m, a.v, a.m_scale, a.v_scale, a.n, base, t.chunks, flags};
      t.chunks += static_cast<uint32_t>(c);
    }
    base += (a.n + kScaleBlock - 1) / kScaleBlock * kScaleBlock;
  }
  return t.count ? hip_status(launch_adam(op->state_bits, t, cut.stream, s)) : MOE_OK;
}

int moe_adam_state_values(const moe_adam_tensor_t* tensors, int32_t count, void* const* m_out, void* const* r_out,
                          int out_dtype, void* stream) {
  if (!ok_dtype(out_dtype)) return MOE_ERR_INVALID;
  if (int st = check_tensors(tensors, count, 8, false)) return st;
  if (count > 0 && (!m_out || !r_out)) return MOE_ERR_INVALID;
  Seen seen;
  if (!seen.make(2 * static_cast<size_t>(count) + 1)) return MOE_ERR_HIP;
  for (int32_t i = 0; i < count; ++i)
    if (tensors[i].n && (!ok_elements(m_out[i], out_dtype) || !ok_elements(r_out[i], out_dtype) ||
                         seen.again(m_out[i]) || seen.again(r_out[i])))
      return MOE_ERR_INVALID;
  hipStream_t s = static_cast<hipStream_t>(stream);
  StageScope sc(MOE_STAGE_ADAM, s);
  const Cut cut = cut_of(tensors, count, kCodeChunk, [&](int32_t) { return 2 + 2 * size_of(out_dtype); });
  StateTable t;
  t.count = 0;
  t.chunks = 0;
  t.chunk = cut.chunk;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adam_tensor_t& a = tensors[i];
    if (a.n == 0) continue;
    const int64_t c = chunks_of(a.n, cut.chunk);
    if (t.count == kStateTensors || (t.count > 0 && t.chunks + c > kListChunks)) {
      if (int st = hip_status(launch_state_values(out_dtype, t, cut.stream, s))) return st;
      t.count = 0;
      t.chunks = 0;
    }
    const bool al = aligned(m_out[i], 16) && aligned(r_out[i], 16) && aligned(a.m, 8) && aligned(a.v, 8);
    t.t[t.count++] = {static_cast<const uint8_t*>(a.m), static_cast<const uint8_t*>(a.v), a.m_scale, a.v_scale,
                      m_out[i], r_out[i], a.n, t.chunks, al ? 1u : 0u};
    t.chunks += static_cast<uint32_t>(c);
  }
  return t.count ? hip_status(launch_state_values(out_dtype, t, cut.stream, s)) : MOE_OK;
}

}  // extern "C"

// Host-side launchers of what a training step needs around the layer: the norm
// in front of it, the gradients' 2-norm and the AdamW update (internal to the
// library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// ---------------- norm ----------------
// Most columns of a row: a workgroup of 1024 threads keeps a row, its weights and
// its columns' gradients in registers, 16 columns to a thread.
constexpr int64_t kNormMaxCols = 16384;

struct NormArgs {
  const void* x;         // [T][d]
  const void* residual;  // [T][d] or null
  const void* w;         // [d] or null (1)
  const void* b;         // [d] or null (0)
  void* sum;             // [T][d] or null
  void* y;               // [T][d]
  float* mean;           // [T] or null
  float* rstd;           // [T] or null
  int64_t T;
  int d;
  int w_bf16;            // type of w and b
  float eps;
};
hipError_t launch_norm(int dtype, bool layer, const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void* dy;     // [T][d]
  const void* x;      // [T][d]: what the forward normalised
  const void* w;      // [d] or null (1)
  const float* mean;  // [T] (layer norm)
  const float* rstd;  // [T]
  const void* dx_in;  // [T][d] or null
  void* dx;           // [T][d]
  float* part_w;      // [parts][d] or null (no weight gradient)
  float* part_b;      // [parts][d] or null
  float* shift;       // [T] or null (norm_grad_shifts)
  int64_t T;
  int d;
  int w_bf16;
};
// Parts that dweight and dbias are summed from, 0 where they are summed beside the rows.
int norm_grad_parts(int dtype, int64_t T, int64_t d);
// Whether dweight of these rows takes [T] of what each row's h is off by.
bool norm_grad_shifts(int dtype, bool layer, int64_t T, int64_t d);
hipError_t launch_norm_grad(int dtype, bool layer, const NormGradArgs& a, float* dw, float* db, hipStream_t s);

// ---------------- lists of tensors ----------------
// A launch takes its tensors by value, as many as kernel arguments hold, so no list
// is copied to the device and a captured graph holds its own.
constexpr size_t kArgBytes = 4096;
constexpr int kAdamTensors = 49;
constexpr int kGradTensors = 169;
constexpr int kStateTensors = 63;
// Elements of a workgroup's turn, rounds of 2048 of its 256 threads: one round for
// the update with 32-bit states, and where more leave compute units without a
// workgroup (measured on 1.1 M fp32 weights in 40 tensors: 8.4 and 10.4 us).
constexpr int kRound = 2048, kListChunk = 4 * kRound, kCodeChunk = 2 * kRound;
constexpr int64_t kListSmall = int64_t(1) << 23;     // elements of a list up to which a turn is one round
constexpr int64_t kListStream = int64_t(128) << 20;  // bytes of a list from which it streams past the cache
constexpr int64_t kListElements = int64_t(1) << 36;  // of one gradient at most
constexpr int64_t kAdamElements = int64_t(1) << 34;  // of one parameter: kListChunks rounds
constexpr int64_t kListChunks = int64_t(1) << 23;    // of one launch at most (fewer than 2^32 threads)
static_assert(kAdamElements / kRound <= kListChunks, "a tensor's turns fit a launch");
constexpr int kScaleBlock = 128;   // elements per scale of the 8-bit states

struct GradEntry {
  const void* g;
  int64_t n;
  uint32_t first;  // chunks of the launch's tensors before this one
  uint32_t flags;  // 1 bf16, 2 aligned for wide loads
};
struct GradTable {
  GradEntry t[kGradTensors];
  int count;
  uint32_t chunks;
  int chunk;       // elements of one
};
// Sums of squares of a table's tensors into parts [grid] (double).
constexpr int kNormGrid = 2048;    // workgroups (parts) of one launch at most
hipError_t launch_square_sums(const GradTable& t, bool stream, int grid, double* parts, hipStream_t s);
hipError_t launch_grad_norm(const double* parts, int n, double scale, double max_norm, float* out, hipStream_t s);

struct AdamEntry {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  int64_t base;     // the tensor's first element in the list's numbering
  uint32_t first;   // chunks of the launch's tensors before this one
  uint32_t flags;   // kAdam*
};
constexpr uint32_t kAdamParamBf16 = 1, kAdamGradBf16 = 2, kAdamAligned = 4;
struct AdamScalars {
  double lr, beta1, beta2, weight_decay;
  double step;           // 1-based
  float b1, c1, b2, c2;  // beta, 1 - beta
  float eps;
  float step_size;       // lr / (1 - beta1^step)
  float inv_root;        // 1 / sqrt(1 - beta2^step)
  float decay;           // lr * weight_decay
};
struct AdamTable {
  AdamEntry t[kAdamTensors];
  int count;
  uint32_t chunks;
  int chunk;
  int stochastic;           // bf16 parameters without master weights rounded stochastically
  const double* lr_step;    // device {lr, step} or null
  const float* gscale;      // device [1] or null
  const uint64_t* rng;      // device {seed, offset} or null
  AdamScalars k;
};
// (beside the gradients' table the kernel takes a pointer)
static_assert(sizeof(AdamTable) <= kArgBytes && sizeof(GradTable) + 8 <= kArgBytes, "kernel arguments");
static_assert(sizeof(AdamTable) + sizeof(AdamEntry) > kArgBytes && sizeof(GradTable) + 8 + sizeof(GradEntry) > kArgBytes,
              "as many as they hold");

// The scalars that depend on lr and step; the kernels form them alike from lr_step.
__host__ __device__ inline double pow_step(double b, double step) {
#pragma clang fp contract(off)
  // squarings: an error of about step * 2^-53, and b^step is 0 long before that counts
  uint64_t e = step < 1.0 ? 0 : step < 9.0e15 ? static_cast<uint64_t>(step) : uint64_t(9000000000000000);
  double r = 1.0;
  while (e) {
    if (e & 1) r = r * b;
    b = b * b;
    e >>= 1;
  }
  return r;
}
__host__ __device__ inline void adam_scalars(AdamScalars& k, double lr, double step) {
#pragma clang fp contract(off)
  k.step_size = static_cast<float>(lr / (1.0 - pow_step(k.beta1, step)));
  k.inv_root = static_cast<float>(1.0 / __builtin_sqrt(1.0 - pow_step(k.beta2, step)));
  k.decay = static_cast<float>(lr * k.weight_decay);
}
hipError_t launch_adam(int bits, const AdamTable& t, bool stream, hipStream_t s);

// What 8-bit states stand for.
struct StateEntry {
  const uint8_t* m;
  const uint8_t* v;
  const uint8_t* ms;
  const uint8_t* vs;
  void* m_out;
  void* r_out;
  int64_t n;
  uint32_t first;
  uint32_t aligned;
};
struct StateTable {
  StateEntry t[kStateTensors];
  int count;
  uint32_t chunks;
  int chunk;
};
static_assert(sizeof(StateTable) <= kArgBytes && sizeof(StateTable) + sizeof(StateEntry) > kArgBytes, "kernel arguments");
hipError_t launch_state_values(int out_dtype, const StateTable& t, bool stream, hipStream_t s);

}  // namespace moe

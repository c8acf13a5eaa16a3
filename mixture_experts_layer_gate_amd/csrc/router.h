// Host-side launchers of the scored router's kernels, its losses and gradients,
// and the dropout beside the combine (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Selection options as the kernels take them (include/moe.h, moe_route_opts_t).
struct SelectOpts {
  int sigmoid;      // scores: 1 sigmoid, 0 softmax
  int groups;       // expert groups (1: none)
  int topk_groups;  // groups kept
  int top2;         // group key: 1 sum of its two largest keys, 0 its largest
  int renorm;       // weights divided by their sum
  float scale;      // weight factor
  int per;          // experts per group
  int lpg_log2;     // log2 of the wave lanes that scan one group: the most that 64 / groups allows
  float inv_per;    // 1 / per
};
constexpr int kMaxGroups = 64;   // one wave lane per group
constexpr int kMaxSeqs = 65535;  // one grid row per sequence

hipError_t launch_select(const SelectOpts& o, const float* logits, const float* balance_bias, int64_t T, int E, int k,
                         int32_t* idx, float* w, hipStream_t s);
// losses' gradient: dlosses non-null adds it (load [S][E], seq_offsets [S+1] or null for one sequence of T)
hipError_t launch_select_backward(const SelectOpts& o, const float* logits, const int32_t* idx, const float* w,
                                  const float* dw, const float* dlosses, const int32_t* load,
                                  const int32_t* seq_offsets, int n_seq, int64_t T, int E, int k, float* dlogits,
                                  hipStream_t s);

// Balance losses: row parts per sequence, and the workspace pieces they need.
int balance_parts(int64_t T, int n_seq, int E);
int balance_blocks(int E);  // expert blocks of the part reduction
hipError_t launch_balance(const SelectOpts& o, const float* logits, const int32_t* idx, const int32_t* seq_offsets,
                          int n_seq, int64_t T, int E, int k, int parts, float* part_p, int32_t* part_f,
                          double* part_z, double* term, uint32_t* done, float* losses, int32_t* load, hipStream_t s);

// Dropout: an element is kept when its 16-bit number is at least thr, and then
// scaled (scale 0 with thr 65536: everything is dropped). rng: {seed, offset},
// read by the kernel from device memory.
struct DropArgs {
  const uint64_t* rng;
  uint32_t thr;
  float scale;
};
hipError_t launch_combine_dropout(int dtype, const DropArgs& a, const void* y, const int32_t* inv_perm, const float* w,
                                  const void* residual, void* out, int64_t T, int64_t d, int k, hipStream_t s);
hipError_t launch_dropout_backward(int dtype, const DropArgs& a, const void* dout, void* dy, int64_t T, int64_t d,
                                   hipStream_t s);

// Gate gradients (bf16 x and wg, fp32 dlogits). ws: gate_backward_ws bytes.
// T in grid rows of 64 tokens, 32-bit row offsets of d, and one launch of 128 x 128 tiles.
inline bool gate_backward_fits(int64_t T, int64_t d) {
  return T <= 65534 * int64_t(64) && d <= (int64_t(1) << 24) && (T / 128 + 1) * (d / 128 + 1) < (int64_t(1) << 23);
}
size_t gate_backward_ws(int64_t T, int64_t d, int E);
hipError_t launch_gate_backward(const void* x, const void* wg, const float* dlogits, const void* dx_in, void* dx,
                                float* dwg, float* dbias, int64_t T, int64_t d, int E, void* ws, hipStream_t s);

}  // namespace moe

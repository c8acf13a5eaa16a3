// Host-side checks of the scored router's and the dropout's entry points for a
// build whose host code is instrumented with AddressSanitizer and
// UndefinedBehaviorSanitizer. Every call returns before anything is enqueued;
// device pointers are placeholders that are never dereferenced, so the program
// refuses to run where a GPU is visible. Exit status 0 when every status code is
// the expected one.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "moe.h"

static int failures = 0;
#define EXPECT(call, want)                                                                 \
  do {                                                                                     \
    const long long got_ = static_cast<long long>(call);                                   \
    if (got_ != static_cast<long long>(want)) {                                            \
      fprintf(stderr, "line %d: %s returned %lld, expected %lld\n", __LINE__, #call, got_, \
              static_cast<long long>(want));                                               \
      ++failures;                                                                          \
    }                                                                                      \
  } while (0)

static moe_dims_t dims(int64_t T, int64_t d, int32_t E, int32_t k, int32_t dtype = MOE_DTYPE_BF16) {
  moe_dims_t m;
  m.T = T, m.d = d, m.f = 256, m.E = E, m.k = k, m.dtype = dtype;
  return m;
}

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    printf("a GPU is visible: the host-only checks do not run here\n");
    return 0;
  }
  void* const A = reinterpret_cast<void*>(uintptr_t(0x10000));
  float* const F = static_cast<float*>(A);
  int32_t* const I = static_cast<int32_t*>(A);
  const uint64_t* const R = static_cast<const uint64_t*>(A);
  const size_t BIG = size_t(1) << 60;
  moe_route_opts_t ok = {MOE_SCORE_SIGMOID, 8, 4, MOE_GROUP_TOP2, 1, 2.5f};
  const moe_dims_t one = dims(64, 256, 256, 8);

  // sizes: growing, and 0 for what the calls refuse; extreme dims on the way
  for (int64_t T : {int64_t(0), int64_t(1), int64_t(4096), int64_t(1) << 22, int64_t(1) << 30, int64_t(1) << 62})
    for (int64_t d : {int64_t(8), int64_t(7168), int64_t(1) << 24, int64_t(1) << 30, int64_t(1) << 40})
      for (int32_t E : {1, 8, 64, 65, 1024, 1025, -5})
        for (int32_t n : {-1, 0, 1, 7, 65535, 65536, INT32_MAX}) {
          const moe_dims_t m = dims(T, d, E, 1);
          const size_t b = moe_balance_workspace_bytes(&m, n), g = moe_gate_backward_workspace_bytes(&m);
          // (dims whose layer workspace could not be counted in size_t are invalid as well)
          const bool good = T < (int64_t(1) << 31) && d < (int64_t(1) << 31) && E >= 1 && E <= 1024 &&
                            T * (E > 0 ? E : 1) < (int64_t(1) << 31) &&
                            !(T >= (int64_t(1) << 30) && d >= (int64_t(1) << 30));
          if (!good && (b || g)) ++failures;
          if ((n < 1 || n > 65535) && b) ++failures;
          if (good && n >= 1 && n <= 65535 && !b) ++failures;
        }
  EXPECT(moe_balance_workspace_bytes(nullptr, 1), 0);
  EXPECT(moe_gate_backward_workspace_bytes(nullptr), 0);

  // options
  for (int q = 0; q < 9; ++q) {
    moe_route_opts_t o = ok;
    switch (q) {
      case 0: o.score = 9; break;
      case 1: o.groups = 0; break;
      case 2: o.groups = 65; break;
      case 3: o.groups = INT32_MIN; break;
      case 4: o.topk_groups = INT32_MAX; break;
      case 5: o.topk_groups = -1; break;
      case 6: o.group_rule = -1; break;
      case 7: o.renormalise = 5; break;
      default: o.scale = NAN;
    }
    EXPECT(moe_route_select(&one, &o, F, nullptr, I, F, nullptr), MOE_ERR_INVALID);
    EXPECT(moe_balance_loss(&one, &o, F, I, nullptr, 1, F, I, A, BIG, nullptr), MOE_ERR_INVALID);
    EXPECT(moe_route_select_backward(&one, &o, F, I, F, F, nullptr, nullptr, nullptr, 1, F, nullptr), MOE_ERR_INVALID);
    EXPECT(moe_route_scored(&one, &o, A, A, nullptr, nullptr, F, I, F, nullptr), MOE_ERR_INVALID);
  }
  EXPECT(moe_route_select(nullptr, &ok, F, nullptr, I, F, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_route_select(&one, &ok, nullptr, nullptr, I, F, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_balance_loss(&one, &ok, F, I, I, INT32_MAX, F, I, A, BIG, nullptr), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_balance_loss(&one, &ok, F, I, I, INT32_MIN, F, I, A, BIG, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_balance_loss(&one, &ok, F, I, I, 4, F, I, A, 1, nullptr), MOE_ERR_WORKSPACE);
  EXPECT(moe_gate_backward(&one, A, A, F, nullptr, A, F, F, A, 1, nullptr), MOE_ERR_WORKSPACE);
  const moe_dims_t wide = dims(1 << 20, int64_t(1) << 24, 8, 1);
  EXPECT(moe_gate_backward(&wide, A, A, F, nullptr, A, F, F, A, BIG, nullptr), MOE_ERR_UNSUPPORTED);
  for (double p : {-1e-9, 1.0000001, double(NAN), double(INFINITY)}) {
    EXPECT(moe_combine_dropout(&one, p, R, A, I, F, nullptr, A, nullptr), MOE_ERR_INVALID);
    EXPECT(moe_dropout_backward(&one, p, R, A, A, nullptr), MOE_ERR_INVALID);
  }
  if (failures) fprintf(stderr, "%d failures\n", failures);
  return failures ? 1 : 0;
}
